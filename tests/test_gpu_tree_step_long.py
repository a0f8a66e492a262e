"""Tree steps of a model with heads of 64 over a long context: the kernels that cut
pairs into shares and the tcgen05 one, between the model's products, one workspace
for all layers; eagerly and in a graph.

The weights' queries and keys are drawn larger than GPT-2's, so that a row of
attention depends on what it sees.  Tolerance: a step's logits stand to the oracle's as
those of gpt2_decode_step_paged over the same tokens do, which differ by the order of
fp32 sums alone: their own errors are taken on the same rows.  Twice the largest and
1e-4 (fp32's bound) for the tree's against the oracle; five times (both sides' errors,
and a maximum over some thirty times as many rows, which for errors of one distribution
is less than half as large again) and 1e-4 between the two."""
import functools

import numpy as np
import pytest
import torch

import oracle
from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import inputs
from gpt_transformer_forward_gb300.runner import GPT2Model

from draft_reference import paths, trees
from gpu_helpers import dev, host, need_gpu, no_device_error

pytestmark = pytest.mark.gpu
ALL = [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16]
NAMES = {v: k for k, v in ab.PRECISIONS.items()}
CFG = inputs.GPT2Config(max_seq_len=2304, vocab_size=500, padded_vocab_size=512, num_layers=2, num_heads=2, channels=128)
BS, MOST, DEEP = 32, 2304 - 64, 6
V = CFG.vocab_size


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@functools.lru_cache(None)
def weights():
    flat = inputs.make_params(CFG, 31, "perturbed")
    v, C = inputs.param_views(CFG, flat), CFG.channels
    v["qkvw"][:, :2 * C] *= 6  # scores of a standard deviation of about 2
    v["qkvw"][:, 2 * C:] *= 4
    v["attprojw"][:] *= 8
    return flat


@functools.lru_cache(None)
def case(B, N):
    """prompts [B, MOST], lengths, who has a tree, parents, tokens, and of each
    sequence the first nodes of its deepest path."""
    rng = np.random.default_rng(100 * B + N)
    prompt = rng.integers(0, V, (B, MOST)).astype(np.int32)
    lens = rng.integers(0, MOST + 1, B).astype(np.int32)
    lens[0], lens[1], lens[-1] = MOST, 1500, 0
    parent = trees(B, N, seed=N, missing=True)
    parent[:3] = trees(3, N, seed=N + 1, missing=False)
    parent[:, 0] = -1
    tok = rng.integers(0, V, (B, N)).astype(np.int32)
    idle = rng.random(B) < 0.15
    idle[:3] = idle[-1] = False
    idle[3] = True
    deepest = [max(paths(p)[0], key=len)[:DEEP] for p in parent]
    return prompt, lens, idle, parent, tok, deepest


@functools.lru_cache(None)
def exact(B, N, b, other=0):
    """The oracle's logits behind the nodes of the deepest path of sequence b; with
    another sequence's first tokens, `other` of them."""
    prompt, lens, _, _, tok, deepest = case(B, N)
    seq = np.concatenate([prompt[b, :lens[b]], tok[b, deepest[b]]])[None].astype(np.int32)
    seq[0, :other] = prompt[B - 1, :other]
    return oracle.forward(CFG, weights(), seq, want_probs=False)[0][0, lens[b]:, :V]


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("B,N", [(6, 64), (80, 16), (80, 20), (7, 5)])
def test_a_step_over_a_long_context(precision, B, N):
    prompt, lens, idle, parent, tok, deepest = case(B, N)
    m = GPT2Model(CFG, weights(), B, MOST, precision)
    rng = np.random.default_rng(1)
    maxb = CFG.max_seq_len // BS
    num_blocks = B * maxb + 3
    table = dev(rng.permutation(num_blocks)[:B * maxb].reshape(B, maxb).astype(np.int32))
    pool = m.new_paged_kvcache(num_blocks, BS)
    kv = ab.paged_kv(pool, table, num_blocks, BS, maxb)
    lg, _ = m.new_outputs(B, MOST, probs=False)
    m.prefill_paged(dev(prompt), lg, kv)
    del lg
    before = pool.clone()

    # token by token along one path of each sequence
    other = pool.clone()
    kv2 = ab.paged_kv(other, table, num_blocks, BS, maxb)
    one, _ = m.new_outputs(B, None, probs=False)
    paged = []
    for k in range(DEEP):
        t = np.array([tok[b, d[min(k, len(d) - 1)]] for b, d in enumerate(deepest)], np.int32)
        m.decode_step_paged(kv2, dev(t), dev(lens + k), one)
        paged.append(host(one)[:, :V])

    pos = np.where(idle, -1, lens).astype(np.int32)
    logits, _ = m.new_outputs(B, N, probs=False)
    ws = m.new_tree_workspace(B, N)
    ws.fill_(255)  # NaN bytes
    t, p, par = dev(tok), dev(pos), dev(parent)
    m.decode_step_tree(kv, t, p, logits, ws, parent=par)
    got = host(logits)[:, :, :V]
    no_device_error()

    worst = 0.0
    for b in (0, 1, 2, B - 1):
        for k in range(len(deepest[b])):
            worst = max(worst, np.abs(paged[k][b] - exact(B, N, b)[k]).max())
    for b in (0, 1, 2, B - 1):
        for k, i in enumerate(deepest[b]):
            err = np.abs(got[b, i] - exact(B, N, b)[k]).max()
            assert err <= 2 * worst + 1e-4, (b, k, err, worst)
    for b in range(B):
        for k, i in enumerate(deepest[b]):
            if not idle[b]:
                err = np.abs(got[b, i] - paged[k][b]).max()
                assert err <= 5 * worst + 1e-4, (b, k, err, worst)
    # (the bounds are below what a seventh of the cached positions changes)
    assert np.abs(exact(B, N, 0, 300)[-1] - exact(B, N, 0)[-1]).max() > 10 * worst + 2e-4

    # nothing but the nodes' rows of sequences with a tree has changed
    a, z = (x.view(CFG.num_layers, 2, num_blocks, CFG.num_heads, BS, -1) for x in (before, pool))
    rows = (a != z).any(-1).any(0).any(0).any(1).cpu().numpy()
    may = np.zeros_like(rows)
    tab = table.cpu().numpy()
    for b in range(B):
        for i, path in enumerate(paths(parent[b])[0]):
            if path and not idle[b]:
                may[tab[b, (lens[b] + i) // BS], (lens[b] + i) % BS] = True
    assert not (rows & ~may).any() and rows[may].all()

    # the same in a graph, over another state of the buffers it was captured with
    after = pool.clone()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    state = [torch.zeros_like(x) for x in (t, p, par)]
    state[1].fill_(-1)
    out = torch.zeros_like(logits)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        m.decode_step_tree(kv, state[0], state[1], out, ws, parent=state[2], stream=s)
    torch.cuda.synchronize()
    pool.copy_(before)
    ws.fill_(127)
    for x, y in zip(state, (t, p, par)):
        x.copy_(y)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    there = dev(np.array([[bool(q) and not idle[b] for q in paths(parent[b])[0]] for b in range(B)]))
    assert torch.equal(out[there], logits[there]) and torch.equal(pool, after)
    no_device_error()
