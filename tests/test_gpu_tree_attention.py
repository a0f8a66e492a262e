"""Attention of trees of drafted tokens over a paged cache [NTU "KV Caching";
FlashAttention Algorithm 0], against a 64-bit form on the CPU that walks each
node's path.

Tolerances: u = 2^-24, w the half step of the element type (relative 2^-8 for
bf16, 2^-11 for fp16; u for fp32).  A score of hs products is off by at most
(hs + 4) u sum|q k| / sqrt(hs) (products, sums, scale and the log2 units), a
probability relative to the row's sum by twice that, the exponential's 8 u and
the sums' (n / 16 + 64) u over n positions; an output by that times max|v|, plus
2^-15 max|v| (bf16) or 2^-22 max|v| (fp16) for probabilities as sums of two
16-bit values, n 2^-25 max|v| for fp16 values below its smallest step, and w |out|
(at least fp16's half smallest step, 2^-25) for the output's own rounding."""
import numpy as np
import pytest
import torch

import oracle
from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import inputs
from gpt_transformer_forward_gb300.runner import GPT2Model

from draft_reference import chain, paths, tree_attention, trees
from gpu_helpers import assert_close, dev, host, need_gpu, no_device_error

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
DT = {ab.GPT2_FP32: torch.float32, ab.GPT2_TF32: torch.float32, ab.GPT2_BF16: torch.bfloat16,
      ab.GPT2_FP16: torch.float16}
HALF = {torch.float32: u, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SPLIT = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -22}
ALL = [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16]
NAMES = {v: k for k, v in ab.PRECISIONS.items()}
TYPES = [ab.GPT2_FP32, ab.GPT2_BF16, ab.GPT2_FP16]
IDS = [NAMES[p] for p in TYPES]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(precision, N, NH, hs, pos, bs, parent, seed, qscale=2.0, spare=2):
    """Inputs as CPU tensors; every sequence has blocks for pos + N positions."""
    g = torch.Generator().manual_seed(seed)
    dt, pos = DT[precision], np.asarray(pos, np.int32)
    B = len(pos)
    row = (max(0, int(pos.max())) + N - 1) // bs + 1
    num_blocks = B * row + 3
    table = torch.full((B, row + spare), -5, dtype=torch.int32)  # entries no call reaches
    table[:, :row] = torch.randperm(num_blocks, generator=g)[:B * row].view(B, row)
    pool = torch.randn(2, num_blocks, NH, bs, hs, generator=g).to(dt)
    qkv = torch.randn(B * N, 3, NH, hs, generator=g)
    qkv[:, 0] *= qscale
    return dict(precision=precision, N=N, NH=NH, hs=hs, bs=bs, pool=pool, table=table, pos=torch.from_numpy(pos.copy()),
                parent=None if parent is None else torch.from_numpy(np.ascontiguousarray(parent)),
                qkv=qkv.reshape(B * N, -1).to(dt))


def call(c, t, out, ws=None, stream=None):
    B, C = c["pos"].shape[0], c["NH"] * c["hs"]
    n = ab.attention_tree_workspace_size(B, c["N"], C, c["NH"], c["precision"])
    if ws is None:
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN bytes
    kv = ab.paged_kv(t["pool"], t["table"], c["pool"].shape[1], c["bs"], c["table"].shape[1])
    ab.attention_tree(out, t["qkv"], kv, t["pos"], t["parent"], B, c["N"], C, c["NH"], c["precision"], ws, n, stream)
    return ws


def on_gpu(c):
    return {k: None if c[k] is None else c[k].cuda() for k in ("pool", "qkv", "table", "pos", "parent")}


def run(c):
    t = on_gpu(c)
    B, N, C = c["pos"].shape[0], c["N"], c["NH"] * c["hs"]
    out = torch.full((B * N + 2, C), 9.0, dtype=DT[c["precision"]], device="cuda")
    call(c, t, out[1:-1])
    torch.cuda.synchronize()
    assert (out[0] == 9).all() and (out[-1] == 9).all(), "rows around the output"
    return out[1:-1].cpu().view(B, N, c["NH"], c["hs"]), t["pool"].cpu()


def parents(c):
    B = c["pos"].shape[0]
    return chain(B, c["N"]) if c["parent"] is None else c["parent"].numpy()


def reference(c):
    B, N, NH, hs = c["pos"].shape[0], c["N"], c["NH"], c["hs"]
    q, k, v = c["qkv"].double().numpy().reshape(B, N, 3, NH, hs).transpose(2, 0, 1, 3, 4)
    cap = c["table"].shape[1] * c["bs"]
    out, sabs, vmax, n, there = tree_attention(q, k, v, c["pool"].double().numpy(), c["table"].numpy(),
                                               c["pos"].numpy(), parents(c), c["bs"], cap)
    dt = DT[c["precision"]]
    n = n[..., None]
    part = 2 * (hs + 4) * u * sabs + 8 * u + (n / 16 + 64) * u + SPLIT[dt]
    if dt == torch.float16:
        part = part + n * 2.0 ** -25
    tol = (part * vmax)[..., None] + HALF[dt] * np.abs(out)
    return out, tol + (2.0 ** -25 if dt == torch.float16 else 0), there


def cache_after(c):
    want, cap = c["pool"].clone(), c["table"].shape[1] * c["bs"]
    B, N = c["pos"].shape[0], c["N"]
    kv = c["qkv"].view(B, N, 3, c["NH"], c["hs"])
    for b in range(B):
        p = int(c["pos"][b])
        if 0 <= p < cap:
            for i, path in enumerate(paths(parents(c)[b], cap - p)[0]):
                blk = int(c["table"][b, (p + i) // c["bs"]]) if path else -1
                if 0 <= blk < want.shape[1]:
                    want[:, blk, :, (p + i) % c["bs"]] = kv[b, i, 1:]
    return want


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check(c):
    out, pool = run(c)
    ref, tol, there = reference(c)
    err = np.abs(out.double().numpy() - ref)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} off, worst {np.nanmax(err / np.maximum(tol, 1e-30)):.3f} of the tolerance"
    assert (out.numpy() if out.dtype != torch.bfloat16 else out.float().numpy())[~there].any() == False  # noqa: E712
    assert same(pool, cache_after(c)), "the cache"
    return out


def ragged(B, most, seed):
    pos = np.random.default_rng(seed).integers(0, most + 1, B)
    pos[0] = most
    pos[-1] = 0 if B > 1 else most
    if B > 3:
        pos[1] = -1
    return pos


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("hs", [16, 32, 64])
@pytest.mark.parametrize("B,N,NH,most,bs", [
    (1, 1, 1, 0, 1), (1, 1, 2, 1, 2), (2, 2, 3, 63, 1), (3, 5, 1, 64, 16), (5, 8, 2, 65, 128), (4, 9, 3, 200, 8),
    (7, 16, 2, 129, 4), (3, 17, 2, 500, 16), (2, 31, 3, 127, 32), (3, 32, 1, 128, 64), (2, 33, 2, 191, 16),
    (3, 48, 2, 70, 2), (2, 63, 1, 1, 16), (5, 64, 2, 321, 32), (1, 64, 1, 64, 16), (1, 7, 1, 6000, 64),
    (33, 3, 2, 90, 16), (70, 4, 12, 40, 8),
])
def test_against_64_bits(precision, hs, B, N, NH, most, bs):
    check(make(precision, N, NH, hs, ragged(B, most, N), bs, trees(B, N, seed=B + N, roots=True), seed=B + N))
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("N", [1, 16, 40, 64])
def test_chains(precision, N):
    c = make(precision, N, 2, 64, [100, 0, 63, 64, 1000], 16, None, seed=N)
    a = check(c)
    b = check(dict(c, parent=torch.from_numpy(chain(5, N))))
    assert same(a, b)
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("B,N,NH,most", [(40, 16, 12, 300), (1, 20, 2, 20000), (6, 64, 3, 4000), (600, 2, 1, 150)])
def test_shares(precision, B, N, NH, most):
    """Few pairs over many shares, many pairs over few tiles each."""
    check(make(precision, N, NH, 64, ragged(B, most, B), 64, trees(B, N, seed=B), seed=B))
    no_device_error()


# Tables that could hold more positions than a CTA takes by itself: pairs are cut
# into shares, of which a few hold many pairs and many hold none.
@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("hs", [16, 32, 64])
@pytest.mark.parametrize("B,N,NH,most,bs", [
    (1, 1, 1, 0, 16), (1, 5, 3, 33, 8), (3, 8, 2, 700, 16), (6, 16, 4, 300, 32), (4, 17, 3, 65, 4), (3, 32, 2, 900, 64),
    (2, 33, 2, 130, 4), (3, 64, 3, 640, 16),
])
def test_short_pairs_in_long_tables(precision, hs, B, N, NH, most, bs):
    c = make(precision, N, NH, hs, ragged(B, most, N), bs, trees(B, N, seed=B + N, roots=True), seed=B, spare=2100 // bs)
    check(c)
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("B,N,NH,hs,most,spare", [
    (500, 3, 4, 16, 90, 40), (300, 12, 8, 16, 40, 40), (330, 20, 3, 32, 70, 40), (160, 40, 3, 16, 70, 40),
    (40, 64, 12, 64, 100, 40), (90, 40, 2, 32, 70, 2), (90, 20, 2, 64, 200, 2), (90, 50, 2, 64, 200, 2),
])
def test_more_pairs_than_shares(precision, B, N, NH, hs, most, spare):
    """Every share holds the ends of several pairs; and as many CTAs as pairs."""
    check(make(precision, N, NH, hs, ragged(B, most, B), 64, trees(B, N, seed=B), seed=B, spare=spare))
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("spare", [2, 140])
@pytest.mark.parametrize("N", [3, 12, 20, 40, 64])
def test_sequences_without_a_tree(precision, N, spare):
    """At the ends, between others, most of them, all of them; some at positions
    that are none."""
    def take(pos):
        c = make(precision, N, 3, 64, [min(max(p, -1), 700) for p in pos], 16, trees(len(pos), N, seed=N), seed=N, spare=spare)
        c["pos"] = torch.tensor(pos, dtype=torch.int32)
        return check(c)
    take([-1, 300, -1, -1, 0, 64, -1, 700, -1])
    take([5, -1, -1, -1, -1, -1, -1, -1, 130])
    assert not take([-1] * 70).any()
    no_device_error()
    out = take([-1, 300, -2, 2**31 - 1, 40, -2**31])
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION
    some = (trees(6, N, seed=N) != -2).any(1)  # (a drawn tree may have no node at all)
    assert [bool(o.any()) for o in out] == [False, some[1], False, False, some[4], False]


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_many_sequences_without_a_tree(precision):
    """More pairs than shares, most of them without a step."""
    for N, hs in ((4, 16), (20, 32), (64, 64)):
        pos = np.where(np.random.default_rng(N).random(400) < 0.7, -1, ragged(400, 90, N))
        check(make(precision, N, 5, hs, pos, 64, trees(400, N, seed=N), seed=N, spare=40))
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("bs", [1, 2, 4, 8, 128])
@pytest.mark.parametrize("long", [False, True])
def test_wide_trees_over_small_blocks(precision, bs, long):
    spare = 900 // bs - 349 // bs - 1 if long else 2  # tables of 900 positions
    check(make(precision, 50, 2, 64, [300, 0, -1, 127, 128, 1], bs, trees(6, 50, seed=bs, roots=True), seed=bs, spare=spare))
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_calls_behind_each_other_in_one_workspace(precision):
    """Larger and smaller trees, without a wait between them: each finds what the
    others left."""
    cs = [make(precision, N, 4, 64, ragged(B, most, N), 16, trees(B, N, seed=N), seed=N, spare=spare)
          for B, N, most, spare in [(5, 64, 500, 2), (9, 5, 900, 140), (3, 20, 300, 140), (7, 8, 200, 2), (4, 40, 700, 2)]]
    want = [run(c) for c in cs]
    ws = torch.full((max(ab.attention_tree_workspace_size(1, c["N"], 256, 4, precision) for c in cs),), 255,
                    dtype=torch.uint8, device="cuda")
    ts = [on_gpu(c) for c in cs]
    outs = [torch.empty(o.shape[0] * o.shape[1], 256, dtype=o.dtype, device="cuda") for o, _ in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, t, out in zip(cs, ts, outs):
            call(c, t, out, ws, stream=s)
    s.synchronize()
    for (o, p), out, t in zip(want, outs, ts):
        assert same(out.cpu().view(o.shape), o) and same(t["pool"].cpu(), p)
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_same_bits_again(precision):
    c = make(precision, 24, 4, 64, ragged(9, 900, 1), 16, trees(9, 24, seed=1), seed=1)
    a, b = run(c), run(c)
    assert same(a[0], b[0]) and same(a[1], b[1])


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_peaked_and_rising_scores(precision):
    """Scores that grow along the cache, one that dominates, and a first node
    that dominates all."""
    c = make(precision, 12, 2, 64, [900, 900, 130], 16, trees(3, 12, seed=5), seed=4, qscale=1.0)
    c["qkv"].view(3, 12, 3, 2, 64)[:, :, 0, 0] = 1.0
    for j in range(900):
        c["pool"][0, c["table"][0, j // 16].long(), 0, j % 16] = (0.2 + 7.8 * j / 900)
    c["pool"][0, c["table"][1, 850 // 16].long(), 1, 850 % 16] *= 6
    c["qkv"].view(3, 12, 3, 2, 64)[2, 0, 1] *= 8
    check(c)
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("N", [6, 30, 64])
@pytest.mark.parametrize("hs,spare", [(32, 2), (32, 140), (64, 2), (64, 140)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_unseen_values_stay_out(precision, N, hs, spare, value):
    """NaN and infinities in cache slots that no position reaches, in the rows of
    missing nodes, and in one node's key and value: only the rows behind it may
    change."""
    for pos in ([70, 0, 200], [61, 3, 128]):
        parent = trees(3, N, seed=N, missing=False)
        parent[0, N // 2] = -2
        c = make(precision, N, 2, hs, pos, 16, parent, seed=N, spare=spare)
        good = check(c)
        kv = c["qkv"].view(3, N, 3, 2, hs)
        used = torch.zeros(c["pool"].shape[1], 16, dtype=torch.bool)
        for b in range(3):
            for j in range(pos[b]):
                used[c["table"][b, j // 16].long(), j % 16] = True
        c["pool"].permute(1, 3, 0, 2, 4)[~used] = value
        seen = [paths(parent[b])[0] for b in range(3)]
        for i in range(N):
            if not seen[0][i]:
                kv[0, i] = value
        sick = N // 3 + 1
        kv[1, sick, 1:, :, 5] = value
        kv[2, sick, 2, 1, 31] = value
        out, pool = run(c)
        assert same(pool, cache_after(c))
        for b in range(3):
            clean = [i for i in range(N) if b == 0 or sick not in seen[b][i]]
            got, want = out[b, clean], good[b, clean]
            # the values are added key by key then: another order of the same sums
            _, tol, _ = reference(dict(c, qkv=torch.nan_to_num(c["qkv"], 0, 0, 0), pool=torch.nan_to_num(c["pool"], 0, 0, 0)))
            assert torch.isfinite(got).all()
            assert (np.abs(got.double().numpy() - want.double().numpy()) <= 2 * tol[b, clean] + 2 * HALF[DT[precision]] * np.abs(want.double().numpy())).all()
        rows = [i for i in range(N) if sick in seen[2][i]]
        assert not torch.isfinite(out[2, rows][:, 1, 31]).any() and torch.isfinite(out[2, rows][:, 0]).all()
        no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_positions_at_the_end_and_outside(precision):
    c = make(precision, 9, 2, 64, [100, 90, 95, 3, 111, 50], 16, trees(6, 9, seed=2, missing=False), seed=3, spare=0)
    cap = c["table"].shape[1] * 16
    good = check(dict(c, pos=torch.tensor([100, 90, 95, 3, cap - 9, 50], dtype=torch.int32)))
    no_device_error()
    c["pos"] = torch.tensor([cap - 1, -2, cap, 3, 2**31 - 1, -2**31], dtype=torch.int32)
    out = check(c)  # of the first sequence one node has a place
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION
    assert same(out[3], good[3]) and (out[[1, 2, 4, 5]] == 0).all() and (out[0, 1:] == 0).all() and (out[0, 0] != 0).any()
    c["pos"] = torch.tensor([-1] * 6, dtype=torch.int32)
    assert (check(c) == 0).all()
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_bad_parents(precision):
    parent = trees(4, 20, seed=3, missing=False)
    parent[0, 7], parent[1, 3], parent[2, 11], parent[3, 0] = 7, 19, -3, 0
    check(make(precision, 20, 2, 32, [40, 64, 5, 100], 16, parent, seed=5))
    assert ab.gpt2_get_error() == ab.DEVERR_TREE


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("value", [-1, 10**6])
def test_bad_blocks(precision, value):
    """A block id outside the pool: read as block 0, never stored through."""
    c = make(precision, 20, 2, 64, [100, 50, 60], 16, trees(3, 20, seed=4, missing=False), seed=6)
    c["table"][0, 2] = value  # cached positions
    check(c)
    assert ab.gpt2_get_error() == ab.DEVERR_BLOCK
    c = make(precision, 20, 2, 64, [96, 50, 60], 16, trees(3, 20, seed=4, missing=False), seed=6)
    c["table"][1, 4] = value  # the nodes'
    check(c)
    assert ab.gpt2_get_error() == ab.DEVERR_BLOCK


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_BF16], ids=["fp32", "bf16"])
def test_offsets_past_32_bits(precision):
    """Blocks beyond element 2^31 of a half."""
    NH, bs, hs = 16, 64, 64
    c = make(precision, 10, NH, hs, [150, 70], bs, trees(2, 10, seed=4), seed=8)
    far = (1 << 31) // (NH * bs * hs) + 5
    t = on_gpu(c)
    big = torch.zeros(2, far + c["pool"].shape[1], NH, bs, hs, dtype=DT[precision], device="cuda")
    big[:, far:] = t["pool"]
    t["pool"], t["table"] = big, torch.where(t["table"] >= 0, t["table"] + far, t["table"])
    out = torch.empty(20, NH * hs, dtype=DT[precision], device="cuda")
    call(dict(c, pool=torch.empty(2, big.shape[1], 0)), t, out)
    ref, tol, _ = reference(c)
    assert (np.abs(out.cpu().double().numpy().reshape(ref.shape) - ref) <= tol).all()
    assert same(big[:, far:].cpu(), cache_after(c)) and not big[:, :far].any()
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
def test_graphs_and_streams(precision):
    """Captured once and replayed on other lengths, trees and values; two graphs
    with workspaces of their own on two streams."""
    cs = [make(precision, 13, 4, 64, ragged(5, 400, s), 16, trees(5, 13, seed=s), seed=s) for s in (1, 2)]
    width = max(c["table"].shape[1] for c in cs)
    blocks = max(c["pool"].shape[1] for c in cs)
    for c in cs:  # of one shape
        c["table"] = torch.cat([c["table"], torch.full((5, width - c["table"].shape[1]), -5, dtype=torch.int32)], 1)
        c["pool"] = torch.cat([c["pool"], torch.zeros(2, blocks - c["pool"].shape[1], 4, 16, 64, dtype=DT[precision])], 1)
    want = [run(c) for c in cs]
    streams, graphs, state = [], [], []
    for _ in range(2):
        t = on_gpu(cs[0])
        out = torch.empty(65, 256, dtype=DT[precision], device="cuda")
        ws = torch.empty(ab.attention_tree_workspace_size(5, 13, 256, 4, precision), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            call(cs[0], t, out, ws, stream=s)
        streams.append(s)
        graphs.append(g)
        state.append((t, out, ws))
    for round in range(4):
        for k in range(2):
            c = cs[(round + k) % 2]
            with torch.cuda.stream(streams[k]):
                for name, x in state[k][0].items():
                    x.copy_(c[name])
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            o, p = want[(round + k) % 2]
            assert same(state[k][1].cpu().view(o.shape), o) and same(state[k][0]["pool"].cpu(), p)
    no_device_error()
