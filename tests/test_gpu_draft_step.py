"""Steps of a model over trees of drafted tokens [NTU "KV Caching"]: a tree step's
logits against the oracle's forward pass over each node's path, and the loop that
drafts, verifies, adjusts and accepts, against the oracle's pass over what it
emitted."""
import numpy as np
import pytest
import torch

import oracle
from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import inputs
from gpt_transformer_forward_gb300.runner import GPT2Model

from draft_reference import adjust, chain, paths, trees
from gpu_helpers import assert_close, dev, host, need_gpu, no_device_error

pytestmark = pytest.mark.gpu
ALL = [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16]
NAMES = {v: k for k, v in ab.PRECISIONS.items()}
LOGIT_TOL = {ab.GPT2_BF16: 2e-2, ab.GPT2_FP16: 2e-2, ab.GPT2_TF32: 2e-2, ab.GPT2_FP32: 1e-4}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def tiny(precision, B, T):
    w = inputs.WORKLOADS["tiny"]
    params, _ = inputs.workload_inputs(w, "perturbed")
    return w.cfg, params, GPT2Model(w.cfg, params, B, T, precision)


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("B,N", [(2, 1), (3, 7), (5, 20), (2, 64)])
def test_tree_step_is_the_forward_pass_of_each_path(precision, B, N):
    bs, most = 8, 40
    cfg, params, m = tiny(precision, max(B, 2), most)
    rng = np.random.default_rng(N)
    # as long as there is room for what the deepest path needs, and for every node's slot
    lens = rng.integers(1, max(2, min(most, cfg.max_seq_len - N)), B).astype(np.int32) if N < 64 else np.zeros(B, np.int32)
    parent = trees(B, N, seed=N) if N > 1 else chain(B, N)
    parent[0, 0] = -1
    tok = rng.integers(0, cfg.vocab_size, (B, N)).astype(np.int32)
    prompt = rng.integers(0, cfg.vocab_size, (B, most)).astype(np.int32)
    maxb = cfg.max_seq_len // bs
    num_blocks = B * maxb + 3
    pool = m.new_paged_kvcache(num_blocks, bs)
    table = dev(rng.permutation(num_blocks)[:B * maxb].reshape(B, maxb).astype(np.int32))
    kv = ab.paged_kv(pool, table, num_blocks, bs, maxb)
    lg, _ = m.new_outputs(B, most, probs=False)
    m.prefill_paged(dev(prompt), lg, kv)
    there = [paths(parent[b])[0] for b in range(B)]
    for b in range(B):
        for i in range(N):
            if not there[b][i]:
                tok[b, i] = -7  # tokens of missing nodes are not read
    logits, probs = m.new_outputs(B, N)
    ws = m.new_tree_workspace(B, N)
    m.decode_step_tree(kv, dev(tok), dev(lens), logits, ws, parent=dev(parent), probs=probs)
    got, p = host(logits), host(probs)
    no_device_error()
    for b in range(B):
        leaves = [path for path in there[b] if path and not any(q[:-1] == path for q in there[b] if q)]
        for path in leaves[:6]:
            seq = np.concatenate([prompt[b, :lens[b]], tok[b, path]])[None].astype(np.int32)
            ref, ref_p = oracle.forward(cfg, params, seq)
            for k, i in enumerate(path):
                at = lens[b] + k
                assert_close(got[b, i, :cfg.vocab_size], ref[0, at, :cfg.vocab_size], atol=LOGIT_TOL[precision],
                             what=f"sequence {b} node {i}")
                assert_close(p[b, i], ref_p[0, at], atol=1e-3, what="probs")


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_one_node_is_the_decode_step(precision):
    """The same cache and token, a whole batch at its own positions; sequences
    without a tree."""
    B, bs, P = 70, 16, 30
    cfg, params, m = tiny(precision, B, P)
    rng = np.random.default_rng(3)
    prompt = rng.integers(0, cfg.vocab_size, (B, P)).astype(np.int32)
    tok = rng.integers(0, cfg.vocab_size, (B, 1)).astype(np.int32)
    lens = rng.integers(0, P + 1, B).astype(np.int32)
    maxb = 4
    table = dev(rng.permutation(B * maxb).reshape(B, maxb).astype(np.int32))
    pools = [m.new_paged_kvcache(B * maxb, bs) for _ in range(2)]
    out = []
    for k, pool in enumerate(pools):
        kv = ab.paged_kv(pool, table, B * maxb, bs, maxb)
        lg, _ = m.new_outputs(B, P, probs=False)
        m.prefill_paged(dev(prompt), lg, kv)
        if k == 0:
            one, _ = m.new_outputs(B, None, probs=False)
            m.decode_step_paged(kv, dev(tok[:, 0]), dev(lens), one)
            out.append(host(one))
        else:
            before = pool.clone()
            idle = lens.copy()
            idle[::3] = -1
            lg, _ = m.new_outputs(B, 1, probs=False)
            ws = m.new_tree_workspace(B, 1)
            m.decode_step_tree(kv, dev(tok), dev(idle), lg, ws)
            out.append(host(lg)[:, 0])
            view = lambda p: p.view(cfg.num_layers, 2, B * maxb, -1)  # noqa: E731
            rows = table[::3].flatten().long()
            assert torch.equal(view(pool)[:, :, rows], view(before)[:, :, rows])
            m.decode_step_tree(kv, dev(tok), dev(lens), lg, ws)
            assert_close(host(lg)[:, 0, :cfg.vocab_size], out[0][:, :cfg.vocab_size], atol=LOGIT_TOL[precision])
    busy = np.arange(B) % 3 != 0
    assert_close(out[1][busy, :cfg.vocab_size], out[0][busy, :cfg.vocab_size], atol=LOGIT_TOL[precision])
    no_device_error()


def test_bad_tokens_and_positions_are_flagged():
    cfg, params, m = tiny(ab.GPT2_FP16, 2, 8)
    pool, table = m.new_paged_kvcache(16, 8), dev(np.arange(16, dtype=np.int32).reshape(2, 8))
    kv = ab.paged_kv(pool, table, 16, 8, 8)
    lg, _ = m.new_outputs(2, 3, probs=False)
    ws = m.new_tree_workspace(2, 3)
    tok = np.array([[1, 2, 3], [4, cfg.vocab_size, 5]], np.int32)
    m.decode_step_tree(kv, dev(tok), dev(np.array([0, 3], np.int32)), lg, ws)
    assert ab.gpt2_get_error() == ab.DEVERR_TOKEN
    tok[1, 1] = 6
    m.decode_step_tree(kv, dev(tok), dev(np.array([62, 64], np.int32)), lg, ws)
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION
    m.decode_step_tree(kv, dev(tok), dev(np.array([61, -1], np.int32)), lg, ws)
    no_device_error()


class Loop:
    """Drafting and verifying on the GPU: tables, tree step, penalties, choice,
    acceptance.  The draft of a node's child is a guess from `guess`."""

    def __init__(self, precision, B, N, num_blocks, seed, rules=True):
        self.cfg, self.params, self.m = tiny(precision, B, 8)
        self.B, self.N, self.bs = B, N, 4
        self.maxb = self.cfg.max_seq_len // self.bs
        self.num_blocks = num_blocks
        self.rng = np.random.default_rng(seed)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.pool = self.m.new_paged_kvcache(num_blocks, self.bs)
        self.table = i32(B, self.maxb)
        self.kv = ab.paged_kv(self.pool, self.table, num_blocks, self.bs, self.maxb)
        self.free = dev(self.rng.permutation(num_blocks).astype(np.int32))
        self.held, self.taken = [i32(B), i32(B)], [i32(1), i32(1)]
        self.pos, self.root = i32(B), dev(self.rng.integers(0, self.cfg.vocab_size, B).astype(np.int32))
        self.logits, _ = self.m.new_outputs(B, N, probs=False)
        self.ws = self.m.new_tree_workspace(B, N)
        self.chosen = i32(B, N)
        self.rules = {}
        if rules:
            W = (self.cfg.vocab_size + 31) // 32
            self.rules = dict(repetition=torch.full((B,), 1.3, device="cuda"), presence=torch.full((B,), 0.2, device="cuda"),
                              frequency=torch.full((B,), 0.1, device="cuda"),
                              bias_ids=dev(self.rng.integers(0, self.cfg.vocab_size, (B, 3)).astype(np.int32)),
                              bias_values=torch.full((B, 3), 0.5, device="cuda"),
                              masks=dev(self.rng.integers(-2**31, 2**31, (2, W)).astype(np.int32) | 0x11111111),
                              mask_rows=dev(self.rng.integers(-1, 2, (B, N)).astype(np.int32)))
        self.text = [[int(t)] for t in self.root.cpu()]  # what is known: the root last
        self.waited = 0

    def step(self, guess):
        """guess(b, tokens): the next token that a draft model would expect."""
        B, N = self.B, self.N
        parent = trees(B, N, int(self.rng.integers(1 << 30)), missing=True)
        parent[:, 0] = -1
        tok = np.zeros((B, N), np.int32)
        tok[:, 0] = [t[-1] for t in self.text]
        for b in range(B):
            for i, path in enumerate(paths(parent[b])[0]):
                if i and path:
                    told = self.text[b] + [int(tok[b, a]) for a in path[1:-1]]
                    tok[b, i] = guess(b, told) if self.rng.random() < 0.7 else self.rng.integers(0, self.cfg.vocab_size)
        tokd, par = dev(tok), dev(parent)
        a, z = self.held
        # positions that need a block, within the longest sequence
        want = torch.clamp(self.pos + N, max=self.cfg.max_seq_len)
        new = torch.clamp(want - a, min=0)
        ab.paged_build_tables(self.table, None, z, self.taken[1], a, new, self.free, self.num_blocks, self.taken[0], None,
                              0, B, N, self.num_blocks, self.bs, self.maxb)
        self.held, self.taken = [z, a], self.taken[::-1]
        room = (z >= want) & (self.pos + N <= self.cfg.max_seq_len)
        pos = torch.where(room, self.pos, torch.full_like(self.pos, -1))
        self.waited += int((~room).sum())
        self.m.decode_step_tree(self.kv, tokd, pos, self.logits, self.ws, parent=par)
        plain = self.logits.clone()
        if self.rules:
            # everything before this tree's first node
            H = max(len(t) for t in self.text)
            hist = np.full((B, H), -1, np.int32)
            for b, t in enumerate(self.text):
                hist[b, :len(t) - 1] = t[:-1]
            n = np.array([len(t) - 1 for t in self.text], np.int32)
            self.m.adjust_logits(self.logits, tokd, par, history=dev(hist), history_len=dev(n),
                                 prompt_len=dev(np.minimum(n, 2)), **self.rules)
            self.last = dict(history=hist, history_len=n, prompt_len=np.minimum(n, 2), tok=tok, parent=parent)
        ab.gpt2_argmax(self.chosen, self.logits, B * N, self.cfg.vocab_size, self.cfg.padded_vocab_size)
        r = self.m.accept_tree(self.kv, tokd, self.chosen, pos, par)
        count, emitted, path = (r[k].cpu().numpy() for k in ("count", "emitted", "path"))
        self.pos = torch.where(room, r["next_pos"], self.pos)
        self.last = dict(getattr(self, "last", {}), plain=host(plain), path=path, count=count, parent=parent, tok=tok)
        for b in range(B):
            self.text[b] += [int(t) for t in emitted[b, :count[b]]]
        return count


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("rules", [False, True])
def test_the_loop_of_drafting_and_verifying(precision, rules):
    """Every token that the loop emits is the best one behind the text before it,
    by the oracle's logits and the penalties' definition, to the precision's
    tolerance; the logits of the accepted nodes are the oracle's."""
    B, N, steps = 4, 9, 6
    loop = Loop(precision, B, N, 4 * 16 + 3, seed=precision + 10 * rules, rules=rules)
    cfg, tol = loop.cfg, LOGIT_TOL[precision]

    memo = {}

    def guess(b, told):  # a good draft model: the oracle without penalties
        key = tuple(told)
        if key not in memo:
            memo[key] = int(oracle.forward(cfg, loop.params, np.array([told], np.int32))[0][0, -1, :cfg.vocab_size].argmax())
        return memo[key]

    accepted = 0
    for _ in range(steps):
        before = [list(t) for t in loop.text]
        count = loop.step(guess)
        no_device_error()
        accepted += int(count.sum()) - B
        L = loop.last
        for b in range(B):
            seq = np.array([loop.text[b]], np.int32)
            ref = oracle.forward(cfg, loop.params, seq)[0][0, :, :cfg.vocab_size]
            for k in range(count[b]):
                node, at = int(L["path"][b, k]), len(before[b]) - 1 + k
                assert_close(L["plain"][b, node, :cfg.vocab_size], ref[at], atol=tol, what=f"sequence {b}, {k} accepted")
                row, scale = ref[at].copy(), 1.0
                if rules:
                    x = np.zeros((1, N, cfg.vocab_size))
                    x[0, node] = ref[at]
                    mine = {k2: v.cpu().numpy()[b:b + 1] for k2, v in loop.rules.items() if k2 not in ("masks", "mask_rows")}
                    row = adjust(x, cfg.vocab_size, L["history"][b:b + 1], L["history_len"][b:b + 1], L["prompt_len"][b:b + 1],
                                 mine["repetition"], mine["presence"], mine["frequency"], mine["bias_ids"],
                                 mine["bias_values"], loop.rules["masks"].cpu().numpy().view(np.uint32),
                                 loop.rules["mask_rows"].cpu().numpy()[b], L["tok"][b:b + 1], L["parent"][b:b + 1])[0][0, node]
                    scale = 1.3  # the repetition penalty stretches what is below 0
                assert row[seq[0, at + 1]] >= row.max() - 2 * tol * scale, (b, k)
    assert accepted > 0
    assert loop.pos.tolist() == [len(t) - 1 for t in loop.text]


def test_the_loop_when_blocks_run_out():
    """A sequence that gets no blocks waits: it keeps its place and its text, the
    others go on, nothing is flagged and nothing is written outside their blocks."""
    loop = Loop(ab.GPT2_FP16, 4, 8, 12, seed=2)
    cfg = loop.cfg
    for _ in range(5):
        texts = [list(t) for t in loop.text]
        count = loop.step(lambda b, told: told[-1])
        no_device_error()
        for b in range(4):
            assert count[b] == 0 and loop.text[b] == texts[b] or len(loop.text[b]) == len(texts[b]) + count[b]
    assert loop.waited > 0
    for b in range(4):
        if len(loop.text[b]) > 1:
            ref = oracle.forward(cfg, loop.params, np.array([loop.text[b]], np.int32))[0]
            assert ref.shape[1] == int(loop.pos[b]) + 1


def test_a_step_in_a_graph():
    """Tree step, penalties, choice and acceptance captured once and replayed."""
    B, N = 3, 6
    a, b = Loop(ab.GPT2_FP16, B, N, 60, seed=4), Loop(ab.GPT2_FP16, B, N, 60, seed=4)
    for l in (a, b):
        l.table.copy_(torch.arange(B * l.maxb, dtype=torch.int32).view(B, l.maxb) % 60)
        l.table[:, 5:] = -1
        l.table[:, :5] = torch.arange(15, dtype=torch.int32).view(3, 5).cuda()
    par = dev(np.array([[-1, 0, 1, 1, 0, 2]] * B, np.int32))
    hist = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    state = {}

    def step(l, tok, pos, stream=None):
        l.m.decode_step_tree(l.kv, tok, pos, l.logits, l.ws, parent=par, stream=stream)
        l.m.adjust_logits(l.logits, tok, par, history=hist, stream=stream, **l.rules)
        ab.gpt2_argmax(l.chosen, l.logits, B * N, l.cfg.vocab_size, l.cfg.padded_vocab_size, stream)
        return l.m.accept_tree(l.kv, tok, l.chosen, pos, par, stream=stream)

    toks = [dev(a.rng.integers(0, a.cfg.vocab_size, (B, N)).astype(np.int32)) for _ in range(4)]
    poss = [dev(np.array(p, np.int32)) for p in ([0, 0, 0], [1, 2, 3], [4, -1, 5], [7, 2, 9])]
    tok, pos = toks[0].clone(), poss[0].clone()
    step(b, tok, pos)  # what a first call sets up
    torch.cuda.synchronize()
    b.pool.zero_()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        state["r"] = step(b, tok, pos, stream=s)
    for t, p in zip(toks, poss):
        want = step(a, t, p)
        with torch.cuda.stream(s):
            tok.copy_(t)
            pos.copy_(p)
            g.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(v, state["r"][k]), k
        assert torch.equal(a.pool, b.pool) and torch.equal(a.logits[p >= 0], b.logits[p >= 0])
    no_device_error()
