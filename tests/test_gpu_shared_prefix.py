"""Decode attention over a shared prefix [NTU "KV Caching"; FlashAttention
Algorithm 0], against a 64-bit form on the CPU that walks each sequence's
positions.

Tolerances: u = 2^-24, w the half step of the element type (relative 2^-8 for
bf16, 2^-11 for fp16; u for fp32).  A score of hs products is off by at most
(hs + 4) u sum|q k| / sqrt(hs) (products, sums, scale and the log2 units), a
probability relative to the row's sum by twice that, the exponential's 8 u and
the sums' (n / 16 + 64) u over n positions; an output by that times max|v|,
plus w max|v| for probabilities rounded to the 16-bit type and w |out| for the
output's own rounding."""
import numpy as np
import pytest
import torch

import oracle
from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import inputs
from gpt_transformer_forward_gb300.runner import GPT2Model

from gpu_helpers import assert_close, dev, host, need_gpu, no_device_error
from serve_reference import shared_attention

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
DT = {ab.GPT2_FP32: torch.float32, ab.GPT2_TF32: torch.float32, ab.GPT2_BF16: torch.bfloat16,
      ab.GPT2_FP16: torch.float16}
HALF = {torch.float32: u, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ALL = [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16]
NAMES = {v: k for k, v in ab.PRECISIONS.items()}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(precision, B, NH, hs, P, own, bs, seed, qscale=2.0):
    """Inputs as CPU tensors; `own`: each sequence's own cached positions."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[precision]
    own = torch.as_tensor(own)
    n_own = (P + int(own.max())) // bs + 1 - P // bs
    num_blocks = P // bs + B * n_own + 3
    ids = torch.randperm(num_blocks, generator=g).to(torch.int32)
    table = torch.empty(B, P // bs + n_own + 1, dtype=torch.int32)
    table[:] = -5  # entries no call reaches
    table[:, :P // bs] = ids[:P // bs]
    table[:, P // bs:P // bs + n_own] = ids[P // bs:P // bs + B * n_own].view(B, n_own)
    pool = torch.randn(2, num_blocks, NH, bs, hs, generator=g).to(dt)
    if P % bs:
        mine = table[:, P // bs].long()
        pool[:, mine, :, :P % bs] = pool[:, mine[:1], :, :P % bs].clone()
    pos = (P + own).to(torch.int32)
    qkv = torch.randn(B, 3, NH, hs, generator=g)
    qkv[:, 0] *= qscale
    return dict(precision=precision, NH=NH, hs=hs, P=P, bs=bs, pool=pool, table=table, pos=pos,
                qkv=qkv.reshape(B, -1).to(dt))


def call(c, pool, qkv, table, pos, out, ws=None, P=None):
    B, C = qkv.shape[0], c["NH"] * c["hs"]
    P = c["P"] if P is None else P
    n = ab.attention_shared_prefix_workspace_size(B, C, c["NH"], P, c["precision"])
    if ws is None:
        ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")  # NaN bytes
    kv = ab.paged_kv(pool, table, c["pool"].shape[1], c["bs"], c["table"].shape[1])
    ab.attention_shared_prefix(out, qkv, kv, pos, B, C, c["NH"], P, c["precision"], ws, n)
    return ws


def run(c, **kw):
    g = {k: c[k].cuda() for k in ("pool", "qkv", "table", "pos")}
    out = torch.full((c["qkv"].shape[0], c["NH"] * c["hs"]), 9.0, dtype=DT[c["precision"]], device="cuda")
    call(c, g["pool"], g["qkv"], g["table"], g["pos"], out, **kw)
    torch.cuda.synchronize()
    return out.cpu(), g["pool"].cpu()


def reference(c):
    B = c["qkv"].shape[0]
    q, k, v = c["qkv"].double().numpy().reshape(B, 3, c["NH"], c["hs"]).transpose(1, 0, 2, 3)
    out, sabs, vmax = shared_attention(q, k, v, c["pool"].double().numpy(), c["table"].numpy(), c["pos"].numpy(),
                                       c["P"], c["bs"])
    w = HALF[DT[c["precision"]]]
    n = c["pos"].numpy()[:, None] + 1
    part = 2 * (c["hs"] + 4) * u * sabs + 8 * u + (n / 16 + 64) * u
    tol = (part + (w if w > u else 0)) * vmax
    return out, tol[..., None] + w * np.abs(out)


def check(c, **kw):
    out, pool = run(c, **kw)
    no_device_error()
    B = out.shape[0]
    ref, tol = reference(c)
    err = np.abs(out.double().numpy().reshape(ref.shape) - ref)
    assert (err <= tol).all(), f"{(err > tol).sum()} off, worst {(err / tol).max():.3f} of the tolerance"
    want = c["pool"].clone()
    k, v = c["qkv"].view(B, 3, c["NH"], c["hs"])[:, 1:].unbind(1)
    blk = c["table"].gather(1, (c["pos"].long() // c["bs"])[:, None])[:, 0].long()
    want[0, blk, :, c["pos"].long() % c["bs"]] = k
    want[1, blk, :, c["pos"].long() % c["bs"]] = v
    assert torch.equal(pool, want), "the cache"
    return out


def own_of(B, most, seed):
    own = np.random.default_rng(seed).integers(0, most + 1, B)
    own[0] = most
    own[-1] = 0
    return own


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("hs", [16, 32, 64])
@pytest.mark.parametrize("B,NH,P,most,bs", [
    (1, 1, 1, 0, 1), (1, 2, 64, 5, 16), (2, 3, 63, 1, 16), (3, 1, 65, 40, 2), (5, 2, 128, 3, 128), (16, 2, 127, 9, 8),
    (17, 2, 129, 9, 4), (31, 3, 500, 17, 16), (33, 2, 1001, 33, 32), (65, 1, 257, 300, 64), (4, 12, 960, 63, 16),
    (130, 2, 777, 20, 16), (1, 1, 5000, 2, 64), (70, 1, 300, 40, 2), (129, 2, 1500, 9, 128), (300, 1, 130, 3, 256),
    (66, 1, 1, 2, 1), (128, 1, 128, 5, 8), (2, 3, 257, 1, 16), (3, 1, 321, 40, 2), (5, 2, 384, 3, 128), (17, 2, 300, 9, 4),
    (16, 1, 4097, 2, 16), (66, 1, 257, 2, 1), (128, 1, 384, 5, 8), (128, 3, 385, 5, 8), (300, 1, 300, 3, 256),
    (4, 2, 256, 9, 16), (40, 12, 64, 3, 8), (12, 12, 200, 80, 16), (2, 1, 100, 2000, 64), (128, 3, 129, 5, 8), (520, 1, 400, 5, 32),
])
def test_against_64_bits(precision, hs, B, NH, P, most, bs):
    check(make(precision, B, NH, hs, P, own_of(B, most, P), bs, seed=B + P))


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_no_prefix(precision):
    check(make(precision, 6, 3, 64, 0, own_of(6, 200, 1), 16, seed=2))


@pytest.mark.parametrize("precision", [ab.GPT2_FP16, ab.GPT2_BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("B", [1, 8, 40, 128, 200, 257])
def test_many_sequences(precision, B):
    check(make(precision, B, 2, 64, 2085, own_of(B, 70, B), 32, seed=B))


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("B", [3, 70])
def test_peaked_and_rising_scores(precision, B):
    """Scores that grow along the prefix (every step raises the running
    maximum), and one that dominates late."""
    c = make(precision, B, 2, 64, 900, own_of(B, 30, 3), 16, seed=4, qscale=1.0)
    rise = torch.linspace(0.2, 8.0, 900)
    for j in range(900):
        c["pool"][0, c["table"][0, j // 16].long(), 0, j % 16] = (rise[j] * torch.ones(64)).to(c["pool"].dtype)
    if 900 % 16:
        mine = c["table"][:, 900 // 16].long()
        c["pool"][:, mine, :, :900 % 16] = c["pool"][:, mine[:1], :, :900 % 16].clone()
    c["qkv"].view(B, 3, 2, 64)[:, 0, 0] = 1.0
    c["pool"][0, c["table"][0, 850 // 16].long(), 1, 850 % 16] *= 6
    check(c)


def test_extreme_values_stay_in_their_rows():
    """Huge values and NaN in cache slots that no position reaches."""
    for precision in ALL:
        c = make(precision, 5, 2, 32, 100, [0, 3, 10, 1, 7], 16, seed=7)
        used = torch.zeros(c["pool"].shape[1], 16, dtype=torch.bool)
        for b in range(5):
            for j in range(int(c["pos"][b]) + 1):
                used[c["table"][b if j >= 100 else 0, j // 16].long(), j % 16] = True
        for b in range(1, 5):  # the other rows' copies of the prefix's tail are not read
            assert not used[c["table"][b, 100 // 16].long(), 0]
        bad = ~used
        c["pool"].permute(1, 3, 0, 2, 4)[bad] = float("nan")
        out, pool = run(c)
        ref, tol = reference(c)
        assert (np.abs(out.double().numpy().reshape(ref.shape) - ref) <= tol).all(), NAMES[precision]
        no_device_error()


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_FP16], ids=["fp32", "fp16"])
def test_bad_positions(precision):
    c = make(precision, 6, 2, 64, 100, [0, 5, 9, 3, 2, 8], 16, seed=3)
    good = run(c)[0]
    cap = c["table"].shape[1] * 16
    bad = dict(c, pos=c["pos"].clone())
    bad["pos"][1], bad["pos"][2], bad["pos"][4], bad["pos"][5] = -1, 99, cap, 2**31 - 1
    out, pool = run(bad)
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION
    assert (out[[1, 2, 4, 5]] == 0).all() and torch.equal(out[[0, 3]], good[[0, 3]])
    changed = (pool.view(torch.uint8) != c["pool"].view(torch.uint8)).flatten(2).any(2).any(0)
    mine = {int(c["table"][b, int(c["pos"][b]) // 16]) for b in (0, 3)}
    assert set(changed.nonzero()[:, 0].tolist()) <= mine


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_FP16], ids=["fp32", "fp16"])
@pytest.mark.parametrize("where", [(0, 2), (3, 7)])
def test_bad_blocks(precision, where):
    """A block id outside the pool, in the prefix (row 0) or in a sequence's
    own positions: flagged and read as block 0."""
    for value in (-1, 10**6):
        c = make(precision, 4, 2, 64, 100, [20, 20, 20, 20], 16, seed=3)
        c["table"][where] = value
        run(c)
        assert ab.gpt2_get_error() == ab.DEVERR_BLOCK


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("B,NH,P", [(4, 2, 96), (4, 2, 688), (70, 40, 1008)])
def test_nothing_is_appended_through_a_bad_entry(precision, B, NH, P):
    """A sequence at a block border whose next entry is missing (the state of a
    request that waits for a block), or past the pool: the cache keeps every
    other sequence's positions and its own, and no output changes."""
    own = own_of(B, 40, 3)
    own[2] = 32
    c = make(precision, B, NH, 64, P, own, 16, seed=5)
    good = check(c)
    for value in (-1, c["pool"].shape[1], -2**31):
        bad = dict(c, table=c["table"].clone())
        bad["table"][2, (P + 32) // 16] = value
        out, pool = run(bad)
        assert ab.gpt2_get_error() == ab.DEVERR_BLOCK
        assert torch.equal(out, good)  # the new token's key and value come from qkv
        want = c["pool"].clone()
        k, v = c["qkv"].view(B, 3, NH, 64)[:, 1:].unbind(1)
        for b in range(B):
            if b != 2:
                at = int(c["pos"][b])
                blk = int(c["table"][b, at // 16])
                want[0, blk, :, at % 16], want[1, blk, :, at % 16] = k[b], v[b]
        assert torch.equal(pool, want)


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
@pytest.mark.parametrize("B,NH,P", [(4, 2, 96), (4, 2, 700), (70, 40, 1000)])
def test_sequences_without_a_token(precision, B, NH, P):
    """pos -1: a zero row, nothing appended, nothing flagged, whatever the row of
    the table holds; the other rows are as with it."""
    c = make(precision, B, NH, 64, P, own_of(B, 40, 3), 16, seed=5)
    good = check(c)
    idle = dict(c, pos=c["pos"].clone(), table=c["table"].clone())
    idle["pos"][[1, B - 1]] = -1
    idle["table"][1] = 0
    idle["table"][B - 1] = -1
    out, pool = run(idle)
    no_device_error()
    rest = torch.ones(B, dtype=torch.bool)
    rest[[1, B - 1]] = False
    assert (out[~rest] == 0).all() and torch.equal(out[rest], good[rest])
    want = c["pool"].clone()
    k, v = c["qkv"].view(B, 3, NH, 64)[:, 1:].unbind(1)
    for b in rest.nonzero()[:, 0].tolist():
        at = int(c["pos"][b])
        blk = int(c["table"][b, at // 16])
        want[0, blk, :, at % 16], want[1, blk, :, at % 16] = k[b], v[b]
    assert torch.equal(pool, want)


def test_entries_that_are_not_reached_may_hold_anything():
    # rows other than 0 over the prefix's whole blocks
    c = make(ab.GPT2_FP16, 5, 2, 64, 96, [4, 0, 30, 2, 9], 16, seed=3)
    good = run(c)[0]
    c["table"][1:, :6] = 10**8
    assert torch.equal(run(c)[0], good)
    no_device_error()


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_repeats_streams_and_graphs(precision):
    """Two captured graphs with workspaces of their own and one that both
    replay in turn; the same values again, on another stream, and with more
    workspace than needed."""
    c = make(precision, 12, 4, 64, 1500, own_of(12, 90, 5), 16, seed=6)
    first, pool1 = run(c)
    big = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    assert torch.equal(run(c, ws=big)[0], first)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(run(c)[0], first)
    d = make(precision, 12, 4, 64, 1500, own_of(12, 90, 6), 16, seed=7)
    second = run(d)[0]
    graphs = []
    for x in (c, d):
        g = {k: x[k].cuda() for k in ("pool", "qkv", "table", "pos")}
        out = torch.zeros(12, 256, dtype=DT[precision], device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(x, g["pool"], g["qkv"], g["table"], g["pos"], out, ws=big)
        graphs.append((graph, out, g))
    for k in (0, 1, 0, 1, 1, 0):
        graph, out, _ = graphs[k]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), (first, second)[k])
    no_device_error()


def test_cache_past_32_bits():
    """Blocks whose offset passes 2^31 elements (bf16, 8.6 GB)."""
    NH, hs, bs, P = 16, 64, 64, 300
    num_blocks = 2 ** 31 // (NH * bs * hs) + 64
    pool = torch.zeros(2, num_blocks, NH, bs, hs, dtype=torch.bfloat16, device="cuda")
    c = make(ab.GPT2_BF16, 3, NH, hs, P, [70, 0, 5], bs, seed=2)
    n = c["pool"].shape[1]
    pool[:, num_blocks - n:] = c["pool"].cuda()
    table = c["table"] + (num_blocks - n)
    out = torch.empty(3, NH * hs, dtype=torch.bfloat16, device="cuda")
    kv = ab.paged_kv(pool, table.cuda(), num_blocks, bs, table.shape[1])
    nb = ab.attention_shared_prefix_workspace_size(3, NH * hs, NH, P, ab.GPT2_BF16)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    tbl = table.cuda()
    kv = ab.paged_kv(pool, tbl, num_blocks, bs, table.shape[1])
    ab.attention_shared_prefix(out, c["qkv"].cuda(), kv, c["pos"].cuda(), 3, NH * hs, NH, P, ab.GPT2_BF16, ws, nb)
    ref, tol = reference(c)
    assert (np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    no_device_error()


# ---------------------------------------- many sequences, a long prefix
# (16-bit caches with heads of 64 take another kernel from this work on)
def long_case(precision, B, NH, P, own, bs, **kw):
    assert B >= 65 and (B + 63) // 64 * 64 * NH * P >= 5_000_000
    return make(precision, B, NH, 64, P, own, bs, **kw)


@pytest.mark.parametrize("precision", [ab.GPT2_FP16, ab.GPT2_BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("B,NH,P,most,bs", [
    (65, 16, 2500, 3, 64), (128, 16, 2443, 5, 16), (129, 13, 2004, 9, 4), (200, 13, 1561, 20, 2), (257, 8, 1999, 3, 128),
    (300, 16, 978, 7, 256), (66, 40, 1000, 2, 1), (520, 1, 8690, 5, 32), (100, 4, 9999, 2, 64), (128, 16, 2560, 5, 8),
])
def test_long_prefix_of_many_sequences(precision, B, NH, P, most, bs):
    check(long_case(precision, B, NH, P, own_of(B, most, P), bs, seed=B + P))


@pytest.mark.parametrize("precision", [ab.GPT2_FP16, ab.GPT2_BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("B,NH", [(70, 20), (150, 14)])
def test_long_prefix_with_rising_scores(precision, B, NH):
    P = 2000
    c = long_case(precision, B, NH, P, own_of(B, 30, 3), 16, seed=4, qscale=1.0)
    blk, at = c["table"][0, :P // 16].long().repeat_interleave(16), torch.arange(P) % 16
    c["pool"][0, blk, 0, at] = torch.linspace(0.2, 8.0, P)[:, None].expand(P, 64).to(c["pool"].dtype)
    c["qkv"].view(B, 3, NH, 64)[:, 0, 0] = 1.0
    c["pool"][0, c["table"][0, 1850 // 16].long(), 1, 1850 % 16] *= 6
    check(c)


@pytest.mark.parametrize("precision", [ab.GPT2_FP16, ab.GPT2_BF16], ids=["fp16", "bf16"])
def test_long_prefix_reads_nothing_behind_it(precision):
    """NaN in every slot that no position reaches, the rest of the prefix's
    last block among them."""
    P, B, NH = 2001, 70, 20
    c = long_case(precision, B, NH, P, own_of(B, 9, 2), 16, seed=7)
    used = torch.zeros(c["pool"].shape[1], 16, dtype=torch.bool)
    for b in range(B):
        j = torch.arange(0 if b == 0 else P, int(c["pos"][b]) + 1)
        used[c["table"][b].long()[j // 16], j % 16] = True
    c["pool"].permute(1, 3, 0, 2, 4)[~used] = float("nan")
    out, _ = run(c)
    ref, tol = reference(c)
    assert (np.abs(out.double().numpy().reshape(ref.shape) - ref) <= tol).all()
    no_device_error()


def test_long_prefix_flags_bad_blocks_and_positions():
    P, B, NH = 2000, 130, 14
    c = long_case(ab.GPT2_FP16, B, NH, P, own_of(B, 20, 1), 16, seed=3)
    good = run(c)[0]
    for value in (-1, 10**6):
        bad = dict(c, table=c["table"].clone())
        bad["table"][0, 60] = value
        run(bad)
        assert ab.gpt2_get_error() == ab.DEVERR_BLOCK
    bad = dict(c, pos=c["pos"].clone())
    bad["pos"][[0, 64, 128]] = torch.tensor([P - 1, -1, 2**31 - 1], dtype=torch.int32)
    out, _ = run(bad)
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION
    rest = torch.ones(B, dtype=torch.bool)
    rest[[0, 64, 128]] = False
    assert (out[~rest] == 0).all() and torch.equal(out[rest], good[rest])


@pytest.mark.parametrize("B", [70, 130])
def test_long_prefix_repeats_streams_and_graphs(B):
    c = long_case(ab.GPT2_BF16, B, 20, 2000, own_of(B, 9, 5), 16, seed=6)
    first = run(c)[0]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert torch.equal(run(c)[0], first)
    g = {k: c[k].cuda() for k in ("pool", "qkv", "table", "pos")}
    nb = ab.attention_shared_prefix_workspace_size(B + 100, 20 * 64, 20, 9000, ab.GPT2_BF16)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, 20 * 64, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, g["pool"], g["qkv"], g["table"], g["pos"], out, ws=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), first)
    no_device_error()


# ------------------------------------------- the prefix's probabilities
@pytest.mark.parametrize("precision", [ab.GPT2_FP16, ab.GPT2_BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("B,NH,P", [(3, 5, 700), (40, 4, 1000), (70, 20, 2000), (150, 14, 2000)])
def test_probabilities_keep_more_than_16_bits(precision, B, NH, P):
    """Few keys dominate and the values' signs cancel, so that what the
    probabilities lose shows beside the output's own rounding.  Keys and queries
    are nonzero in one dimension: a score is one product (its factor of log2
    units and the subtracted maximum: 4 u |s| more).  Probabilities enter the
    products as the sum of two 16-bit values.  In fp16 both are rounded: off by
    w^2 relative, or by 2^-25 (half its smallest step) where that is more, but
    never by more than themselves.  In bf16 the first is cut off, which leaves
    less than a step, 2 w, and the second rounds that: 2 w^2."""
    hs, bs = 64, 16
    c = make(precision, B, NH, hs, P, own_of(B, 20, B), bs, seed=B, qscale=1.0)
    g = torch.Generator().manual_seed(B + P)
    rank = torch.stack([torch.randperm(P, generator=g) for _ in range(NH)])  # [NH, P]
    blk, at = c["table"][0].long()[torch.arange(P) // bs], torch.arange(P) % bs
    c["pool"][0] = 0
    c["pool"][0, blk, :, at, 0] = (-4.0 * rank.clamp(max=60)).t().to(c["pool"].dtype)  # whole numbers: exact
    c["pool"][1] = torch.randint(0, 2, c["pool"][1].shape, generator=g).to(c["pool"].dtype) * 2 - 1
    if P % bs:
        mine = c["table"][:, P // bs].long()
        c["pool"][:, mine, :, :P % bs] = c["pool"][:, mine[:1], :, :P % bs].clone()
    x = c["qkv"].view(B, 3, NH, hs)
    x[:, :2] = 0
    x[:, 0, :, 0] = torch.tensor([0.5, 1.0, 0.75])[torch.arange(B) % 3][:, None].to(x.dtype)
    x[:, 1, :, 0] = -48
    out, _ = run(c)
    no_device_error()
    q, k, v = c["qkv"].double().numpy().reshape(B, 3, NH, hs).transpose(1, 0, 2, 3)
    ref, sabs, vmax = shared_attention(q, k, v, c["pool"].double().numpy(), c["table"].numpy(), c["pos"].numpy(), P, bs)
    w = HALF[DT[precision]]
    n = c["pos"].numpy()[:, None] + 1
    lost = np.full((B, NH), w * w if precision == ab.GPT2_FP16 else 2 * w * w)
    if precision == ab.GPT2_FP16:
        s = q[:, :, 0][:, :, None] * (-4.0 * rank.clamp(max=60)).numpy() / 8  # [B, NH, P]
        lost += np.minimum(np.exp(s), 2.0 ** -25).sum(2)  # the largest is 0
    tol = (2 * 5 * u * sabs + 8 * u + (n / 16 + 64) * u + lost) * vmax
    tol = tol[..., None] + w * np.abs(ref)
    err = np.abs(out.double().numpy().reshape(ref.shape) - ref)
    assert (err <= tol).all(), f"{(err > tol).sum()} off, worst {(err / tol).max():.3f} of the tolerance"


# ------------------------------------------------------------- the model
LOGIT_TOL = {ab.GPT2_BF16: 2e-2, ab.GPT2_FP16: 2e-2, ab.GPT2_TF32: 2e-2, ab.GPT2_FP32: 1e-4}


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_FP16], ids=["fp32", "tf32", "fp16"])
@pytest.mark.parametrize("B", [3, 70])
def test_continuations_of_one_prompt(precision, B):
    """The operators together: a prompt is prefilled once by a slot map, every
    continuation's tables are built on the GPU, decode steps read the prompt's
    blocks once for all, and each step's log probabilities rank the drawn
    tokens.  Against the oracle's forward pass over each whole sequence."""
    w = inputs.WORKLOADS["tiny"]
    cfg = w.cfg
    params, _ = inputs.workload_inputs(w, "perturbed")
    bs, prompt, steps, top = 4, 22, 9, 5
    shared = prompt // bs * bs  # whole blocks; the prompt's last 2 tokens are fed to every continuation
    rng = np.random.default_rng(B)
    seq = np.empty((B, prompt + steps), np.int32)
    seq[:, :prompt] = rng.integers(0, cfg.vocab_size, prompt)
    seq[:, prompt:] = rng.integers(0, cfg.vocab_size, (B, steps))
    ref_logits, _ = oracle.forward(cfg, params, seq[:min(B, 6)])
    m = GPT2Model(cfg, params, B, prompt, precision)
    maxb = -(-(prompt + steps) // bs)
    num_blocks = shared // bs + B * (maxb - shared // bs) + 2
    pool = m.new_paged_kvcache(num_blocks, bs)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    free = dev(rng.permutation(num_blocks).astype(np.int32))
    # the prompt: one request of `shared` new positions
    table1, slots1, len1, taken = i32(1, maxb), i32(1, shared), i32(1), [i32(1), i32(1)]
    ab.paged_build_tables(table1, slots1, len1, taken[1], i32(1), dev(np.array([shared], np.int32)), free, num_blocks,
                          taken[0], None, 0, 1, shared, num_blocks, bs, maxb)
    kv1 = ab.paged_kv(pool, table1, num_blocks, bs, maxb)
    lg, _ = m.new_outputs(1, shared, probs=False)
    m.prefill_slots(dev(seq[:1, :shared]), lg, kv1, slots1)
    assert_close(host(lg)[0][:, :cfg.vocab_size], ref_logits[0, :shared, :cfg.vocab_size], atol=LOGIT_TOL[precision],
                 what="prompt")
    prefix_blocks = table1[0, :shared // bs].clone()
    # the continuations: one position a step, all buffers on the GPU
    table, lens = i32(B, maxb), [torch.full((B,), shared, dtype=torch.int32, device="cuda"), i32(B)]
    kv = ab.paged_kv(pool, table, num_blocks, bs, maxb)
    ws = m.new_shared_workspace(B, shared)
    logits, _ = m.new_outputs(B, None, probs=False)
    plain, _ = m.new_outputs(B, None, probs=False)
    toks = dev(seq)
    cur = 1
    for i, t in enumerate(range(shared, prompt + steps - 1)):
        a, b = i % 2, 1 - i % 2
        ab.paged_build_tables(table, None, lens[b], taken[1 - cur], lens[a], None, free, num_blocks, taken[cur],
                              prefix_blocks, shared, B, 1, num_blocks, bs, maxb)
        cur = 1 - cur
        tok = toks[:, t].contiguous()
        m.decode_step_shared(kv, tok, lens[a], shared, logits, ws)
        got = host(logits)[:, :cfg.vocab_size]
        assert_close(got[:len(ref_logits)], ref_logits[:, t, :cfg.vocab_size], atol=LOGIT_TOL[precision],
                     what=f"step {t}")
        # the unshared step over the same cache agrees to the precision's rounding
        m.decode_step_paged(kv, tok, lens[a], plain)
        assert_close(host(plain)[:, :cfg.vocab_size], got, atol=LOGIT_TOL[precision], what="unshared")
        nxt = toks[:, t + 1].contiguous()
        r = m.logprobs(logits, nxt, top=top)
        lp = torch.log_softmax(logits[:, :cfg.vocab_size].double(), 1)
        assert (r["logprob"] - lp.gather(1, nxt.long()[:, None])[:, 0]).abs().max() < 1e-5
        best = torch.topk(lp, top, 1)
        assert (r["top_logprobs"] - best.values).abs().max() < 1e-5
        assert torch.equal(lens[b], lens[a] + 1)
    no_device_error()


def test_prefill_slots_leaves_padding_out():
    """A padded batch of prompts of different lengths: the outputs are the
    forward pass's, the cache holds what gpt2_prefill_paged writes at the
    stored positions, and nothing else of the pool changes; a slot past the
    pool is flagged."""
    w = inputs.WORKLOADS["tiny"]
    cfg = w.cfg
    params, tok = inputs.workload_inputs(w, "perturbed")
    B, T = tok.shape
    for precision in ALL:
        m = GPT2Model(cfg, params, B, T, precision)
        bs, maxb = 8, 8
        num_blocks = B * maxb + 5
        table = torch.arange(B * maxb, dtype=torch.int32).view(B, maxb).cuda()
        kv = ab.paged_kv(None, table, num_blocks, bs, maxb)
        lens = torch.tensor([T, 13][:B])
        t = torch.arange(T)
        slots = torch.where(t < lens[:, None], table.cpu()[:, t // bs] * bs + t % bs, -1).int().cuda()
        ref_pool, pool = m.new_paged_kvcache(num_blocks, bs), m.new_paged_kvcache(num_blocks, bs)
        lg0, _ = m.new_outputs(B, T, probs=False)
        lg1, _ = m.new_outputs(B, T, probs=False)
        tg = dev(tok)
        kv.pool = ref_pool.data_ptr()
        m.prefill_paged(tg, lg0, kv)
        kv.pool = pool.data_ptr()
        m.prefill_slots(tg, lg1, kv, slots)
        assert torch.equal(lg0, lg1)
        e = 2 if precision in (ab.GPT2_BF16, ab.GPT2_FP16) else 4
        view = lambda p: p.view(cfg.num_layers, 2, num_blocks, cfg.num_heads, bs, -1)  # noqa: E731
        a, b = view(ref_pool), view(pool)
        assert a.shape[-1] == cfg.head_size * e
        want = torch.zeros_like(a)
        for s in range(B):
            for p in range(int(lens[s])):
                want[:, :, table[s, p // bs], :, p % bs] = a[:, :, table[s, p // bs], :, p % bs]
        assert torch.equal(b, want)
        no_device_error()
        slots[0, 3] = num_blocks * bs
        m.prefill_slots(tg, lg1, kv, slots)
        assert ab.gpt2_get_error() == ab.DEVERR_BLOCK
        assert torch.equal(view(pool), want)


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_decode_loop_when_blocks_run_out(precision):
    """Continuations of one prompt with too few free blocks: those that get none
    wait (position -1) while the others go on, and go on themselves once there
    are blocks.  Every step stores at the granted slots and nowhere else (block
    0, which the entries of a new table name, is the prompt's), and a token's
    logits are those of a loop in which nobody waits."""
    w = inputs.WORKLOADS["tiny"]
    cfg = w.cfg
    params, _ = inputs.workload_inputs(w, "perturbed")
    B, bs, shared, n_own = 6, 4, 20, 9
    maxb = -(-(shared + n_own) // bs)
    n_pre, num_blocks = shared // bs, shared // bs + B * (maxb - shared // bs) + 1
    rng = np.random.default_rng(8)
    seq = rng.integers(0, cfg.vocab_size, (B, shared + n_own)).astype(np.int32)
    seq[:, :shared] = seq[0, :shared]
    m = GPT2Model(cfg, params, B, shared, precision)
    ids = dev(np.concatenate([np.arange(n_pre), n_pre + rng.permutation(num_blocks - n_pre)]).astype(np.int32))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    lg, _ = m.new_outputs(1, shared, probs=False)
    toks = dev(seq)

    def loop(free_at):
        """free_at(step): how many free blocks there are by then."""
        pool = m.new_paged_kvcache(num_blocks, bs)
        view = lambda p: p.view(cfg.num_layers, 2, num_blocks, cfg.num_heads, bs, -1)  # noqa: E731
        table = i32(B, maxb)
        kv = ab.paged_kv(pool, table, num_blocks, bs, maxb)
        m.prefill_slots(toks[:1, :shared].contiguous(), lg, kv, torch.arange(shared, dtype=torch.int32, device="cuda")[None])
        lens, taken = [torch.full((B,), shared, dtype=torch.int32, device="cuda"), i32(B)], [i32(1), i32(1)]
        slots, ws = i32(B, 1), m.new_shared_workspace(B, shared)
        pre, free = ids[:n_pre].clone(), ids[n_pre:].clone()
        got, waited, step = {}, 0, 0
        while int(lens[step % 2].min()) < shared + n_own and step < 40:
            a, b = step % 2, 1 - step % 2
            new = (lens[a] < shared + n_own).int()  # none for a sequence that has ended
            ab.paged_build_tables(table, slots, lens[b], taken[b], lens[a], new, free, free_at(step), taken[a], pre,
                                  shared, B, 1, num_blocks, bs, maxb)
            pos = torch.where(lens[b] > lens[a], lens[a], -1).int()
            tok = toks.gather(1, pos.long().clamp(min=0)[:, None])[:, 0].contiguous()
            logits, _ = m.new_outputs(B, None, probs=False)
            before = pool.clone()
            m.decode_step_shared(kv, tok, pos, shared, logits, ws)
            changed = (view(pool) != view(before)).any(5).any(3).any(1).any(0)  # [block, offset]
            assert set(changed.flatten().nonzero()[:, 0].tolist()) == {x for x in slots[:, 0].tolist() if x >= 0}
            for r, p in enumerate(pos.tolist()):
                if p >= 0:
                    got[r, p] = logits[r, :cfg.vocab_size].clone()
                else:
                    waited += int(new[r])
            step += 1
        no_device_error()
        return got, waited

    ample, none = loop(lambda step: num_blocks - n_pre)
    short, some = loop(lambda step: 4 if step < 3 else 7 if step < 6 else num_blocks - n_pre)
    assert none == 0 and some > 0
    assert sorted(ample) == sorted(short) == [(b, p) for b in range(B) for p in range(shared, shared + n_own)]
    for at in ample:
        assert torch.equal(short[at], ample[at]), at
    ref, _ = oracle.forward(cfg, params, seq)
    for (b, p), x in ample.items():
        assert_close(host(x), ref[b, p, :cfg.vocab_size], atol=LOGIT_TOL[precision], what=f"sequence {b} position {p}")


@pytest.mark.parametrize("precision", ALL, ids=[NAMES[p] for p in ALL])
def test_the_first_request_waits(precision):
    """A new request in row 0, through which the shared positions are read, gets
    no block while the others have room: their logits are those of a step whose
    row 0 was granted all along."""
    w = inputs.WORKLOADS["tiny"]
    cfg = w.cfg
    params, _ = inputs.workload_inputs(w, "perturbed")
    B, bs, shared, maxb = 5, 4, 20, 8
    n_pre, num_blocks = shared // bs, shared // bs + 5 + 1
    m = GPT2Model(cfg, params, B, shared, precision)
    toks = dev(inputs.make_tokens(9, B, shared, cfg.vocab_size))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = m.new_paged_kvcache(num_blocks, bs)
    # blocks 1 .. n_pre are the prompt's; 0 is nobody's
    pre = torch.arange(1, n_pre + 1, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pre + 1, num_blocks, dtype=torch.int32, device="cuda")
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    kv = ab.paged_kv(pool, table, num_blocks, bs, maxb)
    lg, _ = m.new_outputs(1, shared, probs=False)
    m.prefill_slots(toks[:1].contiguous(), lg, kv, torch.arange(bs, bs + shared, dtype=torch.int32, device="cuda")[None])
    ws = m.new_shared_workspace(B, shared)

    def step(lens, taken, tok):
        nxt, after = i32(B), i32(1)
        ab.paged_build_tables(table, None, nxt, after, lens, None, free, len(free), taken, pre, shared, B, 1, num_blocks,
                              bs, maxb)
        pos = torch.where(nxt > lens, lens, -1).int()
        logits, _ = m.new_outputs(B, None, probs=False)
        m.decode_step_shared(kv, tok, pos, shared, logits, ws)
        return nxt, after, pos, logits[:, :cfg.vocab_size]

    lens, taken, pos, _ = step(torch.full((B,), shared, dtype=torch.int32, device="cuda"), i32(1), toks[:, 0].contiguous())
    assert pos.tolist() == [shared] * B and int(taken) == B
    kept = pool.clone()
    _, _, pos, want = step(lens, taken, toks[:, 1].contiguous())
    assert pos.tolist() == [shared + 1] * B
    pool.copy_(kept)
    table[0] = -1
    fresh = lens.clone()
    fresh[0] = shared
    nxt, _, pos, got = step(fresh, taken, toks[:, 1].contiguous())
    assert pos.tolist() == [-1] + [shared + 1] * (B - 1) and int(nxt[0]) == shared
    assert torch.equal(got[1:], want[1:])
    no_device_error()
