"""Attention of trees over tables as wide as a model's context whatever the texts'
lengths: both sides of the rules that choose the kernels, repeated and concurrent
calls, many sequences.  Inputs, the 64-bit form and the tolerance are those of
test_gpu_tree_attention."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab

from draft_reference import trees
from gpu_helpers import need_gpu, no_device_error
from test_gpu_tree_attention import DT, IDS, TYPES, cache_after, call, check, make, on_gpu, ragged, reference, run, same

pytestmark = pytest.mark.gpu
TYPES16, IDS16 = [ab.GPT2_BF16, ab.GPT2_FP16], ["bf16", "fp16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def wide(precision, B, N, NH, most, capacity, bs=16, seed=1, hs=64):
    """Texts of 0 to `most` positions in a table of `capacity`."""
    pos = ragged(B, most, seed)
    row = (most + N - 1) // bs + 1
    c = make(precision, N, NH, hs, pos, bs, trees(B, N, seed=seed), seed=seed, spare=capacity // bs - row)
    assert c["table"].shape[1] * bs == capacity
    return c


@pytest.mark.parametrize("precision", TYPES16, ids=IDS16)
@pytest.mark.parametrize("B,NH,capacity,most", [
    (26, 12, 1024, 60), (26, 12, 1024, 500), (26, 12, 1040, 60), (25, 12, 1024, 60), (25, 12, 768, 300),
    (13, 12, 768, 700), (12, 12, 1024, 300), (8, 38, 1024, 960), (1, 12, 1024, 960), (101, 3, 1024, 90),
])
@pytest.mark.parametrize("N", [33, 64])
def test_wide_trees_in_a_models_context(precision, B, NH, capacity, most, N):
    """On both sides of two pairs an SM and one, and of 768 and 1024 positions."""
    check(wide(precision, B, N, NH, most, capacity, seed=B + N))
    no_device_error()


# each of the kernels: pairs of a CTA each, shares, tcgen05
KERNELS = [(6, 40, 2, 700, 768), (40, 16, 12, 300, 512), (9, 16, 3, 900, 2048), (9, 24, 4, 900, 2048), (5, 5, 4, 200, 384),
           (16, 64, 4, 3000, 4096), (30, 48, 3, 700, 2048)]


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("B,N,NH,most,capacity", KERNELS)
def test_the_same_bits_whatever_else_runs(precision, B, N, NH, most, capacity):
    """Over a fresh cache and the one that a first call left, a workspace of other
    calls, and beside another stream's work."""
    c = wide(precision, B, N, NH, most, capacity, bs=64, seed=N)
    t = on_gpu(c)
    pool = t["pool"].clone()
    out = torch.empty(B * N, NH * 64, dtype=DT[precision], device="cuda")
    ws = call(c, t, out)
    want, after = out.clone(), t["pool"].clone()
    side, x = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    for k in range(12):
        out.fill_(9)
        if k % 3 == 0:
            t["pool"].copy_(pool)
        if k % 4 == 1:
            ws.fill_(k)
        side.wait_stream(torch.cuda.current_stream())
        if k >= 6:
            with torch.cuda.stream(side):
                for _ in range(3):
                    x @ x
        call(c, t, out, ws)
        torch.cuda.synchronize()
        assert same(out, want) and same(t["pool"], after), k
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("B,N,NH,most,capacity", KERNELS)
def test_two_graphs_on_two_streams(precision, B, N, NH, most, capacity):
    """With outputs, caches and workspaces of their own, replayed at the same time."""
    cs = [wide(precision, B, N, NH, most, capacity, bs=64, seed=s) for s in (3, 4)]
    want = [run(c) for c in cs]
    graphs = []
    for c in cs:
        t, s, g = on_gpu(c), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        out = torch.empty(B * N, NH * 64, dtype=DT[precision], device="cuda")
        ws = torch.empty(ab.attention_tree_workspace_size(B, N, NH * 64, NH, precision), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            for _ in range(4):
                call(c, t, out, ws, stream=s)
        graphs.append((t, s, g, out, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for _, s, g, _, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (t, _, _, out, _), (o, p) in zip(graphs, want):
        assert same(out.cpu().view(o.shape), o) and same(t["pool"].cpu(), p)
    no_device_error()


@pytest.mark.parametrize("precision", TYPES, ids=IDS)
@pytest.mark.parametrize("N,NH,hs,capacity", [(1, 1, 16, 256), (3, 2, 16, 2048), (20, 1, 32, 2048), (40, 1, 64, 1040)])
def test_thousands_of_sequences(precision, N, NH, hs, capacity):
    """Many more pairs than shares, all of them short; some are compared with 64 bits,
    in this call and in smaller ones."""
    B, most = 4100, 30
    rng = np.random.default_rng(N)
    pos = rng.integers(-1, most + 1, B).astype(np.int32)
    pos[0], pos[-1] = most, 7
    bs, row = 16, (most + N - 1) // 16 + 1
    c = make(precision, N, NH, hs, pos, bs, trees(B, N, seed=N), seed=N, spare=capacity // bs - row)
    out, pool = run(c)
    some = list(range(0, B, 64)) + [B - 1]

    def part(rows):
        rows = torch.as_tensor(rows)
        at = (rows[:, None] * N + torch.arange(N)).flatten()
        return dict(c, pos=c["pos"][rows], parent=c["parent"][rows], table=c["table"][rows].contiguous(), qkv=c["qkv"][at])

    ref, tol, there = reference(part(some))
    assert (np.abs(out[some].double().numpy() - ref) <= tol).all() and (out[some].float().numpy()[~there] == 0).all()
    assert same(pool, cache_after(c))
    for rows in np.array_split(np.arange(B), 40)[::13]:
        few = part(rows)
        small, _ = run(few)
        ref, tol, _ = reference(few)
        assert (np.abs(small.double().numpy() - ref) <= tol).all()
        assert (np.abs(out[rows].double().numpy() - ref) <= tol).all()
    no_device_error()
