"""The accepted path of each tree and its rows of the cache, against a plain form
step by step: whole numbers and copies, equal bit for bit."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab

from draft_reference import accept, chain, moved, trees
from gpu_helpers import dev, need_gpu, no_device_error

pytestmark = pytest.mark.gpu
DT = {ab.GPT2_FP32: torch.float32, ab.GPT2_TF32: torch.float32, ab.GPT2_BF16: torch.bfloat16,
      ab.GPT2_FP16: torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(precision, B, N, L, NH, hs, bs, seed, agree=0.8, missing=True, most=150):
    rng = np.random.default_rng(seed)
    parent = trees(B, N, seed, missing=missing, roots=True)
    tok = rng.integers(0, 30, (B, N)).astype(np.int32)  # few: equal tokens among siblings
    chosen = rng.integers(0, 30, (B, N)).astype(np.int32)
    for b in range(B):
        for i in range(N):
            kids = np.nonzero(parent[b] == i)[0]
            if len(kids) and rng.random() < agree:
                chosen[b, i] = tok[b, rng.choice(kids)]
    pos = rng.integers(0, most, B).astype(np.int32)
    if B > 3:
        pos[1] = -1
    row = (most + N) // bs + 1
    num_blocks = B * row + 2
    table = rng.permutation(num_blocks)[:B * row].reshape(B, row).astype(np.int32)
    for b in range(B):
        table[b, :max(0, pos[b]) // bs] = -7  # not reached
    words = 2 if DT[precision].itemsize == 2 else 4
    pool = rng.integers(0, 256, (L, 2, num_blocks, NH, bs, hs * words), dtype=np.uint8)
    return dict(precision=precision, B=B, N=N, L=L, NH=NH, hs=hs, bs=bs, parent=parent, tok=tok, chosen=chosen, pos=pos,
                table=table, pool=pool)


def config(c):
    return ab.GPT2Config(1 << 20, 100, 104, c["L"], c["NH"], c["NH"] * c["hs"])


def run(c, parent=True, cache=True, cfg=None):
    B, N = c["B"], c["N"]
    o = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B, N), (B,), (B,))]
    pool, table = dev(c["pool"]), dev(c["table"])
    kv = ab.paged_kv(pool, table, c["pool"].shape[2], c["bs"], c["table"].shape[1]) if cache else None
    ab.gpt2_accept_tree(*o, (cfg or config(c)) if cache else None, kv, dev(c["tok"]), dev(c["parent"]) if parent else None,
                        dev(c["chosen"]), dev(c["pos"]), B, N, c["precision"])
    torch.cuda.synchronize()
    path, count, emitted, tok, pos = (t.cpu().numpy() for t in o)
    return (path, emitted, count, tok, pos), pool.cpu().numpy()


def through_bad_entries(c, path):
    """Whether a row that moves needs a table entry outside the pool."""
    n, bs = c["pool"].shape[2], c["bs"]
    return any(not 0 <= c["table"][b, (int(c["pos"][b]) + p) // bs] < n for b in range(c["B"])
               for k, i in enumerate(path[b]) if i >= 0 and i != k for p in (int(i), k))


def check(c, capacity=1 << 30, **kw):
    got, pool = run(c, **kw)
    parent = c["parent"] if kw.get("parent", True) else chain(c["B"], c["N"])
    want = accept(c["tok"], parent, c["chosen"], c["pos"], capacity)
    for a, b, name in zip(got, want, ("path", "emitted", "count", "next_tok", "next_pos")):
        assert np.array_equal(a, b), name
    after = moved(c["pool"], c["table"], want[0], c["pos"], c["bs"]) if kw.get("cache", True) else c["pool"]
    assert np.array_equal(pool, after), "the cache"
    return got


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16])
@pytest.mark.parametrize("B,N,L,NH,hs,bs", [
    (1, 1, 1, 1, 16, 1), (1, 2, 2, 1, 16, 2), (3, 5, 3, 2, 32, 16), (7, 16, 2, 3, 64, 4), (5, 31, 1, 12, 64, 8),
    (4, 32, 4, 2, 16, 32), (6, 33, 2, 1, 64, 16), (9, 64, 3, 4, 64, 16), (70, 64, 1, 2, 32, 64), (300, 3, 1, 1, 16, 8),
])
def test_against_steps(precision, B, N, L, NH, hs, bs):
    c = make(precision, B, N, L, NH, hs, bs, seed=B + N)
    got = check(c)
    assert N < 16 or got[2].max() > 2  # something is accepted
    no_device_error()


def test_all_and_none_of_a_chain():
    c = make(ab.GPT2_FP16, 3, 64, 2, 2, 64, 16, seed=1)
    c["tok"] = np.tile(np.arange(64, dtype=np.int32) + 5, (3, 1))
    c["chosen"] = c["tok"] + 1
    c["chosen"][1, 0] = 3
    got = check(c, parent=False)
    assert got[2].tolist() == [64, 1, 64] and got[3].tolist() == [69, 3, 69]
    no_device_error()


def test_the_lowest_of_equal_children():
    c = make(ab.GPT2_FP16, 1, 8, 1, 1, 16, 4, seed=1)
    c["parent"] = np.array([[-1, 0, 0, 0, 2, 3, 2, 4]], np.int32)
    c["tok"] = np.array([[1, 8, 9, 9, 4, 4, 4, 6]], np.int32)
    c["chosen"] = np.array([[9, 0, 4, 4, 6, 6, 6, 2]], np.int32)
    got = check(c)
    assert got[0][0].tolist() == [0, 2, 4, 7, -1, -1, -1, -1] and got[1][0, :4].tolist() == [9, 4, 6, 2]


def test_every_path_through_a_tree():
    """Paths of all shapes, also ones whose rows overlap the places they go to."""
    N = 40
    for seed in range(6):
        c = make(ab.GPT2_BF16, 64, N, 1, 2, 32, 8, seed=seed, agree=1.0, missing=False)
        got = check(c)
        assert got[2].max() > 4
    no_device_error()


def test_without_a_cache_and_without_outputs():
    c = make(ab.GPT2_FP32, 5, 20, 2, 2, 32, 16, seed=3)
    check(c, cache=False)
    pool, table = dev(c["pool"]), dev(c["table"])
    kv = ab.paged_kv(pool, table, c["pool"].shape[2], c["bs"], c["table"].shape[1])
    ab.gpt2_accept_tree(None, None, None, None, None, config(c), kv, dev(c["tok"]), dev(c["parent"]), dev(c["chosen"]),
                        dev(c["pos"]), 5, 20, c["precision"])
    want = accept(c["tok"], c["parent"], c["chosen"], c["pos"])
    assert np.array_equal(pool.cpu().numpy(), moved(c["pool"], c["table"], want[0], c["pos"], c["bs"]))
    no_device_error()


def test_bad_positions_nodes_and_blocks():
    c = make(ab.GPT2_FP16, 6, 24, 2, 2, 32, 16, seed=5, agree=1.0, missing=False)
    cap = c["table"].shape[1] * 16

    def bits(got):  # entries of positions that make() took for not reached are outside the pool
        return ab.DEVERR_BLOCK if through_bad_entries(c, got[0]) else 0

    c["pos"][:] = [-2, -1, cap, 2**31 - 1, 40, -2**31]
    got = check(c, capacity=cap)
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION | bits(got)
    c["pos"][:] = [cap - 24, cap - 23, cap - 1, 0, cap - 4, 5]
    got = check(c, capacity=cap)  # a path ends where the places do
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION | bits(got)
    c["pos"][:] = [30, 8, 100, 0, 77, 5]
    got = check(c, cfg=ab.GPT2Config(60, 100, 104, 2, 2, 64), capacity=60)  # a model of 60 positions
    assert ab.gpt2_get_error() == ab.DEVERR_POSITION | bits(got)
    c["parent"][2, 9], c["parent"][3, 1] = 9, -4
    c["table"][c["table"] < 0] = 0
    got = check(c)
    assert ab.gpt2_get_error() == ab.DEVERR_TREE | bits(got)
    flagged = []
    for value in (-1, 10**6):
        c = make(ab.GPT2_FP16, 6, 24, 2, 2, 32, 16, seed=5, agree=1.0, missing=False)
        c["table"][:, :] = np.arange(c["table"].size).reshape(c["table"].shape) % c["pool"].shape[2]
        c["pos"][:] = [0, 8, 16, 3, 31, 5]
        c["table"][0, 1] = c["table"][4, 2] = value
        got = check(c)
        flagged.append(bits(got))
        assert ab.gpt2_get_error() == flagged[-1]
    assert any(flagged)


def test_offsets_past_32_bits():
    """A cache whose layers lie beyond byte 2^32."""
    c = make(ab.GPT2_FP16, 2, 20, 2, 4, 64, 64, seed=7, agree=1.0, missing=False)
    far = (1 << 32) // (4 * 64 * 128) + 3
    pool = torch.zeros(2, 2, far + c["pool"].shape[2], 4, 64, 128, dtype=torch.uint8, device="cuda")
    pool[:, :, far:] = dev(c["pool"])
    table = dev(np.where(c["table"] >= 0, c["table"] + far, c["table"]).astype(np.int32))
    kv = ab.paged_kv(pool, table, pool.shape[2], 64, c["table"].shape[1])
    count = torch.empty(2, dtype=torch.int32, device="cuda")
    ab.gpt2_accept_tree(None, count, None, None, None, config(c), kv, dev(c["tok"]), dev(c["parent"]), dev(c["chosen"]),
                        dev(c["pos"]), 2, 20, c["precision"])
    want = accept(c["tok"], c["parent"], c["chosen"], c["pos"])
    assert np.array_equal(count.cpu().numpy(), want[2]) and (want[0][:, 1] > 1).any()
    assert np.array_equal(pool[:, :, far:].cpu().numpy(), moved(c["pool"], c["table"], want[0], c["pos"], c["bs"]))
    assert not pool[:, :, :far].any()
    no_device_error()


@pytest.mark.parametrize("precision", [ab.GPT2_FP32, ab.GPT2_FP16], ids=["fp32", "fp16"])
def test_graph_and_streams(precision):
    """Captured once and replayed on other trees; two on two streams."""
    cs = [make(precision, 6, 21, 2, 3, 16, 4, seed=s) for s in (1, 2)]
    want = [run(c) for c in cs]
    names = ("pool", "table", "tok", "parent", "chosen", "pos")
    state = []
    for _ in range(2):
        t = {k: dev(cs[0][k].copy()) for k in names}
        o = [torch.empty(x, dtype=torch.int32, device="cuda") for x in ((6, 21), (6,), (6, 21), (6,), (6,))]
        kv = ab.paged_kv(t["pool"], t["table"], cs[0]["pool"].shape[2], 4, cs[0]["table"].shape[1])
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            ab.gpt2_accept_tree(*o, config(cs[0]), kv, t["tok"], t["parent"], t["chosen"], t["pos"], 6, 21, precision, s)
        state.append((t, o, s, g))
    for round in range(4):
        for k, (t, o, s, g) in enumerate(state):
            with torch.cuda.stream(s):
                for n in names:
                    t[n].copy_(torch.from_numpy(cs[(round + k) % 2][n]))
                g.replay()
        torch.cuda.synchronize()
        for k, (t, o, s, g) in enumerate(state):
            (path, emitted, count, tok, pos), pool = want[(round + k) % 2]
            for a, b in zip(o, (path, count, emitted, tok, pos)):
                assert np.array_equal(a.cpu().numpy(), b)
            assert np.array_equal(t["pool"].cpu().numpy(), pool)
    no_device_error()


def test_one_node_and_full_trees_of_many_sequences():
    for B, N in ((1, 1), (700, 1), (400, 64)):
        check(make(ab.GPT2_BF16, B, N, 1, 1, 16, 16, seed=B))
    no_device_error()
