"""Block tables and slot maps built on the GPU [NTU "KV Caching"], exactly
against a request-by-request construction on the CPU: growing and admitted
requests, shared prefixes, requests that must wait, bad lengths and block ids,
decode loops with swapped buffers, and a captured step."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab

from gpu_helpers import dev, need_gpu, no_device_error
from serve_reference import tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(B, T, bs, max_cached, prefix_len, seed, spare=4, taken=2, extra=3):
    rng = np.random.default_rng(seed)
    cached = (prefix_len + rng.integers(0, max(1, max_cached - prefix_len + 1), B)).astype(np.int32)
    new = rng.integers(0, T + 1, B).astype(np.int32)
    maxb = -(-(max(max_cached, prefix_len) + T) // bs) + extra
    held = B * maxb
    num_blocks = 2 * held + prefix_len // bs + 8
    ids = rng.permutation(num_blocks).astype(np.int32)
    table = ids[:held].reshape(B, maxb).copy()
    pre = ids[held:held + prefix_len // bs]
    table[:, :prefix_len // bs] = pre
    want = sum(-(-(int(c) + int(n)) // bs) - -(-int(c) // bs) for c, n in zip(cached, new))
    free = ids[held + len(pre):held + len(pre) + taken + max(0, want + spare)].copy()
    return dict(table=table, cached=cached, new=new, free=free, taken=taken, pre=pre, prefix_len=prefix_len, T=T, bs=bs,
                num_blocks=num_blocks)


def run(c, slots=True, **change):
    a = dict(c, **change)
    B, maxb = a["table"].shape
    t = dev(a["table"])
    out = dict(slots=torch.full((B, a["T"]), 77, dtype=torch.int32, device="cuda"),
               nxt=torch.full((B,), 77, dtype=torch.int32, device="cuda"),
               taken=torch.full((1,), 77, dtype=torch.int32, device="cuda"))
    ab.paged_build_tables(t, out["slots"] if slots else None, out["nxt"], out["taken"], dev(a["cached"]),
                          dev(a["new"]) if a["new"] is not None else None, dev(a["free"]) if len(a["free"]) else None,
                          len(a["free"]), dev(np.array([a["taken"]], np.int32)),
                          dev(a["pre"]) if a["prefix_len"] else None, a["prefix_len"], B, a["T"], a["num_blocks"],
                          a["bs"], maxb)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, out["slots"], out["nxt"], out["taken"])]


def check(c, bits=0, **change):
    a = dict(c, **change)
    got = run(c, **change)
    assert ab.gpt2_get_error() == bits
    table, slots, nxt, taken, ref_bits = tables(a["table"], a["cached"], a["new"], a["free"], a["taken"], a["pre"],
                                                a["prefix_len"], a["T"], a["num_blocks"], a["bs"])
    assert ref_bits == bits
    np.testing.assert_array_equal(got[2], nxt)
    np.testing.assert_array_equal(got[0], table)
    np.testing.assert_array_equal(got[1], slots)
    assert got[3][0] == taken
    return got


@pytest.mark.parametrize("B,T,bs,cached,prefix", [
    (1, 1, 1, 0, 0), (1, 1, 16, 15, 0), (3, 1, 16, 64, 0), (32, 1, 16, 1000, 0), (33, 1, 1, 40, 0), (7, 5, 4, 0, 0),
    (5, 300, 16, 100, 32), (64, 37, 8, 200, 64), (256, 129, 16, 512, 256), (1000, 3, 2, 9, 4), (304, 1, 32, 900, 0),
    (305, 2, 64, 900, 128), (4097, 1, 16, 333, 16), (2, 4000, 64, 3, 0), (3, 0, 16, 20, 16),
])
def test_against_cpu(B, T, bs, cached, prefix):
    check(make(B, T, bs, cached, prefix, seed=B + T))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("spare", [-1, -7, -40])
def test_requests_wait_when_blocks_run_out(seed, spare):
    c = make(40, 20, 4, 60, 8, seed=seed, spare=spare)
    got = check(c)
    waiting = got[2] == c["cached"]
    assert (waiting & (c["new"] > 0)).any()
    no = c["new"] == 0
    assert (got[2][no] == c["cached"][no]).all()


@pytest.mark.parametrize("taken", [0, 5, 6, 7, -3])
def test_no_blocks_left(taken):
    c = make(20, 9, 4, 30, 0, seed=9)
    check(c, free=c["free"][:5].copy(), taken=taken)
    check(c, free=c["free"][:0].copy(), taken=0)


def test_defaults():
    # new_len NULL: one token each; taken_in NULL: from the first block; no
    # prefix; outputs that are not asked for
    c = make(50, 1, 16, 100, 0, seed=3, spare=60)
    check(c, new=None)
    t = dev(c["table"])
    ab.paged_build_tables(t, None, None, None, dev(c["cached"]), None, dev(c["free"]), len(c["free"]), None, None, 0, 50,
                          1, c["num_blocks"], 16, t.shape[1])
    ref = tables(c["table"], c["cached"], None, c["free"], 0, c["pre"], 0, 1, c["num_blocks"], 16)
    np.testing.assert_array_equal(t.cpu().numpy(), ref[0])
    no_device_error()


def test_bad_lengths_are_refused_on_the_device():
    c = make(12, 6, 4, 40, 8, seed=5, spare=20)
    cap = c["table"].shape[1] * 4
    cached, new = c["cached"].copy(), c["new"].copy()
    cached[1], new[2], new[3], cached[4], cached[6] = -1, -2, 7, cap + 1, 2**31 - 1
    cached[7], new[7] = cap, 1
    cached[8], new[8] = 7, 3  # shorter than the prefix
    cached[9], new[9] = cap, 0
    got = check(c, bits=ab.DEVERR_POSITION, cached=cached, new=new)
    assert (got[1][[1, 2, 3, 4, 6, 7, 8]] == -1).all()


def test_bad_blocks_are_flagged():
    c = make(12, 6, 4, 40, 8, seed=6, spare=20)
    c["cached"][:] = 4 * (c["cached"] // 4) + 1  # a partly filled block is in use
    c["cached"][:] = np.maximum(c["cached"], 9)
    c["new"][:] = 6
    c = dict(c, free=np.concatenate([c["free"], c["free"]])[:60])
    free, table = c["free"].copy(), c["table"].copy()
    free[c["taken"] + 2] = c["num_blocks"]
    table[5, c["cached"][5] // 4] = -9
    check(c, bits=ab.DEVERR_BLOCK, free=free, table=table)


def test_decode_loop_with_swapped_buffers_in_a_graph():
    B, bs, steps, maxb = 9, 4, 21, 8
    rng = np.random.default_rng(1)
    start = rng.integers(0, 5, B).astype(np.int32)
    num_blocks = B * maxb + 3
    free = rng.permutation(num_blocks).astype(np.int32)
    table = np.full((B, maxb), -1, np.int32)
    used = 0
    for b in range(B):
        n = -(-int(start[b]) // bs)
        table[b, :n] = free[used:used + n]
        used += n
    t, fr = dev(table), dev(free)
    lens = [dev(start), torch.zeros(B, dtype=torch.int32, device="cuda")]
    taken = [dev(np.array([used], np.int32)), torch.zeros(1, dtype=torch.int32, device="cuda")]
    slots = torch.zeros(2, B, 1, dtype=torch.int32, device="cuda")

    def step(i):
        ab.paged_build_tables(t, slots[i], lens[1 - i], taken[1 - i], lens[i], None, fr, num_blocks, taken[i], None, 0, B,
                              1, num_blocks, bs, maxb)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(0)
        step(1)
    ref_t, ref_l, ref_u = table, start.astype(np.int64), used
    for i in range(0, steps, 2):
        graph.replay()
        torch.cuda.synchronize()
        for k in range(2):
            ref_t, ref_s, ref_l, ref_u, bits = tables(ref_t, ref_l, None, free, ref_u, None, 0, 1, num_blocks, bs)
            assert bits == 0
            np.testing.assert_array_equal(slots[k].cpu().numpy(), ref_s)
        np.testing.assert_array_equal(t.cpu().numpy(), ref_t)
        np.testing.assert_array_equal(lens[0].cpu().numpy(), ref_l)
        assert int(taken[0]) == ref_u
    no_device_error()


def test_another_stream():
    c = make(64, 37, 8, 200, 64, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check(c)


@pytest.mark.parametrize("refused", ["waits", "bad length"])
def test_every_row_gets_the_shared_prefix(refused):
    """Request 0 gets nothing while the others, whose last block has room, are
    granted: its row holds the prefix's blocks all the same, since a decode step
    over the shared prefix reads them there."""
    B, bs, P, maxb, num_blocks = 5, 4, 24, 10, 40
    table = np.full((B, maxb), -1, np.int32)
    pre = np.arange(30, 30 + P // bs, dtype=np.int32)
    cached = np.array([P, P + 1, P + 2, P + 3, P + 1], np.int32)
    table[1:, P // bs] = np.arange(3, 3 + B - 1)
    new = np.array([1 if refused == "waits" else 2, 1, 1, 1, 0], np.int32)
    want = table.copy()
    want[:, :P // bs] = pre
    t = dev(table)
    nxt = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    ab.paged_build_tables(t, slots, nxt, None, dev(cached), dev(new), None, 0, None, dev(pre), P, B, 1, num_blocks, bs,
                          maxb)
    assert ab.gpt2_get_error() == (0 if refused == "waits" else ab.DEVERR_POSITION)
    np.testing.assert_array_equal(t.cpu().numpy(), want)
    np.testing.assert_array_equal(nxt.cpu().numpy(), [P, P + 2, P + 3, P + 4, P + 1])
    np.testing.assert_array_equal(slots.cpu().numpy()[:, 0], [-1, 13, 18, 23, -1])
