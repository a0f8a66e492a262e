"""Penalties, biases and masks on logits [llm.c classifier], against a 64-bit
form that goes token by token.

Tolerances: u = 2^-24.  A penalised value passes at most six fp32 roundings (the
penalty by repetition, the frequency's product and difference, the presence's
difference, the bias's sum), each off by at most u times the largest value on the
way, and one rounding to the logits' type: half a step, u (fp32), 2^-11 (fp16,
at least 2^-25) or 2^-8 (bf16) relative to the result.  Everything else is equal
bit for bit."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab

from draft_reference import adjust, chain, trees
from gpu_helpers import need_gpu, no_device_error

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF = {torch.float32: u, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(dtype, B, N, V, H=50, M=9, G=3, seed=0, pad=None, path=True, parent="trees", **without):
    rng = np.random.default_rng(seed)
    kN = 4 if dtype == torch.float32 else 8
    Vp = (V + (int(rng.integers(0, 40)) if pad is None else pad) + kN - 1) // kN * kN
    x = torch.from_numpy(rng.normal(size=(B * N, Vp)).astype(np.float32) * 3).to(dtype)
    few = rng.permutation(V)[:max(1, min(V, 40))].astype(np.int32)  # tokens that come often
    c = dict(dtype=dtype, B=B, N=N, V=V, Vp=Vp, x=x, H=H, M=M, G=G,
             tok=rng.choice(few, (B, N)).astype(np.int32) if path else None,
             parent=trees(B, N, seed, roots=True) if isinstance(parent, str) else parent)
    history = rng.choice(few, (B, H)).astype(np.int32)
    history[rng.random((B, H)) < 0.1] = -1
    n = rng.integers(0, H + 1, B).astype(np.int32)
    c["rules"] = dict(
        history=history if H else None, history_len=n if H else None,
        prompt_len=(n * rng.random(B)).astype(np.int32) if H else None,
        repetition=(0.7 + rng.random(B)).astype(np.float32), presence=rng.normal(size=B).astype(np.float32),
        frequency=rng.normal(size=B).astype(np.float32),
        bias_ids=np.where(rng.random((B, M)) < 0.2, -1, rng.choice(few, (B, M))).astype(np.int32) if M else None,
        bias_values=(rng.normal(size=(B, M)) * 5).astype(np.float32) if M else None,
        masks=rng.integers(0, 2**32, (G, (V + 31) // 32), dtype=np.uint32) if G else None,
        mask_rows=rng.integers(-1, G, B * N).astype(np.int32) if G else None)
    c["rules"].update(without)
    return c


def gpu(a):
    return None if a is None else torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()


def rules_of(c):
    r = {k: gpu(v) for k, v in c["rules"].items()}
    some = lambda k, n: n if c["rules"][k] is not None else 0  # noqa: E731
    return ab.logit_rules(**r, history_stride=some("history", c["H"]), num_bias=some("bias_ids", c["M"]),
                          num_masks=some("masks", c["G"]))


def run(c, in_place=False):
    B, N, Vp = c["B"], c["N"], c["Vp"]
    buf = torch.full((B * N + 2, Vp), 7.0, dtype=c["dtype"], device="cuda")
    x = c["x"].cuda()
    if in_place:
        buf[1:-1] = x
        x = buf[1:-1]
    ab.logits_adjust(buf[1:-1], x, ab.element_type(x), rules_of(c), gpu(c["tok"]), gpu(c["parent"]), B, N, c["V"], Vp)
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[-1] == 7).all(), "rows around the output"
    if not in_place:
        assert torch.equal(x.cpu().view(torch.uint8), c["x"].view(torch.uint8)), "the logits"
    return buf[1:-1].cpu()


def check(c):
    B, N, V = c["B"], c["N"], c["V"]
    dt = c["dtype"]
    parent = chain(B, N) if c["parent"] is None else c["parent"]
    x = c["x"][:, :V].double().numpy().reshape(B, N, V)
    ref, size, there = adjust(x, V, tok=c["tok"], parent=parent, **c["rules"])
    for in_place in (False, True):
        out = run(c, in_place)
        got = out.double().numpy().reshape(B, N, -1)
        assert (got[there][:, V:] == -np.inf).all(), "the padding"
        if not in_place:
            assert (got[~there] == 7).all(), "a missing node's row"
        else:
            assert np.array_equal(got[~there], c["x"].double().numpy().reshape(B, N, -1)[~there], equal_nan=True)
        a, b, s = got[there][:, :V], ref[there], size[there]
        untouched = x[there] == b
        assert (a[untouched] == b[untouched]).all(), "tokens that nothing names"
        inf = np.isinf(b)
        assert np.array_equal(a[inf], b[inf])
        tol = 6 * u * s + HALF[dt] * (np.abs(np.where(inf, 0, b)) + 6 * u * s) + (2.0 ** -25 if dt == torch.float16 else 0)
        err = np.abs(a[~inf] - b[~inf])
        assert (err <= tol[~inf]).all(), (err / np.maximum(tol[~inf], 1e-30)).max()
    return ref, there


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("B,N,V,H,M,G,pad", [
    (1, 1, 1, 0, 0, 0, 0), (1, 1, 1, 3, 1, 1, 7), (2, 1, 31, 5, 2, 1, 0), (3, 2, 32, 40, 9, 2, 1), (1, 5, 33, 1, 0, 3, 0),
    (2, 9, 1000, 300, 17, 0, 0), (5, 3, 1025, 7, 0, 4, 8), (1, 64, 2047, 100, 200, 7, 0), (2, 33, 8192, 64, 3, 2, 0),
    (3, 8, 8193, 500, 1023, 5, 0), (1, 1, 50257, 2000, 20, 1, 47), (40, 16, 8300, 30, 5, 3, 100),
])
def test_against_64_bits(dtype, B, N, V, H, M, G, pad):
    check(make(dtype, B, N, V, H, M, G, seed=V + N, pad=pad))
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_large_rows_of_many_nodes(dtype):
    """Whole vocabularies, segments of the largest size, groups of nodes."""
    check(make(dtype, 24, 12, 50257, 300, 20, 6, seed=5, pad=47))
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("B,N,H,M", [(160, 1, 80, 5), (160, 1, 300, 0), (90, 3, 0, 85), (60, 9, 85, 0), (60, 9, 900, 40)])
def test_tokens_that_share_their_low_bits(dtype, B, N, H, M):
    """Multiples of 128 and of 512: where few tokens of a segment can be named they
    stand in a table of a power of two entries."""
    V = 32003
    c = make(dtype, B, N, V, H, M, 2, seed=H + M, pad=5)
    rng = np.random.default_rng(H)
    pick = lambda shape: (rng.integers(0, V // 512, shape) * 512 + rng.choice([0, 128, 7], shape)).astype(np.int32)  # noqa: E731
    c["tok"] = pick((B, N))
    if H:
        c["rules"]["history"] = pick((B, H))
        c["rules"]["history_len"][:] = H
    if M:
        c["rules"]["bias_ids"] = pick((B, M))
    check(c)
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_histories_of_distinct_tokens(dtype):
    """As many tokens of a segment as a history has, and every token of it."""
    for V, H, B in ((1024, 1024, 3), (8192, 1365, 200), (5000, 4990, 2)):
        c = make(dtype, B, 2, V, H, 3, 0, seed=H, pad=0)
        rng = np.random.default_rng(V)
        c["rules"]["history"] = np.stack([rng.permutation(min(V, 8192 if V != 8192 else 1400))[:H] for _ in range(B)]).astype(np.int32)
        c["rules"]["history_len"][:] = H
        c["rules"]["prompt_len"][:] = H // 3
        check(c)
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_calls_behind_each_other_in_place(dtype):
    """Twice in place, the second on what the first wrote, no wait between them."""
    c = make(dtype, 7, 5, 3000, 60, 5, 3, seed=3, pad=8)
    once = run(c)
    twice = run(dict(c, x=torch.where((once == 7).all(1, keepdim=True), c["x"], once)))
    x = c["x"].cuda()
    rules, tok, parent = rules_of(c), gpu(c["tok"]), gpu(c["parent"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        ab.logits_adjust(x, x, ab.element_type(x), rules, tok, parent, 7, 5, 3000, c["Vp"], s)
    s.synchronize()
    there = ~(once == 7).all(1)
    assert torch.equal(x.cpu()[there], twice[there])
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("left", [
    dict(repetition=None), dict(presence=None), dict(frequency=None), dict(bias_ids=None, bias_values=None),
    dict(masks=None, mask_rows=None), dict(history=None, history_len=None, prompt_len=None), dict(history_len=None),
    dict(prompt_len=None), dict(repetition=None, presence=None, frequency=None),
    dict(history=None, history_len=None, prompt_len=None, bias_ids=None, bias_values=None),
], ids=lambda d: "-".join(d))
@pytest.mark.parametrize("path", [True, False])
def test_parts_left_out(dtype, left, path):
    c = make(dtype, 3, 4, 3001, seed=2, path=path, **left)
    if left.get("history_len", 1) is None and c["rules"]["history"] is not None:
        c["rules"]["prompt_len"] = np.minimum(c["rules"]["prompt_len"], c["H"])
    check(c)
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_values_at_the_ends(dtype):
    """Infinities, NaN, zeros of both signs, the type's largest and lowest
    values; rows whose mask leaves nothing."""
    c = make(dtype, 2, 3, 600, H=200, M=5, G=2, seed=4, parent=None)
    fi = torch.finfo(dtype)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, fi.max, fi.min, fi.tiny], dtype=dtype)
    c["x"][:, :600] = odd[torch.arange(600) % 8]
    c["rules"]["masks"][1] = 0
    c["rules"]["mask_rows"] = np.array([0, 1, -1, -1, 1, 0], np.int32)
    out = run(c)
    again = run(c, True)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
    got = out.double().numpy()
    assert (got[[1, 4]] == -np.inf).all()
    v = np.arange(600)
    free = ((c["rules"]["masks"][0, v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)
    assert (got[0, :600][~free] == -np.inf).all()  # a NaN too
    with np.errstate(all="ignore"):
        ref, _, _ = adjust(c["x"][:, :600].double().numpy().reshape(2, 3, 600), 600, tok=c["tok"], parent=chain(2, 3),
                           **c["rules"])
    ref = torch.from_numpy(ref.reshape(6, 600)).to(dtype).double().numpy()  # overflow is an infinity
    for r in (0, 2, 3, 5):
        a, b = got[r, :600], ref[r]
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b)), r
    no_device_error()


def test_a_later_bias_counts():
    c = make(torch.float32, 1, 1, 100, H=0, M=4, G=0, seed=1, path=False, repetition=None, presence=None, frequency=None)
    c["rules"]["bias_ids"] = np.array([[5, 9, 5, -1]], np.int32)
    out = run(c)
    b = c["rules"]["bias_values"][0]
    assert out[0, 5] == c["x"][0, 5] + float(b[2]) and out[0, 9] == c["x"][0, 9] + float(b[1])


def test_a_token_many_times():
    """The whole history one token, and the longest path."""
    c = make(torch.float32, 2, 64, 500, H=100000, M=0, G=0, seed=1, parent=None)
    c["rules"]["history"][:] = 77
    c["rules"]["history_len"][:] = [100000, 1]
    c["rules"]["prompt_len"][:] = 0
    c["tok"][:] = 77
    check(c)
    no_device_error()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_bad_tokens_lengths_and_masks(dtype):
    c = make(dtype, 3, 4, 700, parent=chain(3, 4), seed=6)
    for name, at, value, bit in (("history", (1, 2), 700, ab.DEVERR_TOKEN), ("history", (0, 0), -2, ab.DEVERR_TOKEN),
                                 ("bias_ids", (2, 3), 2**31 - 1, ab.DEVERR_TOKEN), ("history_len", 1, 51, ab.DEVERR_POSITION),
                                 ("history_len", 0, -1, ab.DEVERR_POSITION), ("prompt_len", 2, -5, ab.DEVERR_POSITION),
                                 ("prompt_len", 2, 1000, ab.DEVERR_POSITION), ("mask_rows", 3, 3, ab.DEVERR_TREE),
                                 ("mask_rows", 11, -2, ab.DEVERR_TREE)):
        d = dict(c, rules={k: None if v is None else v.copy() for k, v in c["rules"].items()})
        d["rules"]["history_len"][:] = 50
        if name == "history_len" and value == -1:
            d["rules"]["prompt_len"][0] = 0
        d["rules"][name][at] = value
        check(d)
        assert ab.gpt2_get_error() == bit, name
    d = dict(c, tok=c["tok"].copy())
    d["tok"][0, 1] = 700
    check(d)
    assert ab.gpt2_get_error() == ab.DEVERR_TOKEN
    d = dict(c, parent=c["parent"].copy())
    d["parent"][1, 2] = 2
    d["tok"] = c["tok"].copy()
    d["tok"][1, 2:] = 10**6  # of missing nodes: not read
    check(d)
    assert ab.gpt2_get_error() == ab.DEVERR_TREE


def test_offsets_past_32_bits():
    """Rows on both sides of element 2^31."""
    V = Vp = 50304
    rows = (1 << 31) // Vp + 3
    N = 3
    B = -(-rows // N)
    x = torch.zeros(B * N, Vp, dtype=torch.float16, device="cuda")
    hist = torch.full((B, 1), 11, dtype=torch.int32, device="cuda")
    pres = torch.arange(B, device="cuda").float() % 50
    ab.logits_adjust(x, x, ab.GPT2_PROBS_F16, ab.logit_rules(history=hist, history_stride=1, presence=pres), None, None, B,
                     N, V, Vp)
    assert torch.equal(x[:, 11].float(), -pres.repeat_interleave(N))
    x[:, 11] = 0
    assert not x.any()
    no_device_error()


def test_graph_and_stream():
    cs = [make(torch.float32, 4, 6, 5000, seed=s) for s in (1, 2)]
    for c in cs:
        c["Vp"] = 5040
        c["x"] = c["x"][:, :5000].contiguous()
        c["x"] = torch.cat([c["x"], torch.zeros(24, 40)], 1)
    want = [run(c) for c in cs]
    t = {k: gpu(v) for k, v in cs[0]["rules"].items()}
    rules = ab.logit_rules(**t, history_stride=50, num_bias=9, num_masks=3)
    x, tok, parent = cs[0]["x"].cuda(), gpu(cs[0]["tok"]), gpu(cs[0]["parent"])
    out = torch.full((24, 5040), 7.0, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        ab.logits_adjust(out, x, 0, rules, tok, parent, 4, 6, 5000, 5040, stream=s)
    for round in range(4):
        c = cs[round % 2]
        with torch.cuda.stream(s):
            out.fill_(7.0)
            x.copy_(c["x"])
            tok.copy_(torch.from_numpy(c["tok"]))
            parent.copy_(torch.from_numpy(c["parent"]))
            for k, v in c["rules"].items():
                t[k].copy_(torch.from_numpy(v.view(np.int32) if v.dtype == np.uint32 else v))
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[round % 2])
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_two_calls_at_once(dtype):
    """On two streams, over the same logits and rules, into outputs of their own."""
    c = make(dtype, 9, 7, 20000, 700, 30, 5, seed=9, pad=16)
    want = run(c)
    x, rules, tok, parent = c["x"].cuda(), rules_of(c), gpu(c["tok"]), gpu(c["parent"])
    outs = [torch.full_like(x, 7.0) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for out, s in zip(outs, streams):
            ab.logits_adjust(out, x, ab.element_type(x), rules, tok, parent, 9, 7, 20000, c["Vp"], s)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out.cpu(), want)
    no_device_error()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("B,H", [(300, 600), (2, 5000)])
def test_single_rows_with_long_histories(dtype, B, H):
    """One token a sequence and as long lists as make segments of the largest size."""
    check(make(dtype, B, 1, 40000, H, 40, 2, seed=H, pad=3))
    no_device_error()
