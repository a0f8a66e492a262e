"""Log probabilities of given tokens with entropy and top alternatives, and
their gradient [llm.c classifier], against 64-bit forms of the formulas.

Tolerances (u = 2^-24, one fp32 rounding).  With d = l - max l, a term exp(d)
is computed as 2^(d log2 e): the exponent's two roundings and ex2's error give
a relative error of at most (2 |d| + 4) u where it counts, |d| <= R (R = 104,
exp(-104) < 2^-149: smaller terms are zero), and a sum over V terms adds at most V u
in the worst order and, over T partial sums of V/T terms each, (V/T + log2 T) u;
T >= 256 here.  E = (2 R + V/256 + 16) u bounds the relative error of
sum exp(d), so the absolute error of log sum; lse adds its own rounding,
|lse| u, and a log probability (l - max l) - log sum those of its two steps.  The entropy log s - sum(e d) / s
has the error E (1 + R_w), R_w = sum(e |d|) / s its weighted mean.  The
gradient's p = exp(l - lse) has the relative error (3 |log p| + 8) u plus that
of the lse it is given, 2 |lse| u, which rows of large |lse| do not rely on: from
|lse| = 1024 on they add E instead."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import inputs
from gpt_transformer_forward_gb300.runner import GPT2Model

from gpu_helpers import need_gpu, no_device_error
from serve_reference import logprobs, logprobs_grad

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def make(N, V, Vp, dtype, seed, scale=3.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, Vp, generator=g) * scale
    if masked:
        x[torch.rand(N, Vp, generator=g) < masked] = -float("inf")
    t = torch.randint(-1, V, (N,), generator=g, dtype=torch.int32)
    return x.to(TYPES[dtype]), t


def forward(x, t, V, K, want=("logprob", "entropy", "lse", "top_ids", "top_logprobs")):
    N, Vp = x.shape
    xg, tg = x.cuda(), t.cuda() if t is not None else None
    out = {k: torch.full((N, K) if k.startswith("top") else (N,), 7,
                         dtype=torch.int32 if k == "top_ids" else torch.float32, device="cuda") for k in want}
    ab.logprobs_forward(*[out.get(k) for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")], xg,
                        ab.element_type(xg), tg, N, V, Vp, K)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def bound(x64, lse):
    """E and R_w of each row."""
    V = x64.shape[1]
    E = (2 * 104 + V / 256 + 16) * u
    with np.errstate(invalid="ignore", under="ignore", over="ignore"):
        m = np.where(np.isfinite(x64.max(1)), x64.max(1), 0.0)[:, None]
        d = np.maximum(x64 - m, -200.0)
        e = np.exp(d)
        rw = (e * -d).sum(1) / np.maximum(e.sum(1), 1e-30)
    return E, np.nan_to_num(rw)


def near(got, ref, tol, what):
    got, ref = got.astype(np.float64), ref.astype(np.float64)
    ref = np.where(np.abs(ref) > float(np.finfo(np.float32).max), np.copysign(np.inf, ref), ref)  # past fp32
    same = (np.isnan(got) & np.isnan(ref)) | (got == ref)
    with np.errstate(invalid="ignore"):
        ok = same | (np.isfinite(ref) & (np.abs(got - ref) <= tol))
    i = np.argmin(ok)
    assert ok.all(), f"{what}: {(~ok).sum()} off, first at {i}: {got.flat[i]} for {ref.flat[i]}"


def check(x, t, V, K):
    got = forward(x, t, V, K) if K else forward(x, t, V, K, want=("logprob", "entropy", "lse"))
    x64 = x[:, :V].double().numpy()
    ref = logprobs(x64, t.numpy(), K)
    E, rw = bound(x64, ref["lse"])
    with np.errstate(invalid="ignore"):
        lse_tol = E + 2 * u * np.abs(ref["lse"])
        near(got["lse"], ref["lse"], lse_tol, "lse")
        near(got["logprob"], ref["logprob"], E + 3 * u * np.abs(ref["logprob"]) + 16 * u, "logprob")
        near(got["entropy"], ref["entropy"], 2 * E * (1 + rw), "entropy")
        if K:
            np.testing.assert_array_equal(got["top_ids"], ref["top_ids"])
            near(got["top_logprobs"], ref["top_logprobs"],
                 E + 3 * u * np.abs(ref["top_logprobs"]) + 16 * u, "top")
    no_device_error()
    return got


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N,V,Vp,K", [
    (1, 1, 8, 1), (1, 3, 8, 5), (2, 7, 8, 32), (3, 31, 32, 32), (1, 33, 40, 32), (5, 255, 256, 3), (4, 1000, 1024, 20),
    (1, 4097, 4104, 32), (9, 32003, 32008, 7), (1, 50257, 50304, 20), (33, 50257, 50304, 5), (200, 5003, 5008, 0),
    (700, 1531, 1536, 1), (3, 128256, 128256, 32),
])
def test_against_64_bits(dtype, N, V, Vp, K):
    check(*make(N, V, Vp, dtype, seed=N + V), V, K)


@pytest.mark.parametrize("dtype,N,V,Vp,K", [
    ("fp32", 1000, 20003, 20008, 20), ("fp32", 1500, 40001, 40008, 3), ("fp32", 1900, 33001, 33008, 32),
    ("bf16", 1300, 50257, 50304, 20), ("fp16", 2500, 9001, 9008, 8), ("fp32", 3000, 3001, 3008, 5),
    ("bf16", 900, 70001, 70008, 1), ("fp32", 1000, 20003, 20008, 0)])
def test_blocks_that_walk_many_rows(dtype, N, V, Vp, K):
    """More rows than the GPU holds blocks, so that a block takes several rows:
    every row against 64 bits, and the same values from every repeat."""
    x, t = make(N, V, Vp, dtype, seed=N)
    xg, tg = x.cuda(), t.cuda()
    outs = []
    for _ in range(6):
        f = [torch.empty(N, device="cuda") for _ in range(3)]
        ids, top = torch.empty(N, max(K, 1), dtype=torch.int32, device="cuda"), torch.empty(N, max(K, 1), device="cuda")
        ab.logprobs_forward(*f, ids if K else None, top if K else None, xg, ab.element_type(xg), tg, N, V, Vp, K)
        outs.append([o.cpu() for o in f + ([ids, top] if K else [])])
    for again in outs[1:]:
        for a, b in zip(outs[0], again):
            assert torch.equal(a, b)
    z = xg[:, :V].double()
    logp = torch.log_softmax(z, 1)
    lse = torch.logsumexp(z, 1).cpu().numpy()
    d = (z - z.amax(1, keepdim=True)).clamp(min=-200.0)
    rw = ((d.exp() * -d).sum(1) / d.exp().sum(1)).cpu().numpy()
    E = (2 * 104 + V / 256 + 16) * u
    near(outs[0][2].numpy(), lse, E + 2 * u * np.abs(lse), "lse")
    near(outs[0][1].numpy(), torch.special.entr(logp.exp()).sum(1).cpu().numpy(), 2 * E * (1 + rw), "entropy")
    lp = logp.gather(1, tg.clamp(min=0).long()[:, None])[:, 0].masked_fill(tg < 0, 0.0).cpu().numpy()
    near(outs[0][0].numpy(), lp, E + 3 * u * np.abs(lp) + 16 * u, "logprob")
    if K:
        # (z distinguishes equal values by id: the lowest first)
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :K]
        assert torch.equal(outs[0][3].cuda().long(), order)
        tp = logp.gather(1, order).cpu().numpy()
        near(outs[0][4].numpy(), tp, E + 3 * u * np.abs(tp) + 16 * u, "top")
    no_device_error()


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("masked", [0.5, 0.99, 0.9999])
@pytest.mark.parametrize("N", [1, 40, 1000])
def test_ruled_out_tokens(dtype, masked, N):
    V = 5003 if N < 1000 else 601
    check(*make(N, V, V + 5 if V % 8 == 3 else V + 7, dtype, seed=N, masked=masked), V, 32)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N", [2, 700])
def test_special_rows(dtype, N):
    """Rows with every token ruled out, of the type's lowest value, constant,
    with one token, with NaN or infinity (first, last, alone), with a
    dominant token, of huge values, and with -0 beside 0."""
    V, Vp = 777, 784
    x, t = make(max(N, 16), V, Vp, dtype, seed=1)
    low = float(torch.finfo(TYPES[dtype]).min)
    inf = float("inf")
    x[0] = -inf
    x[1] = low
    x[2] = 1.25
    x[3] = -inf
    x[3, 500] = 2.0
    x[4, 0] = float("nan")
    x[5, V - 1] = float("nan")
    x[6, 300] = inf
    x[7] = -inf
    x[7, 3] = float("nan")
    x[8] = low
    x[8, 700] = -low
    x[9, 100] = 60000.0
    x[10] = 0.0
    x[10, ::2] = -0.0
    x[11, :400] = low
    x[12] = -inf
    x[12, V:] = 5.0  # only the padding holds values
    x[13, V:] = float("nan")
    x[14] = -inf
    x[14, V - 3:] = 1.0
    t[:12] = torch.tensor([5, 7, 9, 500, 3, -1, 300, 3, 700, 100, 1, 0], dtype=torch.int32)
    check(x, t, V, 32)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("N", [1, 30, 700])
@pytest.mark.parametrize("kind", ["constant", "two values", "ascending", "descending", "stride", "runs"])
def test_ties_and_orders(dtype, N, kind):
    """Many equal logits (the lowest ids are listed) and orders in which one
    thread's or one block's share holds all the largest values."""
    V, Vp, K = 9001, 9008, 32
    i = torch.arange(Vp)
    rows = {"constant": torch.zeros(Vp), "two values": (i * 7919 % 3 == 0).float(),
            "ascending": (i // 16).float() / 8, "descending": -(i // 16).float() / 8,
            "stride": (i % 1024 < 8).float() * 4 + (i // 1024).float() / 4,
            "runs": (i // 1125 == 3).float() * 3 + (i % 125).float() / 128}
    x = rows[kind].expand(N, Vp).clone()
    if N > 1:
        x = x + (torch.arange(N) % 5).float()[:, None] / 4
    check(x.to(TYPES[dtype]), torch.zeros(N, dtype=torch.int32), V, K)


def test_outputs_are_optional():
    x, t = make(6, 1001, 1008, "fp32", seed=4)
    full = forward(x, t, 1001, 8)
    for want in (("lse",), ("entropy",), ("top_ids",), ("top_logprobs",), ("logprob",)):
        got = forward(x, t if "logprob" in want else None, 1001, 8, want)
        for k in want:
            np.testing.assert_array_equal(got[k], full[k])


def test_bad_targets_are_flagged():
    x, _ = make(4, 50, 56, "fp32", seed=4)
    t = torch.tensor([3, -2, 50, -1], dtype=torch.int32)
    got = forward(x, t, 50, 1)
    assert ab.gpt2_get_error() == ab.DEVERR_TOKEN
    assert (got["logprob"][1:] == 0).all() and got["logprob"][0] < 0
    xg = x.cuda()
    lse = torch.from_numpy(got["lse"]).cuda()
    d = torch.empty_like(xg)
    one = torch.ones(4, device="cuda")
    ab.logprobs_backward(d, xg, 0, t.cuda(), lse, None, one, None, 4, 50, 56)
    assert ab.gpt2_get_error() == ab.DEVERR_TOKEN
    assert (d[1:] == 0).all() and (d[0] != 0).any()


def backward(x, t, lse, ent, g, h, V, inplace=False):
    N, Vp = x.shape
    xg = x.cuda()
    d = xg if inplace else torch.full_like(xg, 3.0)
    c = lambda a: a.cuda() if a is not None else None  # noqa: E731
    ab.logprobs_backward(d, xg, ab.element_type(xg), c(t), c(lse), c(ent), c(g), c(h), N, V, Vp)
    torch.cuda.synchronize()
    return d.cpu()


def grad_tol(x64, ref, want, g, h, dtype):
    """p's relative error on each term, one rounding for each of the formula's
    steps, and the output's own."""
    lse, V = np.nan_to_num(ref["lse"], neginf=0.0)[:, None], x64.shape[1]
    with np.errstate(all="ignore"):
        m = np.nan_to_num(x64.max(1), neginf=0.0)[:, None]
        lp = np.where(np.isfinite(x64), (x64 - m) - (lse - m), -200.0)
        lp = np.where(np.abs(lse) < 1e30, lp, (x64 - m) - np.log(np.exp(x64 - m).sum(1, keepdims=True)))
        p = np.exp(lp)
        lp = np.maximum(lp, -200.0)
    of_lse = np.where(np.abs(lse) < 1024, 2 * np.abs(lse), 2 * 104 + V / 256 + 16)
    rel = (3 * np.abs(lp) + of_lse + 8) * u
    gg = np.abs(g.numpy())[:, None] if g is not None else 0.0
    hh = np.abs(h.numpy())[:, None] if h is not None else 0.0
    size = p * (gg + hh * (np.abs(lp) + np.abs(ref["entropy"])[:, None]))
    # (log p itself, off by its lse, times p: in size * rel only where |log p| >= 1)
    size = size + p * hh
    return size * (rel + 4 * u) + 2 * u * gg * (np.abs(want) > 0) + HALF[dtype] * np.abs(want) * 1.01 + TINY[dtype]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("which", ["both", "logprob", "entropy"])
@pytest.mark.parametrize("N,V,Vp,masked", [(1, 1, 8, 0), (2, 7, 8, 0.3), (5, 255, 256, 0), (3, 4097, 4104, 0.5),
                                           (33, 50257, 50304, 0), (700, 1531, 1536, 0.9)])
def test_gradient_against_64_bits(dtype, which, N, V, Vp, masked):
    x, t = make(N, V, Vp, dtype, seed=N + V, masked=masked)
    if N > 2:
        x[1] = -float("inf")
    rng = torch.Generator().manual_seed(3)
    g = torch.randn(N, generator=rng) if which != "entropy" else None
    h = torch.randn(N, generator=rng) if which != "logprob" else None
    x64 = x[:, :V].double().numpy()
    ref = logprobs(x64, t.numpy(), 0)
    lse, ent = torch.from_numpy(ref["lse"]).float(), torch.from_numpy(ref["entropy"]).float()
    got = backward(x, t if which != "entropy" else None, lse, ent if h is not None else None, g, h, V)
    assert (got[:, V:] == 0).all()
    want = logprobs_grad(x64, t.numpy(), ent.double().numpy(),
                         None if g is None else g.double().numpy(), None if h is None else h.double().numpy())
    tol = grad_tol(x64, ref, want, g, h, x.dtype)
    err = np.abs(got[:, :V].double().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()
    # in place: the same values over the logits
    again = backward(x, t if which != "entropy" else None, lse, ent if h is not None else None, g, h, V, inplace=True)
    assert torch.equal(again, got)
    no_device_error()


def test_gradient_against_differences():
    """The loss sum(g logprob + h entropy) through the forward call, central
    differences in 64 bits of step 2^-8: error step^2 |f'''| / 6 <= 2^-16 * 20
    for |g|, |h| <= 2 and these rows."""
    N, V, Vp = 4, 37, 40
    x, t = make(N, V, Vp, "fp32", seed=8, scale=1.0)
    t[0], t[1] = 3, -1
    g, h = torch.tensor([1.0, 2.0, -0.5, 0.25]), torch.tensor([0.5, -1.0, 0.0, 2.0])
    f = forward(x, t, V, 0, want=("logprob", "entropy", "lse"))
    got = backward(x, t, torch.from_numpy(f["lse"]), torch.from_numpy(f["entropy"]), g, h, V).numpy()
    x64, step = x[:, :V].double().numpy(), 2.0 ** -8
    for v in range(V):
        side = []
        for sign in (1, -1):
            y = x64.copy()
            y[:, v] += sign * step
            r = logprobs(y, t.numpy(), 0)
            side.append(g.numpy() * r["logprob"] + h.numpy() * r["entropy"])
        diff = (side[0] - side[1]) / (2 * step)
        assert np.abs(diff - got[:, v]).max() < 20 * 2.0 ** -16


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_gradient_of_large_logits(dtype):
    """Rows whose log-sum-exp is so large that its fp32 rounding would show in
    exp(l - lse): all of the type's lowest or highest value, and spread around
    a large one."""
    V, Vp = 601, 608
    x, t = make(6, V, Vp, dtype, seed=4)
    big = 60000.0 if dtype == "fp16" else 3e38
    x[0], x[1] = -big, big
    x[2], x[3] = -big, -big
    x[2, 5], x[3, ::2] = 1.0, -float("inf")
    x[4] = 2048.0 + 2 * (torch.arange(Vp) % 4).to(x.dtype)
    t[:] = 5
    f = forward(x, t, V, 0, want=("logprob", "entropy", "lse"))
    g, h = torch.linspace(0.5, 1.5, 6), torch.linspace(-1.0, 1.0, 6)
    got = backward(x, t, torch.from_numpy(f["lse"]), torch.from_numpy(f["entropy"]), g, h, V)
    x64 = x[:, :V].double().numpy()
    ref = logprobs(x64, t.numpy(), 0)
    want = logprobs_grad(x64, t.numpy(), f["entropy"].astype(np.float64), g.numpy(), h.numpy())
    err = np.abs(got[:, :V].double().numpy() - want)
    tol = grad_tol(x64, ref, want, g, h, x.dtype)
    assert (err <= tol).all(), (err - tol).max()
    no_device_error()


def test_nan_rows_have_nan_gradients():
    x, t = make(3, 50, 56, "fp32", seed=2)
    x[1, 5] = float("nan")
    t[:] = 4
    f = forward(x, t, 50, 2)
    d = backward(x, t, torch.from_numpy(f["lse"]), torch.from_numpy(f["entropy"]), torch.ones(3), torch.ones(3), 50)
    assert torch.isnan(d[1, :50]).all() and torch.isfinite(d[[0, 2]]).all()


@pytest.mark.parametrize("N", [1, 30, 700])
def test_repeats_streams_and_graphs(N):
    """The same values again, on another stream, and from a replayed graph
    whose inputs changed in between."""
    V, Vp, K = 5003, 5008, 20
    x, t = make(N, V, Vp, "fp32", seed=5)
    y, t2 = make(N, V, Vp, "fp32", seed=6)
    first, other = forward(x, t, V, K), forward(y, t2, V, K)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for k, v in forward(x, t, V, K).items():
            np.testing.assert_array_equal(v, first[k])
    xg, tg = x.cuda(), t.cuda()
    out = [torch.empty(N, device="cuda") for _ in range(3)]
    ids, top = torch.empty(N, K, dtype=torch.int32, device="cuda"), torch.empty(N, K, device="cuda")
    d, one = torch.empty_like(xg), torch.ones(N, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ab.logprobs_forward(*out, ids, top, xg, 0, tg, N, V, Vp, K)
        ab.logprobs_backward(d, xg, 0, tg, out[2], out[1], one, one, N, V, Vp)
    for a, b, want in ((y, t2, other), (x, t, first)):
        xg.copy_(a)
        tg.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for got, k in zip(out + [ids, top], ("logprob", "entropy", "lse", "top_ids", "top_logprobs")):
            np.testing.assert_array_equal(got.cpu().numpy(), want[k])
        eager = backward(a, b, out[2].cpu(), out[1].cpu(), one.cpu(), one.cpu(), V)
        assert torch.equal(d.cpu(), eager)


def test_rows_past_32_bits():
    """Rows whose offset passes 2^31 elements (bf16, 5 GB)."""
    V = Vp = 50304
    N = 2 ** 31 // Vp + 40
    x = torch.zeros(N, Vp, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-8:] = (torch.randn(8, Vp, generator=g, device="cuda") * 3).bfloat16()
    lse, ids = torch.empty(N, device="cuda"), torch.empty(N, 2, dtype=torch.int32, device="cuda")
    ent = torch.empty(N, device="cuda")
    ab.logprobs_forward(None, ent, lse, ids, None, x, ab.element_type(x), None, N, V, Vp, 2)
    ref = logprobs(x[-8:].double().cpu().numpy(), None, 2)
    E, _ = bound(x[-8:].double().cpu().numpy(), ref["lse"])
    near(lse[-8:].cpu().numpy(), ref["lse"], E + 2 * u * np.abs(ref["lse"]), "lse")
    np.testing.assert_array_equal(ids[-8:].cpu().numpy(), ref["top_ids"])
    assert (ids[:-8] == torch.tensor([0, 1], device="cuda")).all()
    h = torch.ones(N, device="cuda")
    ab.logprobs_backward(x, x, ab.element_type(x), None, lse, ent, None, h, N, V, Vp)
    assert (x[:100].abs() < 1e-6).all() and (x[-8:].abs().amax(1) > 1e-4).all()
    no_device_error()


def test_runner_logprobs():
    w = inputs.WORKLOADS["tiny"]
    params, tok = inputs.workload_inputs(w, "perturbed")
    m = GPT2Model(w.cfg, params, w.B, w.T, ab.GPT2_FP32)
    logits, _ = m.new_outputs(w.B, w.T, probs=False)
    tg = torch.from_numpy(tok).cuda()
    m.forward(tg, logits)
    nxt = torch.full_like(tg, -1)
    nxt[:, :-1] = tg[:, 1:]
    r = m.logprobs(logits, nxt, top=3)
    ref = torch.log_softmax(logits[..., :w.cfg.vocab_size].double(), -1)
    want = ref.gather(-1, nxt.clamp(min=0).long()[..., None])[..., 0].masked_fill(nxt < 0, 0.0)
    assert (r["logprob"] - want).abs().max() < 1e-5
    assert r["top_ids"].shape == (w.B, w.T, 3) and r["entropy"].shape == (w.B, w.T)
    nxt1 = torch.empty(w.B * w.T, dtype=torch.int32, device="cuda")
    ab.gpt2_argmax(nxt1, logits, w.B * w.T, w.cfg.vocab_size, w.cfg.padded_vocab_size)
    assert torch.equal(r["top_ids"][..., 0].reshape(-1), nxt1)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_runner_logprobs_allocates_on_the_stream_it_runs_on(monkeypatch, raw):
    w = inputs.WORKLOADS["tiny"]
    params, _ = inputs.workload_inputs(w, "perturbed")
    m = GPT2Model(w.cfg, params, 1, 4, ab.GPT2_FP32)
    logits = torch.randn(5, w.cfg.padded_vocab_size, device="cuda")
    tg = torch.arange(5, dtype=torch.int32, device="cuda")
    want = m.logprobs(logits, tg, top=2)
    s, real, at = torch.cuda.Stream(), torch.empty, []
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (at.append(torch.cuda.current_stream().cuda_stream),
                                                         real(*a, **k))[1])
    torch.cuda.synchronize()
    got = m.logprobs(logits, tg, top=2, stream=s.cuda_stream if raw else s)
    assert at == [s.cuda_stream] * 5
    assert torch.cuda.current_stream().cuda_stream != s.cuda_stream
    s.synchronize()
    for k, v in want.items():
        assert torch.equal(got[k], v), k


@pytest.mark.parametrize("inplace", [True, False], ids=["in place", "apart"])
def test_gradient_of_rows_past_32_bits(inplace):
    """Both sides of the row that holds element 2^31, and the last rows, against
    64 bits, with the target's term and the padding's zeros; the uniform rows
    between them (p = 1 / V, log p + H = 0 but for roundings) for their one
    value and their target's."""
    V, Vp = 50300, 50304
    N = 2 ** 31 // Vp + 40
    at = torch.cat([2 ** 31 // Vp + torch.arange(-4, 5), torch.arange(N - 6, N)])
    g0 = torch.Generator().manual_seed(4)
    rows = (torch.randn(len(at), Vp, generator=g0) * 3).bfloat16()
    x = torch.zeros(N, Vp, dtype=torch.bfloat16, device="cuda")
    x[at.cuda()] = rows.cuda()
    t = torch.randint(0, V, (N,), generator=g0, dtype=torch.int32)
    g, h = torch.randn(N, generator=g0), torch.randn(N, generator=g0)
    x64 = rows[:, :V].double().numpy()
    ref = logprobs(x64, t[at].numpy(), 0)
    lse, ent = torch.full((N,), float(np.log(V))), torch.full((N,), float(np.log(V)))
    lse[at], ent[at] = torch.from_numpy(ref["lse"]).float(), torch.from_numpy(ref["entropy"]).float()
    d = x if inplace else torch.full_like(x, 3.0)
    ab.logprobs_backward(d, x, ab.element_type(x), t.cuda(), lse.cuda(), ent.cuda(), g.cuda(), h.cuda(), N, V, Vp)
    no_device_error()
    got = d[at.cuda()].cpu()
    want = logprobs_grad(x64, t[at].numpy(), ent[at].double().numpy(), g[at].double().numpy(), h[at].double().numpy())
    tol = grad_tol(x64, ref, want, g[at], h[at], x.dtype)
    err = np.abs(got[:, :V].double().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()
    rest = torch.ones(N, dtype=torch.bool)
    rest[at] = False
    gd, td = g.cuda(), t.cuda().long()
    # -g / V, its entropy term off by h / V (|log V| (4 + 2) + 8) u, each rounded to bf16
    size = gd.abs() / V * (2.0 ** -8 + 1e-5) + h.cuda().abs() / V * 80 * u + 2.0 ** -126
    own = d.gather(1, td[:, None])[:, 0].float()
    assert ((own - gd * (1 - 1 / V)).abs() <= size + gd.abs() * 2.0 ** -8)[rest.cuda()].all()
    d.scatter_(1, td[:, None], 0.0)
    for lo in range(0, N, 4096):
        r = torch.arange(lo, min(N, lo + 4096))
        r = r[rest[r]].cuda()
        y = d[r]
        assert (y[:, V:] == 0).all()
        hit = torch.zeros(len(r), V, dtype=torch.bool, device="cuda").scatter_(1, td[r, None], True)
        assert (((y[:, :V].float() + gd[r, None] / V).abs() <= size[r, None]) | hit).all()


def test_runner_logprobs_of_a_single_row():
    w = inputs.WORKLOADS["tiny"]
    params, _ = inputs.workload_inputs(w, "perturbed")
    m = GPT2Model(w.cfg, params, 1, 4, ab.GPT2_FP32)
    logits = torch.randn(1, w.cfg.padded_vocab_size, device="cuda")
    tg = torch.tensor([5], dtype=torch.int32, device="cuda")
    want, got = m.logprobs(logits, tg, top=3), m.logprobs(logits[0], tg[0], top=3)
    assert sorted(got) == sorted(want)
    for k in want:
        assert torch.equal(got[k], want[k][0]), k
    no_device_error()
