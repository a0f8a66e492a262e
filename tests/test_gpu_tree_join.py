"""The launch that joins the parts of an attention over trees (FlashAttention
Algorithm 1's running maximum and sum, one pair's shares one behind the other), over
workspaces that an attention whose waits gave up may leave: entries that nobody
wrote hold anything, and are followed nowhere.

Tolerance: u = 2^-24; over F parts, four at a time, a weight is an exponential, off
by 8 u, and one more for each four parts behind it; sums F u each, the quotient 4 u:
(16 ceil(F / 4) + 2 F + 20) u sum|o| w / sum l w, and half a step of the output's
type."""
import numpy as np
import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab

from gpu_helpers import need_gpu, no_device_error

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
DT = {ab.GPT2_FP32: torch.float32, ab.GPT2_BF16: torch.bfloat16, ab.GPT2_FP16: torch.float16}
HALF = {torch.float32: u, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [ab.GPT2_FP32, ab.GPT2_BF16, ab.GPT2_FP16]
NAMES = {v: k for k, v in ab.PRECISIONS.items()}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Workspace:
    """The workspace between two guards, and its parts: outputs [2 shares][N][hs],
    (maximum, sum) [2 shares][N], entries."""

    def __init__(self, N, hs, NH, precision, seed):
        most = 152 * (12 if N <= 16 else 6 if N <= 32 else 3)
        self.bytes = ab.attention_tree_workspace_size(1, N, NH * hs, NH, precision)
        g = torch.Generator().manual_seed(seed)
        self.memory = torch.randint(0, 256, (self.bytes + 2 * 4096,), dtype=torch.uint8, generator=g).cuda()
        self.ws = self.memory[4096:-4096]
        up = lambda x: (x + 255) // 256 * 256  # noqa: E731
        rows = 2 * most * N
        o, ml = rows * hs * 4, rows * 8
        self.o = self.ws[:o].view(torch.float32).view(2 * most, N, hs)
        self.ml = self.ws[up(o):up(o) + ml].view(torch.float32).view(2 * most, N, 2)
        at = up(o) + up(ml)
        self.split = self.ws[at:at + most * 16].view(torch.int32).view(most, 4)
        self.shares = most


@pytest.mark.parametrize("precision", TYPES, ids=[NAMES[p] for p in TYPES])
@pytest.mark.parametrize("hs", [16, 32, 64])
@pytest.mark.parametrize("N", [1, 8, 17, 64])
@pytest.mark.parametrize("shares", [None, 5])
def test_entries_that_nobody_wrote(precision, hs, N, shares):
    B, NH = 3, 4
    dt, pairs = DT[precision], B * NH
    w = Workspace(N, hs, NH, precision, seed=N + hs)
    F = shares or w.shares
    rng = np.random.default_rng(hs + N)
    w.o.copy_(torch.from_numpy(rng.standard_normal(w.o.shape).astype(np.float32)))
    ml = np.stack([rng.uniform(-3, 3, w.ml.shape[:2]), rng.uniform(0.5, 2, w.ml.shape[:2])], -1).astype(np.float32)
    ml[2 * 1 + 1, 0, 1] = -1  # the first node of the pair that begins in share 1 is missing
    w.ml.copy_(torch.from_numpy(ml))
    low, top = -2**31, 2**31 - 1
    entries = [[-1, 0, 0, 0], [2, 1, 4, 0], [pairs, 0, 1, 0], [top, 0, 1, 0], [low, 0, 1, 0], [3, -1, 2, 0],
               [4, low, 1, 0], [7, 0, 1, 0], [5, 0, F, 0], [6, 2, top, 0], [8, 3, 2, 0], [9, top, top, 0]]
    w.split.copy_(torch.full_like(w.split, -1))
    w.split[:len(entries)] = torch.tensor(entries, dtype=torch.int32)
    before = w.memory.clone()
    C = NH * hs
    out = torch.full((B * N + 2 * N, C), 9.0, dtype=dt, device="cuda")
    # with as many entries as shares at least five of them are read, with all all of them
    ab.gpt2_diag_tree_join(out[N:-N], B, N, C, NH, F, precision, w.ws, w.bytes)
    no_device_error()
    assert torch.equal(w.memory, before)
    got = out.double().cpu().numpy().reshape(B + 2, N, NH, hs)
    read = min(F, pairs)
    want = np.full_like(got, 9.0)
    tol = np.zeros_like(got)
    o, ml = w.o.double().cpu().numpy(), w.ml.double().cpu().numpy()
    for pair, first, last, _ in [e for e in entries[:read] if e in ([2, 1, 4, 0], [7, 0, 1, 0])]:
        slots = [2 * first + 1] + [2 * f for f in range(first + 1, last + 1)]
        n = len(slots)
        p, l = o[slots], ml[slots, :, 1]
        e = 2.0 ** (ml[slots, :, 0] - ml[slots, :, 0].max(0))
        z = (e * l).sum(0)
        x = (p * e[..., None]).sum(0) / z[:, None]
        t = (16 * -(-n // 4) + 2 * n + 20) * u * (np.abs(p) * e[..., None]).sum(0) / z[:, None]
        t = t + HALF[dt] * np.abs(x) + (2.0 ** -25 if dt == torch.float16 else 0)
        missing = (l < 0).any(0)
        x[missing], t[missing] = 0, 0
        b, h = 1 + pair // NH, pair % NH
        want[b, :, h], tol[b, :, h] = x, t
    assert (np.abs(got - want) <= tol).all()
    assert (got != 9).any()


@pytest.mark.parametrize("precision", TYPES, ids=[NAMES[p] for p in TYPES])
@pytest.mark.parametrize("byte", [0x00, 0x7f, 0x80, 0xff])
def test_a_workspace_of_one_byte(precision, byte):
    B, N, NH, hs = 50, 9, 5, 32
    w = Workspace(N, hs, NH, precision, seed=1)
    w.memory.fill_(byte)
    C = NH * hs
    out = torch.full((B * N + 2, C), 9.0, dtype=DT[precision], device="cuda")
    ab.gpt2_diag_tree_join(out[1:-1], B, N, C, NH, w.shares, precision, w.ws, w.bytes)
    no_device_error()
    assert (w.memory == byte).all()
    if byte:
        assert (out == 9).all()
    else:  # every entry names the first pair, with one part that holds nothing
        out[1:1 + N, :hs] = 9
        assert (out == 9).all()
