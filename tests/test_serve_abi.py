"""The calls of include/gpt2fwd_serve.h on the host: every one is exported and
bound, sizes answer without a GPU, and invalid arguments are refused before
anything is launched (the addresses here are aligned and never read)."""
import ctypes
import types

import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import build, inputs, runner
from gpt_transformer_forward_gb300.runner import GPT2Model

FAKE = 1 << 20
A, S, AL, W, U = -1, -2, -3, -4, -7  # GPT2_ERR_ARG, _SHAPE, _ALIGN, _WORKSPACE, _UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ab.load(build_if_missing=False)


def refused(code, call, *args, **kw):
    with pytest.raises(ab.GPT2Error) as e:
        call(*args, **kw, stream=0)
    assert e.value.code == code, (e.value.code, code)


def test_every_declared_function_is_bound(lib):
    names = ab.header_functions("gpt2fwd_serve.h")
    assert sorted(names) == sorted(ab._SERVE_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    assert not set(names) & set(ab.header_functions())


TABLES = dict(block_table=FAKE, slots=FAKE, next_len=FAKE + 64, taken_out=FAKE + 128, cached_len=FAKE + 192,
              new_len=FAKE + 256, free_blocks=FAKE, num_free=4, taken_in=FAKE + 320, prefix_blocks=None, prefix_len=0,
              B=2, T=3, num_blocks=10, block_size=16, max_blocks_per_seq=8)


@pytest.mark.parametrize("change,code", [
    (dict(block_table=None), A), (dict(cached_len=None), A), (dict(B=-1), A), (dict(T=-1), A), (dict(num_free=-1), A),
    (dict(free_blocks=None), A), (dict(num_blocks=0), A), (dict(block_size=0), A), (dict(block_size=24), A),
    (dict(max_blocks_per_seq=0), A), (dict(prefix_len=16), A), (dict(prefix_blocks=FAKE), A),
    (dict(prefix_len=-16, prefix_blocks=FAKE), A), (dict(taken_out=FAKE + 320), A), (dict(next_len=FAKE + 192), A),
    (dict(next_len=FAKE + 256), A),
    (dict(prefix_len=8, prefix_blocks=FAKE), S), (dict(prefix_len=160, prefix_blocks=FAKE), S),
    (dict(B=65537), S), (dict(max_blocks_per_seq=1025), S), (dict(num_blocks=1 << 27), S),
    (dict(slots=FAKE + 2), AL), (dict(taken_out=FAKE + 1), AL), (dict(cached_len=FAKE + 3), AL),
])
def test_tables_refuse(change, code):
    refused(code, ab.paged_build_tables, **{**TABLES, **change})


@pytest.mark.parametrize("change", [dict(T=(1 << 30) + 1), dict(T=2**31 - 1), dict(T=2**31 - 1, B=1, slots=None)])
def test_tables_refuse_more_new_positions_than_their_loops_count(change):
    refused(S, ab.paged_build_tables, **{**TABLES, **change})


def shared_args(**kw):
    d = dict(out=FAKE, qkv=2 * FAKE, kv=ab.paged_kv(FAKE, FAKE, 64, 16, 32), pos=FAKE, B=4, C=256, NH=4, prefix_len=300,
             precision=ab.GPT2_FP16, workspace=FAKE, ws_bytes=1 << 30)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(out=None), A), (dict(qkv=None), A), (dict(kv=None), A), (dict(pos=None), A), (dict(B=-1), A),
    (dict(C=0), A), (dict(NH=0), A), (dict(prefix_len=-1), A), (dict(precision=4), A), (dict(qkv=FAKE), A),
    (dict(kv=ab.paged_kv(None, FAKE, 64, 16, 32)), A), (dict(kv=ab.paged_kv(FAKE, None, 64, 16, 32)), A),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 0, 16, 32)), A), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 12, 32)), A),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 0)), A),
    (dict(NH=3), S), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 1025)), S), (dict(prefix_len=512), S),
    (dict(B=65536), S), (dict(C=512), U), (dict(C=96), U),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 1024, 1 << 21, 1024), prefix_len=1 << 30, ws_bytes=16), S),
    (dict(workspace=None), W), (dict(ws_bytes=16), W),
    (dict(out=FAKE + 8), AL), (dict(qkv=FAKE + 8), AL), (dict(workspace=FAKE + 8), AL), (dict(pos=FAKE + 2), AL),
    (dict(kv=ab.paged_kv(FAKE + 8, FAKE, 64, 16, 32)), AL),
])
def test_shared_prefix_refuses(change, code):
    refused(code, ab.attention_shared_prefix, **shared_args(**change))


def test_shared_prefix_sizes():
    size = ab.attention_shared_prefix_workspace_size
    assert size(4, 256, 4, 0, ab.GPT2_FP16) == 0
    for bad in [(0, 256, 4, 10, 3), (4, 256, 3, 10, 3), (4, 512, 4, 10, 3), (4, 256, 4, -1, 3), (4, 256, 4, 10, 9),
                (65536, 256, 4, 10, 3)]:
        assert size(*bad) == 0, bad
    # a workspace for a batch serves smaller ones and shorter prefixes
    for precision in (ab.GPT2_FP32, ab.GPT2_FP16):
        for P in (1, 64, 65, 1000, 3328, 3329, 20000):
            for B in (1, 16, 17, 32, 33, 64, 65, 128, 129, 300):
                most = size(B, 768, 12, P, precision)
                assert most > 0 or P <= 256  # a short prefix may need none
                for b in (1, B // 2 + 1, B - 1):
                    assert b < 1 or size(b, 768, 12, P, precision) <= most, (precision, P, B, b)
                for q in (1, P // 2 + 1, P - 1):
                    assert q < 1 or size(B, 768, 12, q, precision) <= most, (precision, P, B, q)
    cfg = inputs.TINY
    base = ab.gpt2_workspace_size(cfg, 3, 1, ab.GPT2_FP16)
    assert ab.gpt2_shared_workspace_size(cfg, 3, 0, ab.GPT2_FP16) == base
    assert ab.gpt2_shared_workspace_size(cfg, 3, 600, ab.GPT2_FP16) == base + size(3, 64, 4, 600, ab.GPT2_FP16)
    assert size(3, 64, 4, 600, ab.GPT2_FP16) > 0
    assert ab.gpt2_shared_workspace_size(cfg, 3, -1, ab.GPT2_FP16) == 0


@pytest.mark.parametrize("NH", [1, 4, 12, 16])
def test_shared_prefix_sizes_where_the_kernel_changes(NH):
    # 16-bit caches with heads of 64: the kernel, and with it the splits, goes
    # by the batch and by batch x heads x prefix
    size = ab.attention_shared_prefix_workspace_size
    lengths = sorted({int(257 * 1.17 ** i) for i in range(34)} | {-(-n // (r * NH)) + d for n in (3000000, 5000000)
                                                                 for r in (128, 192, 256, 320) for d in (-1, 0, 1)})
    batches = (1, 33, 64, 65, 100, 128, 129, 192, 200, 256, 257, 300)
    got = {(B, P): size(B, 64 * NH, NH, P, ab.GPT2_BF16) for B in batches for P in lengths}
    for B in batches:
        for k, P in enumerate(lengths):
            assert got[B, P] > 0
            assert k == 0 or got[B, lengths[k - 1]] <= got[B, P], (B, lengths[k - 1], P)
    for P in lengths:
        for k in range(1, len(batches)):
            assert got[batches[k - 1], P] <= got[batches[k], P], (batches[k - 1], batches[k], P)


def step_args(**kw):
    d = dict(cfg=inputs.TINY, params=FAKE, packed=FAKE, kv=ab.paged_kv(FAKE, FAKE, 64, 16, 4), tok=FAKE, pos=FAKE, B=4,
             prefix_len=32, logits=FAKE, probs=None, workspace=FAKE, ws_bytes=1 << 30, precision=ab.GPT2_FP16)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(params=None), A), (dict(tok=None), A), (dict(pos=None), A), (dict(logits=None), A), (dict(workspace=None), A),
    (dict(kv=None), A), (dict(packed=None), A), (dict(B=0), A), (dict(prefix_len=-1), A), (dict(precision=7), A),
    (dict(prefix_len=64), S), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 2)), S), (dict(B=65536), S),
    (dict(ws_bytes=100), W), (dict(logits=FAKE + 4), AL), (dict(workspace=FAKE + 16), AL),
])
def test_shared_step_refuses(change, code):
    refused(code, ab.gpt2_decode_step_shared, **step_args(**change))


def slots_args(**kw):
    d = dict(cfg=inputs.TINY, params=FAKE, packed=FAKE, tok=FAKE, B=4, T=8, logits=FAKE, probs=None,
             kv=ab.paged_kv(FAKE, None, 64, 16, 0), slots=FAKE, workspace=FAKE, ws_bytes=1 << 30,
             precision=ab.GPT2_FP16)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(slots=None), A), (dict(kv=None), A), (dict(tok=None), A), (dict(T=0), A), (dict(packed=None), A),
    (dict(kv=ab.paged_kv(None, None, 64, 16, 0)), A), (dict(kv=ab.paged_kv(FAKE, None, 64, 20, 0)), A),
    (dict(kv=ab.paged_kv(FAKE, None, 0, 16, 0)), A), (dict(kv=ab.paged_kv(FAKE, None, 1 << 27, 16, 0)), S),
    (dict(T=65), S), (dict(ws_bytes=64), W), (dict(slots=FAKE + 1), AL),
    (dict(kv=ab.paged_kv(FAKE + 8, None, 64, 16, 0)), AL),
])
def test_prefill_slots_refuses(change, code):
    refused(code, ab.gpt2_prefill_slots, **slots_args(**change))


def lp_args(**kw):
    d = dict(logprob=FAKE, entropy=FAKE, lse=FAKE, top_ids=FAKE, top_logprobs=FAKE, logits=FAKE,
             logits_type=ab.GPT2_PROBS_F32, targets=FAKE, N=2, V=10, Vp=12, K=3)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), A), (dict(targets=None), A), (dict(N=-1), A), (dict(V=0), A), (dict(V=13), A), (dict(K=-1), A),
    (dict(logits_type=3), A), (dict(logits_type=-1), A), (dict(Vp=14), S), (dict(K=33), S),
    (dict(logits_type=ab.GPT2_PROBS_F16), S), (dict(logits_type=ab.GPT2_PROBS_BF16), S),
    (dict(logits=FAKE + 8), AL), (dict(lse=FAKE + 2), AL), (dict(targets=FAKE + 1), AL),
    (dict(V=(1 << 30) + 1, Vp=(1 << 30) + 8, logits=FAKE + 8), S),
])
def test_logprobs_refuse(change, code):
    refused(code, ab.logprobs_forward, **lp_args(**change))


def test_nothing_to_do_is_no_launch(lib):
    # no rows, or no output asked for: an answer without a GPU
    ab.logprobs_forward(**lp_args(N=0), stream=0)
    ab.logprobs_forward(**lp_args(logprob=None, entropy=None, lse=None, K=0), stream=0)
    ab.attention_shared_prefix(**shared_args(B=0), stream=0)
    ab.paged_build_tables(**{**TABLES, "B": 0, "taken_out": None}, stream=0)


def lb_args(**kw):
    d = dict(dlogits=FAKE, logits=FAKE, logits_type=ab.GPT2_PROBS_F32, targets=FAKE, lse=FAKE, entropy=FAKE,
             dlogprob=FAKE, dentropy=FAKE, N=2, V=10, Vp=12)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(dlogits=None), A), (dict(logits=None), A), (dict(lse=None), A), (dict(targets=None), A),
    (dict(entropy=None), A), (dict(V=0), A), (dict(Vp=9), A), (dict(logits_type=5), A), (dict(Vp=14), S),
    (dict(logits_type=ab.GPT2_PROBS_F16), S), (dict(dlogits=FAKE + 4), AL), (dict(dentropy=FAKE + 2), AL),
    (dict(V=(1 << 30) + 1, Vp=(1 << 30) + 8, dlogits=FAKE + 8), S),
])
def test_logprobs_backward_refuses(change, code):
    refused(code, ab.logprobs_backward, **lb_args(**change))


@pytest.fixture(scope="module")
def cpu_model():
    """A model whose buffers are in host memory, for checks that come before
    any launch."""
    w = inputs.WORKLOADS["tiny"]
    params, _ = inputs.workload_inputs(w, "perturbed")
    return GPT2Model(w.cfg, params, 2, 4, ab.GPT2_FP32, device="cpu")


@pytest.mark.parametrize("logits,targets", [
    (lambda x: x[:, :-1], None),                                     # rows of part of the positions
    (lambda x: x.transpose(0, 1), None),
    (lambda x: x, lambda t: t.long()),
    (lambda x: x, lambda t: t[:, :-1]),                              # fewer targets than rows
    (lambda x: x, lambda t: torch.cat([t, t], 1)[:, ::2]),           # strided
    (lambda x: x, lambda t: t.flatten()),
    (lambda x: x.double(), None),
])
def test_runner_logprobs_refuses_what_it_would_misread(cpu_model, logits, targets):
    x = torch.zeros(2, 4, cpu_model.cfg.padded_vocab_size)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError)):
        cpu_model.logprobs(logits(x), targets and targets(t), top=2, stream=0)


def test_runner_serving_calls_refuse_what_they_would_misread(cpu_model):
    tok = torch.zeros(2, 4, dtype=torch.int32)
    for slots in (torch.zeros(2, 8, dtype=torch.int32)[:, :4], torch.zeros(2, 4, dtype=torch.int64),
                  torch.zeros(2, 3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="slots"):
            cpu_model.prefill_slots(tok, None, None, slots, stream=0)
    for pos in (torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.int32)[::2],
                torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="pos"):
            cpu_model.decode_step_shared(None, tok[:, 0], pos, 1, None, None, stream=0)


def test_runner_logprobs_takes_a_single_row(cpu_model, monkeypatch):
    """Logits [Vp] are one row, whose results have no leading shape."""
    calls = []
    monkeypatch.setattr(ab, "logprobs_forward", lambda *a: calls.append(a))
    r = cpu_model.logprobs(torch.zeros(cpu_model.cfg.padded_vocab_size), torch.tensor(3, dtype=torch.int32), top=2)
    assert {k: tuple(v.shape) for k, v in r.items()} == dict(entropy=(), lse=(), logprob=(), top_ids=(2,),
                                                             top_logprobs=(2,))
    assert calls[0][8:12] == (1, cpu_model.cfg.vocab_size, cpu_model.cfg.padded_vocab_size, 2)
    r = cpu_model.logprobs(torch.zeros(cpu_model.cfg.padded_vocab_size))
    assert {k: tuple(v.shape) for k, v in r.items()} == dict(entropy=(), lse=())
    assert [c[7] is None for c in calls] == [False, True]


@pytest.mark.parametrize("tok", [
    lambda t: t.long(),                              # the default type of token ids: every second one would be 0
    lambda t: torch.cat([t, t], -1)[..., ::2],       # strided, as a column of a longer sequence
    lambda t: t.to(torch.int16),
])
def test_runner_serving_calls_refuse_tokens_they_would_misread(cpu_model, tok):
    t = torch.ones(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="tok"):
        cpu_model.prefill_slots(tok(t), None, None, torch.zeros(2, 4, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="tok"):
        cpu_model.decode_step_shared(None, tok(t[:, 0].contiguous()), torch.ones(2, dtype=torch.int32), 1, None,
                                     torch.zeros(1, dtype=torch.uint8), stream=0)


@pytest.mark.parametrize("which", ["logits", "probs"])
@pytest.mark.parametrize("change", [
    lambda t: t.half(),                              # half the bytes that are written
    lambda t: t.double(),
    lambda t: t[:1].contiguous(),                    # fewer rows
    lambda t: t[..., :-4].contiguous(),              # rows without the padding
    lambda t: torch.cat([t, t], -1)[..., ::2],
])
def test_runner_serving_calls_refuse_outputs_they_would_overrun(cpu_model, monkeypatch, which, change):
    reached = []
    for name in ("gpt2_prefill_slots", "gpt2_decode_step_shared"):
        monkeypatch.setattr(ab, name, lambda *a, name=name: reached.append(name))
    tok = torch.ones(2, 4, dtype=torch.int32)
    Vp = cpu_model.cfg.padded_vocab_size
    ws = torch.zeros(1, dtype=torch.uint8)
    for call, shape in ((lambda lg, pr: cpu_model.prefill_slots(tok, lg, None, tok, pr), (2, 4, Vp)),
                        (lambda lg, pr: cpu_model.decode_step_shared(None, tok[:, 0].contiguous(), tok[:, 0].contiguous(),
                                                                     1, lg, ws, pr), (2, Vp))):
        good = [torch.zeros(shape), torch.zeros(shape)]
        call(*good)
        call(good[0], None)
        bad = [change(t) if which == n else t for n, t in zip(("logits", "probs"), good)]
        with pytest.raises(ValueError, match=which):
            call(*bad)
    with pytest.raises(ValueError, match="logits"):
        cpu_model.prefill_slots(tok, None, None, tok)
    with pytest.raises(ValueError, match="workspace"):
        cpu_model.decode_step_shared(None, tok[:, 0].contiguous(), tok[:, 0].contiguous(), 1, torch.zeros(2, Vp),
                                     torch.zeros(64))
    assert reached == ["gpt2_prefill_slots"] * 2 + ["gpt2_decode_step_shared"] * 2


def test_runner_serving_calls_refuse_tensors_of_another_device(cpu_model, monkeypatch):
    for name in ("gpt2_prefill_slots", "gpt2_decode_step_shared", "logprobs_forward"):
        monkeypatch.setattr(ab, name, lambda *a: None)
    Vp = cpu_model.cfg.padded_vocab_size
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    prefill = dict(tok=i(2, 4), logits=torch.zeros(2, 4, Vp), kv=None, slots=i(2, 4), probs=torch.zeros(2, 4, Vp))
    step = dict(kv=None, tok=i(2), pos=i(2), prefix_len=1, logits=torch.zeros(2, Vp),
                workspace=torch.zeros(1, dtype=torch.uint8), probs=torch.zeros(2, Vp))
    rows = dict(logits=torch.zeros(3, Vp), targets=i(3))
    for call, args in ((cpu_model.prefill_slots, prefill), (cpu_model.decode_step_shared, step),
                       (cpu_model.logprobs, rows)):
        call(**args)
        for name, t in args.items():
            if torch.is_tensor(t):
                with pytest.raises(ValueError, match=name):
                    call(**{**args, name: t.to("meta")})
    # the model's device is the current one
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    second = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="current"):
        runner._check_device(torch.device("cuda", 1), logits=second)
    runner._check_device(torch.device("cuda", 0), logits=types.SimpleNamespace(device=torch.device("cuda", 0)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_runner_calls_that_write_fp32_probs_refuse_others(cpu_model, monkeypatch, dtype):
    reached = []
    for name in ("gpt2_decode_step", "gpt2_prefill_paged", "gpt2_decode_step_paged"):
        monkeypatch.setattr(ab, name, lambda *a, name=name: reached.append(name))
    tok = torch.ones(2, 4, dtype=torch.int32)
    lg, pr = cpu_model.new_outputs(2, 4, probs_dtype=dtype)
    lg1, pr1 = cpu_model.new_outputs(2, None, probs_dtype=dtype)
    for call in (lambda p4, p1: cpu_model.decode_step(None, tok[:, 0], 3, lg1, p1),
                 lambda p4, p1: cpu_model.prefill_paged(tok, lg, None, p4),
                 lambda p4, p1: cpu_model.decode_step_paged(None, tok[:, 0], tok[:, 0], lg1, p1)):
        with pytest.raises(ValueError, match="probs"):
            call(pr, pr1)
        call(pr.float(), pr1.float())
        call(None, None)
    assert len(reached) == 6


def test_element_types():
    assert ab.element_type(torch.empty(1)) == ab.GPT2_PROBS_F32
    assert ab.element_type(torch.empty(1, dtype=torch.bfloat16)) == ab.GPT2_PROBS_BF16
    with pytest.raises(TypeError):
        ab.element_type(torch.empty(1, dtype=torch.float64))
    assert ctypes.sizeof(ab.GPT2PagedKVCache) == 32
