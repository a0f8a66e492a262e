"""The calls of include/gpt2fwd_draft.h on the host: every one is exported and
bound, sizes answer without a GPU, and invalid arguments are refused before
anything is launched (the addresses here are aligned and never read)."""
import ctypes

import pytest
import torch

from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import build, inputs
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
    names = ab.header_functions("gpt2fwd_draft.h")
    assert sorted(names) == sorted(ab._DRAFT_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    assert not set(names) & set(ab.header_functions() + ab.header_functions("gpt2fwd_serve.h"))
    assert ctypes.sizeof(ab.GPT2LogitRules) == 10 * 8 + 16


def attention_args(**kw):
    d = dict(out=FAKE, qkv=2 * FAKE, kv=ab.paged_kv(FAKE, FAKE, 64, 16, 32), pos=FAKE, parent=FAKE, B=4, N=8, C=256,
             NH=4, precision=ab.GPT2_FP16, workspace=FAKE, ws_bytes=1 << 30)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(out=None), A), (dict(qkv=None), A), (dict(kv=None), A), (dict(pos=None), A), (dict(B=-1), A), (dict(N=0), A),
    (dict(C=0), A), (dict(NH=0), A), (dict(precision=4), A), (dict(qkv=FAKE), A),
    (dict(kv=ab.paged_kv(None, FAKE, 64, 16, 32)), A), (dict(kv=ab.paged_kv(FAKE, None, 64, 16, 32)), A),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 0, 16, 32)), A), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 12, 32)), A),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 0)), A),
    (dict(NH=3), S), (dict(N=65), S), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 1025)), S), (dict(B=65536), S),
    (dict(C=512), U), (dict(C=96), U), (dict(workspace=None), W), (dict(ws_bytes=1000), W),
    (dict(out=FAKE + 8), AL), (dict(qkv=FAKE + 8), AL), (dict(workspace=FAKE + 8), AL), (dict(pos=FAKE + 2), AL),
    (dict(parent=FAKE + 1), AL), (dict(kv=ab.paged_kv(FAKE + 8, FAKE, 64, 16, 32)), AL),
    (dict(kv=ab.paged_kv(FAKE, FAKE + 2, 64, 16, 32)), AL),
    # 32 rows of 256 values: the output's last bytes are the first queries', or the other way round
    (dict(qkv=FAKE + 32 * 256 * 2 - 16), A), (dict(qkv=FAKE - 3 * 32 * 256 * 2 + 16), A),
])
def test_tree_attention_refuses(change, code):
    refused(code, ab.attention_tree, **attention_args(**change))


def test_tree_sizes():
    size = ab.attention_tree_workspace_size
    for bad in [(0, 8, 256, 4, 3), (4, 0, 256, 4, 3), (4, 65, 256, 4, 3), (4, 8, 256, 3, 3), (4, 8, 512, 4, 3),
                (4, 8, 256, 4, 9), (65536, 8, 256, 4, 3), (4, 8, 0, 4, 3), (4, 8, 256, 0, 3)]:
        assert size(*bad) == 0, bad
    for precision in (ab.GPT2_FP32, ab.GPT2_TF32, ab.GPT2_BF16, ab.GPT2_FP16):
        for hs in (16, 32, 64):
            got = [size(3, N, hs * 12, 12, precision) for N in range(1, 65)]
            assert all(g > 0 for g in got) and got == sorted(got)  # enough for every smaller tree
            assert len({size(B, 20, hs * 12, 12, precision) for B in (1, 7, 300)}) == 1  # and any batch
    cfg = inputs.TINY
    base, part = ab.gpt2_workspace_size(cfg, 3, 9, ab.GPT2_FP16), size(3, 9, 64, 4, ab.GPT2_FP16)
    assert ab.gpt2_tree_workspace_size(cfg, 3, 9, ab.GPT2_FP16) == base + part
    for bad in [(0, 9, 3), (3, 0, 3), (3, 65, 3), (3, 9, 7), (65536, 9, 3)]:
        assert ab.gpt2_tree_workspace_size(cfg, *bad) == 0, bad


def step_args(**kw):
    d = dict(cfg=inputs.TINY, params=FAKE, packed=FAKE, kv=ab.paged_kv(FAKE, FAKE, 64, 16, 4), tok=FAKE, parent=FAKE,
             pos=FAKE, B=4, N=7, logits=FAKE, probs=None, workspace=FAKE, ws_bytes=1 << 30, precision=ab.GPT2_FP16)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(params=None), A), (dict(tok=None), A), (dict(pos=None), A), (dict(logits=None), A), (dict(workspace=None), A),
    (dict(kv=None), A), (dict(packed=None), A), (dict(B=0), A), (dict(N=0), A), (dict(precision=7), A),
    (dict(N=65), S), (dict(B=65536), S), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 1025)), S),
    (dict(ws_bytes=100), W), (dict(ws_bytes=ab.GPT2_FP16), W), (dict(logits=FAKE + 4), AL),
    (dict(workspace=FAKE + 16), AL), (dict(tok=FAKE + 2), AL), (dict(parent=FAKE + 2), AL), (dict(pos=FAKE + 1), AL),
    (dict(probs=FAKE + 8), AL), (dict(packed=FAKE + 16), AL),
])
def test_tree_step_refuses(change, code):
    refused(code, ab.gpt2_decode_step_tree, **step_args(**change))


RULES = dict(history=FAKE, history_len=FAKE, prompt_len=FAKE, history_stride=9, repetition=FAKE, presence=FAKE,
             frequency=FAKE, bias_ids=FAKE, bias_values=FAKE, num_bias=3, masks=FAKE, mask_rows=FAKE, num_masks=2)


def adjust_args(rules=(), **kw):
    d = dict(out=FAKE, logits=FAKE, logits_type=ab.GPT2_PROBS_F32, rules=ab.logit_rules(**{**RULES, **dict(rules)}),
             tok=FAKE, parent=FAKE, B=2, N=3, V=10, Vp=12)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(out=None), A), (dict(logits=None), A), (dict(B=-1), A), (dict(N=0), A), (dict(V=0), A), (dict(V=13), A),
    (dict(logits_type=3), A), (dict(logits_type=-1), A), (dict(rules=None), A),
    (dict(N=65), S), (dict(B=65536), S), (dict(Vp=14), S), (dict(logits_type=ab.GPT2_PROBS_F16), S),
    (dict(logits_type=ab.GPT2_PROBS_BF16), S), (dict(V=(1 << 30) + 1, Vp=(1 << 30) + 8), S),
    (dict(logits=FAKE + 8), AL), (dict(out=FAKE + 8), AL), (dict(tok=FAKE + 2), AL), (dict(parent=FAKE + 1), AL),
    (dict(out=FAKE + 2 * 3 * 48 - 16), A), (dict(logits=FAKE + 48), A),  # they share a row
])
def test_adjust_refuses(change, code):
    refused(code, ab.logits_adjust, **{**adjust_args(), **change})


@pytest.mark.parametrize("change,code", [
    (dict(history=None), A), (dict(history_stride=-1), A), (dict(num_bias=-1), A), (dict(num_masks=-1), A),
    (dict(bias_ids=None), A), (dict(bias_values=None), A), (dict(masks=None), A), (dict(mask_rows=None), A),
    (dict(history_stride=(1 << 20) + 1), S), (dict(num_bias=1024), S),
    *((dict([(n, FAKE + 2)]), AL) for n in ("history", "history_len", "prompt_len", "repetition", "presence",
                                            "frequency", "bias_ids", "bias_values", "masks", "mask_rows")),
])
def test_adjust_refuses_rules(change, code):
    refused(code, ab.logits_adjust, **adjust_args(rules=change))


def accept_args(**kw):
    d = dict(path=FAKE, count=FAKE + 64, emitted=FAKE + 128, next_tok=FAKE + 192, next_pos=FAKE + 256, cfg=inputs.TINY,
             kv=ab.paged_kv(FAKE, FAKE, 64, 16, 4), tok=FAKE + 320, parent=FAKE + 384, next=FAKE + 448, pos=FAKE + 512,
             B=2, N=3, precision=ab.GPT2_FP16)
    d.update(kw)
    return d


@pytest.mark.parametrize("change,code", [
    (dict(tok=None), A), (dict(next=None), A), (dict(pos=None), A), (dict(B=-1), A), (dict(N=0), A),
    (dict(precision=4), A), (dict(cfg=None), A), (dict(kv=ab.paged_kv(None, FAKE, 64, 16, 4)), A),
    (dict(kv=ab.paged_kv(FAKE, None, 64, 16, 4)), A), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 15, 4)), A),
    (dict(kv=ab.paged_kv(FAKE, FAKE, 0, 16, 4)), A),
    # outputs that another CTA's inputs, or another output, would share
    (dict(next_pos=FAKE + 512), A), (dict(next_tok=FAKE + 320), A), (dict(emitted=FAKE + 448), A),
    (dict(path=FAKE + 384), A), (dict(count=FAKE + 256), A), (dict(path=FAKE + 128), A),
    (dict(path=FAKE + 384 - 20), A), (dict(next_tok=FAKE + 320 + 20), A), (dict(count=FAKE + 4), A),
    (dict(N=65), S), (dict(B=65536), S), (dict(kv=ab.paged_kv(FAKE, FAKE, 64, 16, 1025)), S),
    (dict(path=FAKE + 2), AL), (dict(next_pos=FAKE + 257), AL), (dict(tok=FAKE + 322), AL), (dict(pos=FAKE + 513), AL),
    (dict(parent=FAKE + 386), AL), (dict(kv=ab.paged_kv(FAKE + 8, FAKE, 64, 16, 4)), AL),
])
def test_accept_refuses(change, code):
    refused(code, ab.gpt2_accept_tree, **accept_args(**change))


def test_nothing_to_do_is_no_launch():
    ab.attention_tree(**attention_args(B=0), stream=0)
    ab.logits_adjust(**adjust_args(B=0), stream=0)
    ab.gpt2_accept_tree(**accept_args(B=0), stream=0)
    ab.gpt2_accept_tree(**accept_args(B=0, kv=None, cfg=None), stream=0)


@pytest.fixture(scope="module")
def cpu_model():
    """A model whose buffers are in host memory, for checks that come before
    any launch."""
    w = inputs.WORKLOADS["tiny"]
    params, _ = inputs.workload_inputs(w, "perturbed")
    return GPT2Model(w.cfg, params, 2, 4, ab.GPT2_FP32, device="cpu")


def calls_of(m, monkeypatch):
    """The runner's calls with good arguments, and what they reach."""
    reached = []
    for name in ("gpt2_decode_step_tree", "logits_adjust", "gpt2_accept_tree"):
        monkeypatch.setattr(ab, name, lambda *a, name=name: reached.append(name))
    Vp, V = m.cfg.padded_vocab_size, m.cfg.vocab_size
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    step = dict(kv=None, tok=i(2, 3), pos=i(2), logits=f(2, 3, Vp), workspace=torch.zeros(1, dtype=torch.uint8),
                parent=i(2, 3), probs=f(2, 3, Vp))
    adjust = dict(logits=f(2, 3, Vp), tok=i(2, 3), parent=i(2, 3), out=f(2, 3, Vp), history=i(2, 9), history_len=i(2),
                  prompt_len=i(2), repetition=f(2), presence=f(2), frequency=f(2), bias_ids=i(2, 5), bias_values=f(2, 5),
                  masks=i(4, (V + 31) // 32), mask_rows=i(2, 3))
    accept = dict(kv=None, tok=i(2, 3), chosen=i(2, 3), pos=i(2), parent=i(2, 3))
    return reached, [(m.decode_step_tree, step), (m.adjust_logits, adjust), (m.accept_tree, accept)]


def test_runner_calls_reach_the_library(cpu_model, monkeypatch):
    reached, calls = calls_of(cpu_model, monkeypatch)
    for call, args in calls:
        call(**args)
    calls[0][0](**{**calls[0][1], "parent": None, "probs": None})
    x = calls[1][1]["logits"]
    assert calls[1][0](x) is x and calls[1][0](x[:, 0].contiguous()).shape == x[:, 0].shape
    r = calls[2][0](**{**calls[2][1], "parent": None})
    assert {k: tuple(v.shape) for k, v in r.items()} == dict(path=(2, 3), count=(2,), emitted=(2, 3), next_tok=(2,),
                                                             next_pos=(2,))
    assert sorted(reached) == sorted(["gpt2_decode_step_tree", "logits_adjust", "gpt2_accept_tree"] * 2 + ["logits_adjust"])


@pytest.mark.parametrize("change", [
    lambda t: t.to(torch.int64 if t.dtype == torch.int32 else torch.float64),
    lambda t: torch.cat([t, t], -1)[..., ::2],                # strided
    lambda t: torch.cat([t, t]),                              # more rows
    lambda t: t[..., :-1].contiguous(),                       # shorter rows
    lambda t: t.to("meta"),
])
def test_runner_calls_refuse_what_they_would_misread(cpu_model, monkeypatch, change):
    reached, calls = calls_of(cpu_model, monkeypatch)
    for call, args in calls:
        for name, t in args.items():
            if not torch.is_tensor(t) or name == "workspace":
                continue
            bad = change(t)
            if bad.dtype == t.dtype and bad.device == t.device and bad.is_contiguous() and (
                    (name == "history" and bad.shape == (2, 8)) or (name == "masks" and len(bad) == 8)):
                continue  # a history of another length, other masks
            with pytest.raises((ValueError, TypeError)):
                call(**{**args, name: bad})
    assert not reached


def test_runner_calls_refuse_parts_without_their_others(cpu_model, monkeypatch):
    reached, calls = calls_of(cpu_model, monkeypatch)
    adjust, args = calls[1]
    for gone in ("history", "bias_ids", "bias_values", "masks", "mask_rows"):
        with pytest.raises(ValueError):
            adjust(**{**args, gone: None})
    step, args = calls[0]
    with pytest.raises(ValueError, match="workspace"):
        step(**{**args, "workspace": torch.zeros(8)})
    assert not reached
