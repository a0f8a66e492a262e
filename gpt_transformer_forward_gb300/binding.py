"""Thin Python binding of libgpt2fwd.so: the C ABI, name for name.

Argument marshalling only.  Pointer arguments accept a torch tensor (its
data_ptr), a raw integer address or None; `stream` accepts a torch.cuda.Stream,
a raw cudaStream_t integer or None (torch's current stream).  A negative
return code raises GPT2Error.  Every step of the forward pass runs in the
CUDA library; there is no Python or CPU fallback, and importing this module
fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import build as _build

GPT2_FP32, GPT2_TF32, GPT2_BF16, GPT2_FP16 = 0, 1, 2, 3
GPT2_PROBS_F32, GPT2_PROBS_F16, GPT2_PROBS_BF16 = 0, 1, 2
PRECISIONS = {"fp32": GPT2_FP32, "tf32": GPT2_TF32, "bf16": GPT2_BF16, "fp16": GPT2_FP16}

GPT2_OK = 0
ERRORS = {-1: "GPT2_ERR_ARG", -2: "GPT2_ERR_SHAPE", -3: "GPT2_ERR_ALIGN", -4: "GPT2_ERR_WORKSPACE",
          -5: "GPT2_ERR_CUDA", -6: "GPT2_ERR_DEVICE", -7: "GPT2_ERR_UNSUPPORTED"}
DEVERR_TOKEN, DEVERR_TIMEOUT, DEVERR_POSITION, DEVERR_BLOCK, DEVERR_TREE = 1, 2, 4, 8, 16


class GPT2Error(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        detail = ""
        if code == -5:
            detail = ": " + _lib().gpt2_last_cuda_error().decode()
        super().__init__(f"{fn} returned {ERRORS.get(code, code)}{detail}")


class GPT2Config(ctypes.Structure):
    _fields_ = [("max_seq_len", ctypes.c_int), ("vocab_size", ctypes.c_int),
                ("padded_vocab_size", ctypes.c_int), ("num_layers", ctypes.c_int),
                ("num_heads", ctypes.c_int), ("channels", ctypes.c_int)]

    @classmethod
    def of(cls, cfg) -> "GPT2Config":
        if isinstance(cfg, cls):
            return cfg
        return cls(cfg.max_seq_len, cfg.vocab_size, cfg.padded_vocab_size, cfg.num_layers,
                   cfg.num_heads, cfg.channels)


class GPT2PagedKVCache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("num_blocks", ctypes.c_int),
                ("block_size", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int)]


class GPT2LogitRules(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("history", "history_len", "prompt_len", "repetition", "presence",
                                               "frequency", "bias_ids", "bias_values", "masks", "mask_rows")] + [
        (n, ctypes.c_int) for n in ("history_stride", "num_bias", "num_masks")]


_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_CFG = ctypes.POINTER(GPT2Config)
_PKV = ctypes.POINTER(GPT2PagedKVCache)
_RULES = ctypes.POINTER(GPT2LogitRules)

# name -> (restype, argtypes), in the order of include/gpt2fwd.h
_SIGNATURES = {
    "encoder_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "layernorm_forward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _P]),
    "matmul_workspace_size": (_Z, [_I, _I, _I, _I]),
    "matmul_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]),
    "matmul_forward_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "attention_workspace_size": (_Z, [_I, _I, _I, _I]),
    "attention_forward": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "attention_backward_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "attention_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "gelu_forward": (_I, [_P, _P, _I, _P]),
    "residual_forward": (_I, [_P, _P, _P, _I, _P]),
    "softmax_forward": (_I, [_P, _P, _I, _I, _I, _P]),
    "softmax_forward_ex": (_I, [_P, _I, _P, _I, _I, _I, _P]),
    "gpt2_argmax": (_I, [_P, _P, _I, _I, _I, _P]),
    "gpt2_num_parameters": (_Z, [_CFG]),
    "gpt2_packed_weights_size": (_Z, [_CFG, _I]),
    "gpt2_prepare_weights": (_I, [_CFG, _P, _P, _Z, _I, _P]),
    "gpt2_workspace_size": (_Z, [_CFG, _I, _I, _I]),
    "gpt2_kvcache_size": (_Z, [_CFG, _I, _I]),
    "gpt2_forward": (_I, [_CFG, _P, _P, _P, _I, _I, _P, _P, _P, _P, _Z, _I, _P]),
    "gpt2_forward_ex": (_I, [_CFG, _P, _P, _P, _I, _I, _P, _P, _I, _P, _P, _Z, _I, _P]),
    "gpt2_decode_step": (_I, [_CFG, _P, _P, _P, _P, _I, _I, _P, _P, _P, _Z, _I, _P]),
    "gpt2_train_workspace_size": (_Z, [_CFG, _I, _I, _I]),
    "gpt2_forward_backward": (_I, [_CFG, _P, _P, _P, _P, _I, _I, _P, _P, _Z, _I, _P]),
    "gpt2_adamw": (_I, [_P, _P, _P, _P, _Z, ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                        ctypes.c_float, _I, _P]),
    "gpt2_paged_kvcache_size": (_Z, [_CFG, _I, _I, _I]),
    "gpt2_prefill_paged": (_I, [_CFG, _P, _P, _P, _I, _I, _P, _P, _PKV, _P, _Z, _I, _P]),
    "gpt2_decode_step_paged": (_I, [_CFG, _P, _P, _PKV, _P, _P, _I, _P, _P, _P, _Z, _I, _P]),
    "gpt2_forward_profile": (_I, [_CFG, _P, _P, _P, _I, _I, _P, _P, _I, _P, _Z, _I, _P, _P, _I]),
    "gpt2_get_error": (_I, [_P]),
    "gpt2_strerror": (ctypes.c_char_p, [_I]),
    "gpt2_last_cuda_error": (ctypes.c_char_p, []),
    "gpt2_diag_wait_timeout": (_I, [ctypes.c_longlong, _P, _P]),
}

# the same for include/gpt2fwd_serve.h
_SERVE_SIGNATURES = {
    "paged_build_tables": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "gpt2_prefill_slots": (_I, [_CFG, _P, _P, _P, _I, _I, _P, _P, _PKV, _P, _P, _Z, _I, _P]),
    "attention_shared_prefix_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "attention_shared_prefix": (_I, [_P, _P, _PKV, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "gpt2_shared_workspace_size": (_Z, [_CFG, _I, _I, _I]),
    "gpt2_decode_step_shared": (_I, [_CFG, _P, _P, _PKV, _P, _P, _I, _I, _P, _P, _P, _Z, _I, _P]),
    "logprobs_forward": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _P]),
    "logprobs_backward": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
}

# the same for include/gpt2fwd_draft.h
_DRAFT_SIGNATURES = {
    "attention_tree_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "attention_tree": (_I, [_P, _P, _PKV, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "gpt2_tree_workspace_size": (_Z, [_CFG, _I, _I, _I]),
    "gpt2_decode_step_tree": (_I, [_CFG, _P, _P, _PKV, _P, _P, _P, _I, _I, _P, _P, _P, _Z, _I, _P]),
    "logits_adjust": (_I, [_P, _P, _I, _RULES, _P, _P, _I, _I, _I, _I, _P]),
    "gpt2_accept_tree": (_I, [_P, _P, _P, _P, _P, _CFG, _PKV, _P, _P, _P, _P, _I, _I, _I, _P]),
    "gpt2_diag_tree_join": (_I, [_P, _I, _I, _I, _I, _I, _I, _P, _Z, _P]),
}

_handle = None


def library_path() -> str:
    return _build.LIB


def _lib():
    global _handle
    if _handle is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"libgpt2fwd.so is not built ({path}); run "
                              "`python -m gpt_transformer_forward_gb300.build`")
        h = ctypes.CDLL(path)
        for name, (res, args) in {**_SIGNATURES, **_SERVE_SIGNATURES, **_DRAFT_SIGNATURES}.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _handle = h
    return _handle


def load(build_if_missing: bool = True):
    """Loads the library (building it first when asked and needed)."""
    if build_if_missing:
        _build.build()
    return _lib()


def header_functions(header: str = "gpt2fwd.h") -> list:
    """Function names declared in a header of include/."""
    path = os.path.join(_build.INCLUDE, header)
    with open(path) as f:
        return re.findall(r"^GPT2_API [^(]*?\b([a-z_0-9]+)\(", f.read(), flags=re.M)


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    try:  # a torch tensor
        return x.data_ptr()
    except AttributeError:
        pass
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(s):
    if s is None:
        import torch
        # the handle alone (0.3 us; building the stream object takes 3 us, as
        # long as a small call's kernel)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn: str, rc: int):
    if rc < 0:
        raise GPT2Error(fn, rc)
    return rc


def _cfg(cfg):
    return ctypes.byref(GPT2Config.of(cfg))


# --------------------------------------------------------------- the ABI
def encoder_forward(out, tok, wte, wpe, B, T, C, V, stream=None):
    _check("encoder_forward", _lib().encoder_forward(_ptr(out), _ptr(tok), _ptr(wte), _ptr(wpe), B, T, C, V,
                                                     _stream(stream)))


def layernorm_forward(out, mean, rstd, inp, w, b, N, C, stream=None):
    _check("layernorm_forward", _lib().layernorm_forward(_ptr(out), _ptr(mean), _ptr(rstd), _ptr(inp), _ptr(w),
                                                         _ptr(b), N, C, _stream(stream)))


def matmul_workspace_size(N, C, OC, precision) -> int:
    return _lib().matmul_workspace_size(N, C, OC, precision)


def matmul_forward(out, inp, W, bias, N, C, OC, precision, workspace=None, ws_bytes=0, stream=None):
    _check("matmul_forward", _lib().matmul_forward(_ptr(out), _ptr(inp), _ptr(W), _ptr(bias), N, C, OC, precision,
                                                   _ptr(workspace), ws_bytes, _stream(stream)))


def matmul_forward_noalloc(out, inp, W, bias, N, C, OC, precision, stream=None):
    """matmul_forward with its scratch in the library's fixed 16 MiB device
    array instead of a caller workspace (for callers that cannot allocate)."""
    _check("matmul_forward_noalloc", _lib().matmul_forward_noalloc(_ptr(out), _ptr(inp), _ptr(W), _ptr(bias), N, C,
                                                                   OC, precision, _stream(stream)))


def attention_workspace_size(B, T, C, precision) -> int:
    return _lib().attention_workspace_size(B, T, C, precision)


def attention_forward(out, qkv, B, T, C, NH, precision, workspace=None, ws_bytes=0, stream=None):
    _check("attention_forward", _lib().attention_forward(_ptr(out), _ptr(qkv), B, T, C, NH, precision,
                                                         _ptr(workspace), ws_bytes, _stream(stream)))


def attention_backward_workspace_size(B, T, C, NH, precision) -> int:
    return _lib().attention_backward_workspace_size(B, T, C, NH, precision)


def attention_backward(dqkv, dout, qkv, out, B, T, C, NH, precision, workspace=None, ws_bytes=0, stream=None):
    _check("attention_backward", _lib().attention_backward(_ptr(dqkv), _ptr(dout), _ptr(qkv), _ptr(out), B, T, C, NH,
                                                           precision, _ptr(workspace), ws_bytes, _stream(stream)))


def gelu_forward(out, inp, n, stream=None):
    _check("gelu_forward", _lib().gelu_forward(_ptr(out), _ptr(inp), n, _stream(stream)))


def residual_forward(out, a, b, n, stream=None):
    _check("residual_forward", _lib().residual_forward(_ptr(out), _ptr(a), _ptr(b), n, _stream(stream)))


def softmax_forward(probs, logits, N, V, Vp, stream=None):
    _check("softmax_forward", _lib().softmax_forward(_ptr(probs), _ptr(logits), N, V, Vp, _stream(stream)))


def softmax_forward_ex(probs, probs_type, logits, N, V, Vp, stream=None):
    _check("softmax_forward_ex", _lib().softmax_forward_ex(_ptr(probs), probs_type, _ptr(logits), N, V, Vp,
                                                           _stream(stream)))


def gpt2_argmax(next_tok, logits, B, V, Vp, stream=None):
    _check("gpt2_argmax", _lib().gpt2_argmax(_ptr(next_tok), _ptr(logits), B, V, Vp, _stream(stream)))


def gpt2_num_parameters(cfg) -> int:
    return _lib().gpt2_num_parameters(_cfg(cfg))


def gpt2_packed_weights_size(cfg, precision) -> int:
    return _lib().gpt2_packed_weights_size(_cfg(cfg), precision)


def gpt2_prepare_weights(cfg, params, packed, nbytes, precision, stream=None):
    _check("gpt2_prepare_weights", _lib().gpt2_prepare_weights(_cfg(cfg), _ptr(params), _ptr(packed), nbytes,
                                                               precision, _stream(stream)))


def gpt2_workspace_size(cfg, B, T, precision) -> int:
    return _lib().gpt2_workspace_size(_cfg(cfg), B, T, precision)


def gpt2_kvcache_size(cfg, B, precision) -> int:
    return _lib().gpt2_kvcache_size(_cfg(cfg), B, precision)


def gpt2_forward(cfg, params, packed, tok, B, T, logits, probs, kvcache, workspace, ws_bytes, precision,
                 stream=None):
    _check("gpt2_forward", _lib().gpt2_forward(_cfg(cfg), _ptr(params), _ptr(packed), _ptr(tok), B, T, _ptr(logits),
                                               _ptr(probs), _ptr(kvcache), _ptr(workspace), ws_bytes, precision,
                                               _stream(stream)))


def gpt2_forward_ex(cfg, params, packed, tok, B, T, logits, probs, probs_type, kvcache, workspace, ws_bytes,
                    precision, stream=None):
    _check("gpt2_forward_ex", _lib().gpt2_forward_ex(_cfg(cfg), _ptr(params), _ptr(packed), _ptr(tok), B, T,
                                                     _ptr(logits), _ptr(probs), probs_type, _ptr(kvcache),
                                                     _ptr(workspace), ws_bytes, precision, _stream(stream)))


def gpt2_decode_step(cfg, params, packed, kvcache, tok, B, pos, logits, probs, workspace, ws_bytes, precision,
                     stream=None):
    _check("gpt2_decode_step", _lib().gpt2_decode_step(_cfg(cfg), _ptr(params), _ptr(packed), _ptr(kvcache),
                                                       _ptr(tok), B, pos, _ptr(logits), _ptr(probs),
                                                       _ptr(workspace), ws_bytes, precision, _stream(stream)))


STAGES = ["encoder", "ln1", "qkv", "attention", "attproj", "ln2", "fc", "fcproj", "lnf", "lm_head", "softmax"]


def gpt2_train_workspace_size(cfg, B, T, precision) -> int:
    return _lib().gpt2_train_workspace_size(_cfg(cfg), B, T, precision)


def gpt2_forward_backward(cfg, params, grads, tok, targets, B, T, loss, workspace, ws_bytes, precision,
                          stream=None):
    _check("gpt2_forward_backward", _lib().gpt2_forward_backward(
        _cfg(cfg), _ptr(params), _ptr(grads), _ptr(tok), _ptr(targets), B, T, _ptr(loss), _ptr(workspace), ws_bytes,
        precision, _stream(stream)))


def gpt2_adamw(params, grads, m, v, n, lr, beta1, beta2, eps, weight_decay, t, stream=None):
    _check("gpt2_adamw", _lib().gpt2_adamw(_ptr(params), _ptr(grads), _ptr(m), _ptr(v), n, lr, beta1, beta2, eps,
                                           weight_decay, t, _stream(stream)))


def paged_kv(pool, block_table, num_blocks, block_size, max_blocks_per_seq) -> GPT2PagedKVCache:
    """The C struct describing a paged cache (pool and block_table: device
    tensors or addresses)."""
    return GPT2PagedKVCache(_ptr(pool), _ptr(block_table), num_blocks, block_size, max_blocks_per_seq)


def gpt2_paged_kvcache_size(cfg, num_blocks, block_size, precision) -> int:
    return _lib().gpt2_paged_kvcache_size(_cfg(cfg), num_blocks, block_size, precision)


def gpt2_prefill_paged(cfg, params, packed, tok, B, T, logits, probs, kv, workspace, ws_bytes, precision,
                       stream=None):
    _check("gpt2_prefill_paged", _lib().gpt2_prefill_paged(
        _cfg(cfg), _ptr(params), _ptr(packed), _ptr(tok), B, T, _ptr(logits), _ptr(probs),
        ctypes.byref(kv) if kv is not None else None, _ptr(workspace), ws_bytes, precision, _stream(stream)))


def gpt2_decode_step_paged(cfg, params, packed, kv, tok, pos, B, logits, probs, workspace, ws_bytes, precision,
                           stream=None):
    _check("gpt2_decode_step_paged", _lib().gpt2_decode_step_paged(
        _cfg(cfg), _ptr(params), _ptr(packed), ctypes.byref(kv) if kv is not None else None, _ptr(tok), _ptr(pos), B,
        _ptr(logits), _ptr(probs), _ptr(workspace), ws_bytes, precision, _stream(stream)))


# ------------------------------------------- gpt2fwd_serve.h
LOGPROBS_MAX_TOP = 32


_element_types: dict = {}  # torch dtype -> code, filled at the first use


def element_type(t) -> int:
    """The GPT2ProbsType code of a tensor's dtype (fp32, fp16 or bf16)."""
    code = _element_types.get(t.dtype)
    if code is None:
        import torch
        _element_types.update({torch.float32: GPT2_PROBS_F32, torch.float16: GPT2_PROBS_F16,
                               torch.bfloat16: GPT2_PROBS_BF16})
        code = _element_types.get(t.dtype)
        if code is None:
            raise TypeError(f"element type {t.dtype}: fp32, fp16 or bf16 expected")
    return code


def paged_build_tables(block_table, slots, next_len, taken_out, cached_len, new_len, free_blocks, num_free, taken_in,
                       prefix_blocks, prefix_len, B, T, num_blocks, block_size, max_blocks_per_seq, stream=None):
    _check("paged_build_tables", _lib().paged_build_tables(
        _ptr(block_table), _ptr(slots), _ptr(next_len), _ptr(taken_out), _ptr(cached_len), _ptr(new_len),
        _ptr(free_blocks), num_free, _ptr(taken_in), _ptr(prefix_blocks), prefix_len, B, T, num_blocks, block_size,
        max_blocks_per_seq, _stream(stream)))


def gpt2_prefill_slots(cfg, params, packed, tok, B, T, logits, probs, kv, slots, workspace, ws_bytes, precision,
                       stream=None):
    _check("gpt2_prefill_slots", _lib().gpt2_prefill_slots(
        _cfg(cfg), _ptr(params), _ptr(packed), _ptr(tok), B, T, _ptr(logits), _ptr(probs),
        ctypes.byref(kv) if kv is not None else None, _ptr(slots), _ptr(workspace), ws_bytes, precision,
        _stream(stream)))


def attention_shared_prefix_workspace_size(B, C, NH, prefix_len, precision) -> int:
    return _lib().attention_shared_prefix_workspace_size(B, C, NH, prefix_len, precision)


def attention_shared_prefix(out, qkv, kv, pos, B, C, NH, prefix_len, precision, workspace=None, ws_bytes=0,
                            stream=None):
    """kv: one layer's slab and the block table (paged_kv)."""
    _check("attention_shared_prefix", _lib().attention_shared_prefix(
        _ptr(out), _ptr(qkv), ctypes.byref(kv) if kv is not None else None, _ptr(pos), B, C, NH, prefix_len, precision,
        _ptr(workspace), ws_bytes, _stream(stream)))


def gpt2_shared_workspace_size(cfg, B, prefix_len, precision) -> int:
    return _lib().gpt2_shared_workspace_size(_cfg(cfg), B, prefix_len, precision)


def gpt2_decode_step_shared(cfg, params, packed, kv, tok, pos, B, prefix_len, logits, probs, workspace, ws_bytes,
                            precision, stream=None):
    _check("gpt2_decode_step_shared", _lib().gpt2_decode_step_shared(
        _cfg(cfg), _ptr(params), _ptr(packed), ctypes.byref(kv) if kv is not None else None, _ptr(tok), _ptr(pos), B,
        prefix_len, _ptr(logits), _ptr(probs), _ptr(workspace), ws_bytes, precision, _stream(stream)))


def logprobs_forward(logprob, entropy, lse, top_ids, top_logprobs, logits, logits_type, targets, N, V, Vp, K,
                     stream=None):
    _check("logprobs_forward", _lib().logprobs_forward(
        _ptr(logprob), _ptr(entropy), _ptr(lse), _ptr(top_ids), _ptr(top_logprobs), _ptr(logits), logits_type,
        _ptr(targets), N, V, Vp, K, _stream(stream)))


def logprobs_backward(dlogits, logits, logits_type, targets, lse, entropy, dlogprob, dentropy, N, V, Vp, stream=None):
    _check("logprobs_backward", _lib().logprobs_backward(
        _ptr(dlogits), _ptr(logits), logits_type, _ptr(targets), _ptr(lse), _ptr(entropy), _ptr(dlogprob),
        _ptr(dentropy), N, V, Vp, _stream(stream)))


# ------------------------------------------- gpt2fwd_draft.h
TREE_MAX_NODES = 64
LOGIT_MAX_BIASES = 1023
LOGIT_MAX_HISTORY = 1 << 20


def attention_tree_workspace_size(B, N, C, NH, precision) -> int:
    return _lib().attention_tree_workspace_size(B, N, C, NH, precision)


def attention_tree(out, qkv, kv, pos, parent, B, N, C, NH, precision, workspace=None, ws_bytes=0, stream=None):
    """kv: one layer's slab and the block table (paged_kv)."""
    _check("attention_tree", _lib().attention_tree(
        _ptr(out), _ptr(qkv), ctypes.byref(kv) if kv is not None else None, _ptr(pos), _ptr(parent), B, N, C, NH,
        precision, _ptr(workspace), ws_bytes, _stream(stream)))


def gpt2_tree_workspace_size(cfg, B, N, precision) -> int:
    return _lib().gpt2_tree_workspace_size(_cfg(cfg), B, N, precision)


def gpt2_decode_step_tree(cfg, params, packed, kv, tok, parent, pos, B, N, logits, probs, workspace, ws_bytes,
                          precision, stream=None):
    _check("gpt2_decode_step_tree", _lib().gpt2_decode_step_tree(
        _cfg(cfg), _ptr(params), _ptr(packed), ctypes.byref(kv) if kv is not None else None, _ptr(tok), _ptr(parent),
        _ptr(pos), B, N, _ptr(logits), _ptr(probs), _ptr(workspace), ws_bytes, precision, _stream(stream)))


def logit_rules(history=None, history_len=None, prompt_len=None, history_stride=0, repetition=None, presence=None,
                frequency=None, bias_ids=None, bias_values=None, num_bias=0, masks=None, mask_rows=None,
                num_masks=0) -> GPT2LogitRules:
    """The C struct of logits_adjust (device tensors or addresses); it keeps
    what it was made of."""
    kept = (history, history_len, prompt_len, repetition, presence, frequency, bias_ids, bias_values, masks, mask_rows)
    r = GPT2LogitRules(*map(_ptr, kept), history_stride, num_bias, num_masks)
    r.kept = kept
    return r


def logits_adjust(out, logits, logits_type, rules, tok, parent, B, N, V, Vp, stream=None):
    _check("logits_adjust", _lib().logits_adjust(
        _ptr(out), _ptr(logits), logits_type, ctypes.byref(rules) if rules is not None else None, _ptr(tok),
        _ptr(parent), B, N, V, Vp, _stream(stream)))


def gpt2_accept_tree(path, count, emitted, next_tok, next_pos, cfg, kv, tok, parent, next, pos, B, N, precision,
                     stream=None):
    _check("gpt2_accept_tree", _lib().gpt2_accept_tree(
        _ptr(path), _ptr(count), _ptr(emitted), _ptr(next_tok), _ptr(next_pos), _cfg(cfg) if cfg is not None else None,
        ctypes.byref(kv) if kv is not None else None, _ptr(tok), _ptr(parent), _ptr(next), _ptr(pos), B, N, precision,
        _stream(stream)))


def gpt2_diag_tree_join(out, B, N, C, NH, shares, precision, workspace, ws_bytes, stream=None):
    """The last launch of an attention_tree over long tables, by itself (see the
    header)."""
    _check("gpt2_diag_tree_join", _lib().gpt2_diag_tree_join(
        _ptr(out), B, N, C, NH, shares, precision, _ptr(workspace), ws_bytes, _stream(stream)))


def gpt2_forward_profile(cfg, params, packed, tok, B, T, logits, probs, workspace, ws_bytes, precision,
                         stream=None, probs_type=GPT2_PROBS_F32) -> dict:
    """Runs one forward pass with per-stage CUDA events; returns {stage: ms}."""
    ms = (ctypes.c_float * len(STAGES))()
    _check("gpt2_forward_profile", _lib().gpt2_forward_profile(
        _cfg(cfg), _ptr(params), _ptr(packed), _ptr(tok), B, T, _ptr(logits), _ptr(probs), probs_type,
        _ptr(workspace), ws_bytes, precision, _stream(stream), ctypes.cast(ms, ctypes.c_void_p), len(STAGES)))
    return dict(zip(STAGES, list(ms)))


def gpt2_get_error(stream=None) -> int:
    return _check("gpt2_get_error", _lib().gpt2_get_error(_stream(stream)))


def gpt2_strerror(code) -> str:
    return _lib().gpt2_strerror(code).decode()


def gpt2_last_cuda_error() -> str:
    return _lib().gpt2_last_cuda_error().decode()


def gpt2_diag_wait_timeout(limit_ns, gave_up, stream=None):
    """Runs the bounded-wait path once (see the header); gave_up: a device
    int32 tensor of one element."""
    _check("gpt2_diag_wait_timeout", _lib().gpt2_diag_wait_timeout(int(limit_ns), _ptr(gave_up), _stream(stream)))
