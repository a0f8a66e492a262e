"""Device buffers around the C ABI: a GPT-2 model ready to run forward passes
and decode steps on one GPU.

PyTorch only provides device memory and the stream here; every kernel that
touches the data is the CUDA library's, reached through `binding`.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding as ab

# the probabilities' element type from the output tensor's dtype
_PROBS_TYPE = {torch.float32: ab.GPT2_PROBS_F32, torch.float16: ab.GPT2_PROBS_F16,
               torch.bfloat16: ab.GPT2_PROBS_BF16}


def probs_type(probs) -> int:
    return ab.GPT2_PROBS_F32 if probs is None else _PROBS_TYPE[probs.dtype]


def _allocating_on(stream):
    """Memory allocated within belongs to `stream` (a torch stream or a raw
    handle; None: the current one), where its kernel runs: that of another
    stream may still be in use there by work queued earlier."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _check_int32(t, name: str, shape) -> None:
    """The calls take plain pointers: a tensor of another type, shape or
    layout would be read as something else."""
    if t.dtype != torch.int32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: contiguous int32 of shape {tuple(shape)} expected, not {t.dtype} of shape "
                         f"{tuple(t.shape)}{'' if t.is_contiguous() else ', strided'}")


def _check_fp32_probs(probs) -> None:
    """Only forward writes probabilities of other types; into a 16-bit buffer the
    fp32 rows of the other calls go past its end."""
    if probs is not None and probs.dtype != torch.float32:
        raise ValueError(f"probs: fp32 expected, not {probs.dtype}")


def _check_outputs(logits, probs, shape) -> None:
    """Buffers of another type or size than the fp32 rows that a call writes
    would be written past their end."""
    for name, t in (("logits", logits), ("probs", probs)):
        if name == "probs" and t is None:
            continue
        if t is None or t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
            got = "none" if t is None else f"{t.dtype} of shape {tuple(t.shape)}{'' if t.is_contiguous() else ', strided'}"
            raise ValueError(f"{name}: contiguous fp32 of shape {tuple(shape)} expected, not {got}")


def _check_device(device, **tensors) -> None:
    """Kernels run on the current device and take plain addresses: those of host
    memory or of another device are not theirs to read."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name}: on {t.device}, the model is on {device}")
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError(f"the model is on {device}, the current device is cuda:{torch.cuda.current_device()}")


class GPT2Model:
    """Parameters (fp32, plus the packed bf16 weights in GPT2_BF16 mode) and a
    workspace sized for batches of up to B sequences of up to T tokens."""

    def __init__(self, cfg, params, B: int, T: int, precision: int = ab.GPT2_BF16, device="cuda"):
        ab.load()
        self.cfg = cfg
        self.precision = precision
        self.device = torch.device(device)
        p = torch.as_tensor(params)
        n = ab.gpt2_num_parameters(cfg)
        if p.numel() != n:
            raise ValueError(f"parameter buffer has {p.numel()} values, the config needs {n}")
        self.params = p.to(self.device, dtype=torch.float32).contiguous()
        nbytes = ab.gpt2_packed_weights_size(cfg, precision)
        self.packed = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
        if self.packed is not None:
            ab.gpt2_prepare_weights(cfg, self.params, self.packed, nbytes, precision)
        self.B, self.T = B, T
        self.ws_bytes = max(ab.gpt2_workspace_size(cfg, B, T, precision),
                            ab.gpt2_workspace_size(cfg, B, 1, precision))
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    # ---------------------------------------------------------------- buffers
    def new_outputs(self, B: int, T: int, probs: bool = True, probs_dtype=torch.float32):
        Vp = self.cfg.padded_vocab_size
        shape = (B, T, Vp) if T is not None else (B, Vp)
        logits = torch.empty(shape, dtype=torch.float32, device=self.device)
        pr = torch.empty(shape, dtype=probs_dtype, device=self.device) if probs else None
        return logits, pr

    def new_kvcache(self, B: int):
        nbytes = ab.gpt2_kvcache_size(self.cfg, B, self.precision)
        return torch.zeros(nbytes, dtype=torch.uint8, device=self.device)

    def new_paged_kvcache(self, num_blocks: int, block_size: int):
        """A zeroed pool of num_blocks blocks of block_size positions."""
        nbytes = ab.gpt2_paged_kvcache_size(self.cfg, num_blocks, block_size, self.precision)
        return torch.zeros(nbytes, dtype=torch.uint8, device=self.device)

    # ----------------------------------------------------------------- calls
    def forward(self, tok, logits, probs=None, kvcache=None, stream=None):
        """probs (optional): fp32, fp16 or bf16, [B, T, Vp]."""
        B, T = tok.shape
        ab.gpt2_forward_ex(self.cfg, self.params, self.packed, tok, B, T, logits, probs, probs_type(probs), kvcache,
                           self.workspace, self.ws_bytes, self.precision, stream)

    def forward_profile(self, tok, logits, probs=None, stream=None) -> dict:
        B, T = tok.shape
        return ab.gpt2_forward_profile(self.cfg, self.params, self.packed, tok, B, T, logits, probs,
                                       self.workspace, self.ws_bytes, self.precision, stream,
                                       probs_type=probs_type(probs))

    def decode_step(self, kvcache, tok, pos: int, logits, probs=None, stream=None):
        _check_fp32_probs(probs)
        B = tok.shape[0]
        ab.gpt2_decode_step(self.cfg, self.params, self.packed, kvcache, tok, B, pos, logits, probs,
                            self.workspace, self.ws_bytes, self.precision, stream)

    def prefill_paged(self, tok, logits, kv, probs=None, stream=None):
        """gpt2_forward writing positions [0, T) through the paged cache kv
        (a binding.GPT2PagedKVCache)."""
        _check_fp32_probs(probs)
        B, T = tok.shape
        ab.gpt2_prefill_paged(self.cfg, self.params, self.packed, tok, B, T, logits, probs, kv, self.workspace,
                              self.ws_bytes, self.precision, stream)

    def decode_step_paged(self, kv, tok, pos, logits, probs=None, stream=None):
        """One decode step, sequence b at position pos[b] (a device int32
        tensor)."""
        _check_fp32_probs(probs)
        B = tok.shape[0]
        ab.gpt2_decode_step_paged(self.cfg, self.params, self.packed, kv, tok, pos, B, logits, probs, self.workspace,
                                  self.ws_bytes, self.precision, stream)

    # ------------------------------------- many continuations of one prompt
    def prefill_slots(self, tok, logits, kv, slots, probs=None, stream=None):
        """gpt2_forward storing token (b, t) at slot slots[b, t] of kv's pool
        (none where it is -1).  tok, slots: contiguous int32 [B, T]."""
        B, T = tok.shape
        _check_int32(slots, "slots", (B, T))
        _check_int32(tok, "tok", (B, T))
        _check_outputs(logits, probs, (B, T, self.cfg.padded_vocab_size))
        _check_device(self.params.device, tok=tok, slots=slots, logits=logits, probs=probs)
        ab.gpt2_prefill_slots(self.cfg, self.params, self.packed, tok, B, T, logits, probs, kv, slots, self.workspace,
                              self.ws_bytes, self.precision, stream)

    def new_shared_workspace(self, B: int, prefix_len: int):
        """A workspace for decode_step_shared with up to B sequences and this prefix."""
        nbytes = ab.gpt2_shared_workspace_size(self.cfg, B, prefix_len, self.precision)
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def decode_step_shared(self, kv, tok, pos, prefix_len: int, logits, workspace, probs=None, stream=None):
        """decode_step_paged for sequences that share their first prefix_len
        positions; tok, pos: contiguous int32 [B], position -1 for a sequence
        without a token in this step; workspace from new_shared_workspace."""
        B = tok.shape[0]
        _check_int32(pos, "pos", (B,))
        _check_int32(tok, "tok", (B,))
        _check_outputs(logits, probs, (B, self.cfg.padded_vocab_size))
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: new_shared_workspace's expected")
        _check_device(self.params.device, tok=tok, pos=pos, logits=logits, probs=probs, workspace=workspace)
        ab.gpt2_decode_step_shared(self.cfg, self.params, self.packed, kv, tok, pos, B, prefix_len, logits, probs,
                                   workspace, workspace.numel(), self.precision, stream)

    def logprobs(self, logits, targets=None, top: int = 0, stream=None) -> dict:
        """The log probability of each row's target (targets: int32 of the
        logits' leading shape, -1 for none), its entropy, log-sum-exp and
        `top` alternatives, of logits [..., Vp]; results have the logits'
        leading shape and belong to `stream`.  Logits are contiguous: to
        score a part of the positions give the others target -1."""
        shape, Vp = logits.shape[:-1], logits.shape[-1]
        kind = ab.element_type(logits)
        if not logits.is_contiguous():
            raise ValueError(f"logits: contiguous rows expected, not strides {logits.stride()} of shape "
                             f"{tuple(logits.shape)}")
        if targets is not None:
            _check_int32(targets, "targets", shape)
        _check_device(self.params.device, logits=logits, targets=targets)
        new = lambda *more, dtype=torch.float32: torch.empty((*shape, *more), dtype=dtype, device=logits.device)  # noqa: E731
        with _allocating_on(stream):
            r = {"entropy": new(), "lse": new()}
            if targets is not None:
                r["logprob"] = new()
            if top:
                r["top_ids"], r["top_logprobs"] = new(top, dtype=torch.int32), new(top)
        ab.logprobs_forward(r.get("logprob"), r["entropy"], r["lse"], r.get("top_ids"), r.get("top_logprobs"), logits,
                            kind, targets, r["lse"].numel(), self.cfg.vocab_size, Vp, top, stream)
        return r

    # ------------------------------------------------ trees of drafted tokens
    def new_tree_workspace(self, B: int, N: int):
        """A workspace for decode_step_tree with up to B trees of up to N nodes."""
        nbytes = ab.gpt2_tree_workspace_size(self.cfg, B, N, self.precision)
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def decode_step_tree(self, kv, tok, pos, logits, workspace, parent=None, probs=None, stream=None):
        """One step for a tree of tokens a sequence: tok (and parent, None for
        chains): contiguous int32 [B, N], pos: int32 [B], -1 for a sequence
        without a tree in this step; logits (and probs) fp32 [B, N, Vp];
        workspace from new_tree_workspace."""
        B, N = tok.shape
        _check_int32(tok, "tok", (B, N))
        _check_int32(pos, "pos", (B,))
        if parent is not None:
            _check_int32(parent, "parent", (B, N))
        _check_outputs(logits, probs, (B, N, self.cfg.padded_vocab_size))
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: new_tree_workspace's expected")
        _check_device(self.params.device, tok=tok, pos=pos, parent=parent, logits=logits, probs=probs,
                      workspace=workspace)
        ab.gpt2_decode_step_tree(self.cfg, self.params, self.packed, kv, tok, parent, pos, B, N, logits, probs,
                                 workspace, workspace.numel(), self.precision, stream)

    def adjust_logits(self, logits, tok=None, parent=None, out=None, *, history=None, history_len=None,
                      prompt_len=None, repetition=None, presence=None, frequency=None, bias_ids=None,
                      bias_values=None, masks=None, mask_rows=None, stream=None):
        """Penalties, biases and masks on logits [B, N, Vp] (or [B, Vp]: one row a
        sequence), in place or into `out`, which is returned.  tok, parent: int32
        [B, N], the trees; history [B, H], history_len, prompt_len [B], bias_ids
        [B, M]: int32; repetition, presence, frequency [B], bias_values [B, M]:
        fp32; masks: int32 [G, ceil(V / 32)], mask_rows int32 of the logits'
        leading shape.  All contiguous."""
        V, Vp = self.cfg.vocab_size, self.cfg.padded_vocab_size
        if logits.dim() not in (2, 3) or logits.shape[-1] != Vp or not logits.is_contiguous():
            raise ValueError(f"logits: contiguous rows of {Vp} expected, not shape {tuple(logits.shape)}, strides "
                             f"{logits.stride()}")
        kind = ab.element_type(logits)
        out = logits if out is None else out
        if out.dtype != logits.dtype or out.shape != logits.shape or not out.is_contiguous():
            raise ValueError(f"out: contiguous {logits.dtype} of shape {tuple(logits.shape)} expected, not {out.dtype} "
                             f"of shape {tuple(out.shape)}")
        lead = tuple(logits.shape[:-1])
        B, N = lead if len(lead) == 2 else (lead[0], 1)
        rows = lambda t: t.shape[1] if t is not None and t.dim() == 2 else 0  # noqa: E731
        H, M = rows(history), rows(bias_ids)
        G = masks.shape[0] if masks is not None else 0
        ints = dict(tok=(tok, (B, N)), parent=(parent, (B, N)), history=(history, (B, H)),
                    history_len=(history_len, (B,)), prompt_len=(prompt_len, (B,)), bias_ids=(bias_ids, (B, M)),
                    masks=(masks, (G, (V + 31) // 32)), mask_rows=(mask_rows, lead))
        for name, (t, shape) in ints.items():
            if t is not None:
                _check_int32(t, name, shape)
        floats = dict(repetition=(repetition, (B,)), presence=(presence, (B,)), frequency=(frequency, (B,)),
                      bias_values=(bias_values, (B, M)))
        for name, (t, shape) in floats.items():
            if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape):
                raise ValueError(f"{name}: contiguous fp32 of shape {shape} expected, not {t.dtype} of shape "
                                 f"{tuple(t.shape)}")
        for a, b in (("history_len", "history"), ("prompt_len", "history"), ("bias_values", "bias_ids"),
                     ("bias_ids", "bias_values"), ("mask_rows", "masks"), ("masks", "mask_rows")):
            given = {**ints, **floats}
            if given[a][0] is not None and given[b][0] is None:
                raise ValueError(f"{a} without {b}")
        _check_device(self.params.device, logits=logits, out=out, **{n: t for n, (t, _) in {**ints, **floats}.items()})
        rules = ab.logit_rules(history, history_len, prompt_len, H, repetition, presence, frequency, bias_ids,
                               bias_values, M, masks, mask_rows, G)
        ab.logits_adjust(out, logits, kind, rules, tok, parent, B, N, V, Vp, stream)
        return out

    def accept_tree(self, kv, tok, chosen, pos, parent=None, stream=None) -> dict:
        """The path of each tree that agrees with `chosen` (each node's next
        token), its rows of the cache moved together (kv None: no cache): path,
        emitted [B, N], count, next_tok, next_pos [B], which belong to `stream`.
        tok, chosen, parent: contiguous int32 [B, N], pos: int32 [B]."""
        B, N = tok.shape
        for name, t in (("tok", tok), ("chosen", chosen), ("parent", parent)):
            if t is not None:
                _check_int32(t, name, (B, N))
        _check_int32(pos, "pos", (B,))
        _check_device(self.params.device, tok=tok, chosen=chosen, parent=parent, pos=pos)
        with _allocating_on(stream):
            new = lambda *s: torch.empty(s, dtype=torch.int32, device=tok.device)  # noqa: E731
            r = dict(path=new(B, N), count=new(B), emitted=new(B, N), next_tok=new(B), next_pos=new(B))
        ab.gpt2_accept_tree(*r.values(), self.cfg, kv, tok, parent, chosen, pos, B, N, self.precision, stream)
        return r
