"""Cases and plain forms of the serving operators: block tables built on the
GPU, decode attention over a shared prefix, and the log probabilities of given
tokens with entropy and top alternatives (forward and backward).

`run` computes a case in elementary torch operations, or through the
framework's entry points where `own` is set; `exact` computes it from the
definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence's decode step, the alternatives shown to a user
        dict(name="logprobs-one-row", op="logprobs", N=1, V=50257, Vp=50304, K=20, dtype="fp32", masked=0.0),
        # a decode step of the 32-sequence batch: the drawn tokens' log probabilities
        dict(name="logprobs-decode", op="logprobs", N=32, V=50257, Vp=50304, K=5, dtype="fp32", masked=0.0),
        # scoring whole prompts, four sequences of 1024 positions
        dict(name="logprobs-score", op="logprobs", N=4096, V=50257, Vp=50304, K=1, dtype="fp32", masked=0.0),
        # an odd number of rows and tokens, most tokens ruled out by a grammar, many alternatives
        dict(name="logprobs-masked", op="logprobs", N=777, V=32003, Vp=32008, K=32, dtype="bf16", masked=0.7),
        # the gradient of a policy's log probabilities and entropy over a large batch
        dict(name="logprobs-grad", op="logprobs_grad", N=4096, V=50257, Vp=50304, dtype="fp32", masked=0.0),
        # the same over few rows of 16-bit logits
        dict(name="logprobs-grad-small", op="logprobs_grad", N=100, V=50257, Vp=50304, dtype="bf16", masked=0.3),
        # one decode step of 32 sequences: a block for those that cross a border
        dict(name="tables-decode", op="tables", B=32, T=1, block=16, cached=1000, prefix=0),
        # admission of 256 requests of up to 1024 new positions behind a shared prompt
        dict(name="tables-admit", op="tables", B=256, T=1024, block=16, cached=512, prefix=512),
        # four continuations of a short prompt
        dict(name="shared-few", op="attention", B=4, NH=12, hs=64, P=256, own_max=16, block=16, dtype="fp16"),
        # the decode batch, a prompt of most of the context
        dict(name="shared-decode", op="attention", B=32, NH=12, hs=64, P=960, own_max=63, block=16, dtype="fp16"),
        # many continuations of a very long prompt
        dict(name="shared-long", op="attention", B=256, NH=16, hs=64, P=16384, own_max=255, block=64, dtype="bf16"),
        # fp32 cache, a head of 32 dimensions, odd sizes: the prefix ends inside a block
        dict(name="shared-fp32", op="attention", B=24, NH=8, hs=32, P=2001, own_max=100, block=32, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "tables", "attention"])
    if op in ("logprobs", "logprobs_grad"):
        N, V = _log(rng, 1, 4096), _log(rng, 1000, 50257)
        case = dict(op=op, N=N, V=V, Vp=(V + rng.randint(0, 40) + 7) // 8 * 8, dtype=rng.choice(sorted(DTYPES)),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.9]))
        if op == "logprobs":
            case["K"] = rng.randint(0, 32)
        return case
    if op == "tables":
        block = rng.choice([8, 16, 32, 64])
        B = _log(rng, 1, 1024)
        T = rng.choice([1, _log(rng, 1, min(1024, (256 * 1024) // B))])
        return dict(op=op, B=B, T=T, block=block, cached=_log(rng, 64, 4096), prefix=block * rng.choice([0, 0, 4]))
    B, P = _log(rng, 1, 256), _log(rng, 64, 16384)
    own_max = _log(rng, 1, 255)
    block = rng.choice([b for b in (8, 16, 32, 64, 128) if (P + own_max) // b + 1 <= 1024])
    dtype = rng.choice(sorted(DTYPES))
    return dict(op=op, B=B, NH=rng.choice([4, 8, 12, 16]), hs=rng.choice([16, 32, 64, 64]), P=P, own_max=own_max,
                block=block, dtype=dtype)


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    dev = dict(device="cuda")
    if case["op"] in ("logprobs", "logprobs_grad"):
        N, V, Vp = case["N"], case["V"], case["Vp"]
        x = torch.randn(N, Vp, generator=g, **dev) * 2.5 - 1.0
        if case["masked"]:
            x.masked_fill_(torch.rand(N, Vp, generator=g, **dev) < case["masked"], -math.inf)
        logits = x.to(DTYPES[case["dtype"]])
        del x
        targets = torch.randint(0, V, (N,), generator=g, dtype=torch.int32, **dev)
        targets[torch.rand(N, generator=g, **dev) < 0.05] = -1  # padding positions
        s = dict(case=case, logits=logits, targets=targets)
        if case["op"] == "logprobs_grad":
            # what the forward pass kept, and the loss's gradients
            z = logits[:, :V].float()
            lse = torch.logsumexp(z, 1)
            z = z - lse[:, None]
            s["lse"], s["entropy"] = lse, -(z.exp() * z.clamp(min=-1e4)).sum(1)
            s["dlogprob"] = torch.randn(N, generator=g, **dev)
            s["dentropy"] = torch.randn(N, generator=g, **dev) * 0.01
        return s
    if case["op"] == "tables":
        B, T, bs, prefix = case["B"], case["T"], case["block"], case["prefix"]
        cached = prefix + torch.randint(0, max(1, case["cached"] - prefix), (B,), generator=g, dtype=torch.int32, **dev)
        new = torch.randint(1, T + 1, (B,), generator=g, dtype=torch.int32, **dev)
        max_blocks = (max(case["cached"], prefix + 1) + T) // bs + 1
        num_blocks = B * max_blocks + prefix // bs + 16
        ids = torch.randperm(num_blocks, generator=g, **dev).to(torch.int32)
        held = B * ((max(case["cached"], prefix + 1) + bs - 1) // bs)  # blocks the requests hold already
        table = torch.full((B, max_blocks), -1, dtype=torch.int32, **dev)
        table[:, :held // B] = ids[:held].view(B, -1)
        pre = ids[held:held + prefix // bs].contiguous()
        table[:, :prefix // bs] = pre
        free = ids[held + prefix // bs:].contiguous()
        return dict(case=case, table=table, cached=cached, new=new, free=free, prefix_blocks=pre if prefix else None,
                    taken=torch.full((1,), 3, dtype=torch.int32, **dev), num_blocks=num_blocks)
    B, NH, hs, P, bs = case["B"], case["NH"], case["hs"], case["P"], case["block"]
    dtype = DTYPES[case["dtype"]]
    own_blocks = (P + case["own_max"]) // bs + 1 - P // bs
    num_blocks = P // bs + B * own_blocks + 5
    ids = torch.randperm(num_blocks, generator=g, **dev).to(torch.int32)
    table = torch.empty(B, P // bs + own_blocks, dtype=torch.int32, **dev)
    table[:, :P // bs] = ids[:P // bs]
    table[:, P // bs:] = ids[P // bs:P // bs + B * own_blocks].view(B, own_blocks)
    pool = torch.randn(2, num_blocks, NH, bs, hs, generator=g, **dev).to(dtype)
    if P % bs:  # the prefix's last positions: a copy of them in each sequence's own block
        own_rows = table[:, P // bs].long()
        pool[:, own_rows, :, :P % bs] = pool[:, own_rows[:1], :, :P % bs]
    pos = (P + torch.randint(0, case["own_max"] + 1, (B,), generator=g, **dev)).to(torch.int32)
    qkv = torch.randn(B, 3 * NH * hs, generator=g, **dev)
    qkv[:, :NH * hs] *= 2.0
    return dict(case=case, pool=pool, table=table, pos=pos, qkv=qkv.to(dtype), num_blocks=num_blocks)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _plain_logprobs(s):
    V, K = s["case"]["V"], s["case"]["K"]
    x = s["logits"][:, :V].float()
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    some = z[:, 0] > 0
    lse = m + torch.log(z)
    logp = x - lse
    entropy = torch.where(some, -torch.where(e > 0, e / z * logp, torch.zeros_like(e)).sum(1), torch.zeros_like(z[:, 0]))
    t = s["targets"].long()
    lp = logp.gather(1, t.clamp(min=0)[:, None])[:, 0]
    lp = torch.where(t < 0, torch.zeros_like(lp), torch.where(some, lp, torch.full_like(lp, -math.inf)))
    out = dict(logprob=lp, entropy=entropy, lse=lse[:, 0])
    if K:
        # one 64-bit key orders by value, then by the lowest token id
        b = (x + 0.0).view(torch.int32).long()
        key = torch.where(b >= 0, b, b ^ 0x7FFFFFFF) * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device=x.device))
        ids = 0xFFFFFFFF - (torch.topk(key, K, dim=1).values & 0xFFFFFFFF)
        top = x.gather(1, ids)
        none = top == -math.inf
        out["top_ids"] = torch.where(none, torch.full_like(ids, -1), ids).int()
        out["top_logprobs"] = torch.where(none, top, top - lse)
    return out


def _plain_logprobs_grad(s):
    V, Vp = s["case"]["V"], s["case"]["Vp"]
    x = s["logits"][:, :V].float()
    t = s["targets"].long()
    g = torch.where(t < 0, torch.zeros_like(s["dlogprob"]), s["dlogprob"])[:, None]
    h = s["dentropy"][:, None]
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    d = torch.where(p > 0, -p * (g + h * (logp + s["entropy"][:, None])), torch.zeros_like(p))
    d.scatter_add_(1, t.clamp(min=0)[:, None], g)
    out = torch.zeros_like(s["logits"])
    out[:, :V] = d.to(out.dtype)
    return dict(dlogits=out)


def _plain_tables(s):
    c = s["case"]
    bs, T, prefix = c["block"], c["T"], c["prefix"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"].long()
    have, need = (cached + bs - 1) // bs, (cached + new + bs - 1) // bs
    want = need - have
    incl = torch.cumsum(want, 0)
    ok = (want == 0) | (incl <= s["free"].numel() - s["taken"].long())
    j = torch.arange(table.shape[1], device=table.device)
    at = s["taken"].long() + (incl - want)[:, None] + j - have[:, None]
    fresh = ok[:, None] & (j >= have[:, None]) & (j < need[:, None])
    table = torch.where(fresh, s["free"].long()[at.clamp(0, s["free"].numel() - 1)], table)
    if prefix:
        table[:, :prefix // bs] = torch.where(ok[:, None], s["prefix_blocks"].long(), table[:, :prefix // bs])
    p = cached[:, None] + torch.arange(T, device=table.device)
    slot = table.gather(1, (p // bs).clamp(max=table.shape[1] - 1)) * bs + p % bs
    slot = torch.where(ok[:, None] & (p < (cached + new)[:, None]), slot, torch.full_like(slot, -1))
    s["table"].copy_(table)
    return dict(table=s["table"], slots=slot.int(), next_len=torch.where(ok, cached + new, cached).int(),
                taken=(s["taken"] + (want * ok).sum()).int())


def _plain_attention(s):
    c = s["case"]
    B, NH, hs, P, bs, own_max = c["B"], c["NH"], c["hs"], c["P"], c["block"], c["own_max"]
    pool, table, pos = s["pool"], s["table"].long(), s["pos"].long()
    q, k, v = (t.view(B, NH, hs) for t in s["qkv"].split(NH * hs, 1))
    blk, off = table.gather(1, (pos // bs)[:, None])[:, 0], pos % bs
    pool[0, blk, :, off] = k
    pool[1, blk, :, off] = v
    n = (P + bs - 1) // bs
    pre = pool[:, table[0, :n]].permute(0, 2, 1, 3, 4).reshape(2, NH, n * bs, hs)[:, :, :P].float()
    scale = 1.0 / math.sqrt(hs)
    sp = torch.matmul(q.float().transpose(0, 1), pre[0].transpose(1, 2)).transpose(0, 1) * scale  # [B, NH, P]
    j = P + torch.arange(own_max + 1, device=pos.device)
    jb = table[:, (j // bs).clamp(max=table.shape[1] - 1)]
    mine = pool[:, jb, :, (j % bs).expand(B, -1)].float()  # [B, own, 2, NH, hs]
    so = (q.float()[:, None] * mine[:, :, 0]).sum(-1).transpose(1, 2) * scale  # [B, NH, own]
    so = so.masked_fill((j[None] > pos[:, None])[:, None], -math.inf)
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    ep, eo = torch.exp(sp - m), torch.exp(so - m)
    o = torch.matmul(ep.transpose(0, 1), pre[1]).transpose(0, 1) + (eo.transpose(1, 2)[..., None] * mine[:, :, 1]).sum(1)
    o = o / (ep.sum(-1) + eo.sum(-1))[..., None]
    return dict(out=o.reshape(B, NH * hs).to(pool.dtype), pool=pool)


_plain = dict(logprobs=_plain_logprobs, logprobs_grad=_plain_logprobs_grad, tables=_plain_tables,
              attention=_plain_attention)


# ----------------------------------------- the framework's calls (own = True)
def _kept(s, name, make):
    """A buffer that a program keeps beside its inputs, made at its first use."""
    if name not in s:
        s[name] = make()
    return s[name]


def _binding():
    from gpt_transformer_forward_gb300 import binding
    return binding


def _own_logprobs(s):
    ab, c = _binding(), s["case"]
    N, K = c["N"], c["K"]

    def buffers():
        f = [torch.empty(N, device="cuda") for _ in range(3)]
        return f + ([torch.empty(N, K, dtype=torch.int32, device="cuda"), torch.empty(N, K, device="cuda")] if K
                    else [None, None])

    lp, ent, lse, ids, top = _kept(s, "outputs", buffers)
    ab.logprobs_forward(lp, ent, lse, ids, top, s["logits"], ab.element_type(s["logits"]), s["targets"], N, c["V"],
                        c["Vp"], K)
    out = dict(logprob=lp, entropy=ent, lse=lse)
    if K:
        out.update(top_ids=ids, top_logprobs=top)
    return out


def _own_logprobs_grad(s):
    ab, c = _binding(), s["case"]
    d = _kept(s, "dlogits", lambda: torch.empty_like(s["logits"]))
    ab.logprobs_backward(d, s["logits"], ab.element_type(s["logits"]), s["targets"], s["lse"], s["entropy"],
                         s["dlogprob"], s["dentropy"], c["N"], c["V"], c["Vp"])
    return dict(dlogits=d)


def _own_tables(s):
    ab, c = _binding(), s["case"]
    slots, next_len, taken = _kept(s, "outputs", lambda: [
        torch.empty(c["B"], c["T"], dtype=torch.int32, device="cuda"),
        torch.empty(c["B"], dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")])
    ab.paged_build_tables(s["table"], slots, next_len, taken, s["cached"], s["new"], s["free"], s["free"].numel(),
                          s["taken"], s["prefix_blocks"], c["prefix"], c["B"], c["T"], s["num_blocks"], c["block"],
                          s["table"].shape[1])
    return dict(table=s["table"], slots=slots, next_len=next_len, taken=taken)


def _own_attention(s):
    ab, c = _binding(), s["case"]
    B, NH, C = c["B"], c["NH"], c["NH"] * c["hs"]
    precision = ab.PRECISIONS[c["dtype"]]
    kv = ab.paged_kv(s["pool"], s["table"], s["num_blocks"], c["block"], s["table"].shape[1])
    nbytes = ab.attention_shared_prefix_workspace_size(B, C, NH, c["P"], precision)
    ws = _kept(s, "workspace", lambda: torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda"))
    out = _kept(s, "out", lambda: torch.empty(B, C, dtype=s["pool"].dtype, device="cuda"))
    ab.attention_shared_prefix(out, s["qkv"], kv, s["pos"], B, C, NH, c["P"], precision, ws, nbytes)
    return dict(out=out, pool=s["pool"])


_own = dict(logprobs=_own_logprobs, logprobs_grad=_own_logprobs_grad, tables=_own_tables, attention=_own_attention)


# ------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "logprobs":
        e = DTYPES[case["dtype"]].itemsize
        n = case["N"]
        return {"bytes": n * (case["V"] * e + 16 + 8 * case["K"]), "flops": 5 * n * case["V"]}
    if case["op"] == "logprobs_grad":
        e = DTYPES[case["dtype"]].itemsize
        n = case["N"]
        return {"bytes": n * ((case["V"] + case["Vp"]) * e + 20), "flops": 6 * n * case["V"]}
    if case["op"] == "tables":
        B, T, bs = case["B"], case["T"], case["block"]
        fresh = B * (T + 1) // 2 // bs + B * case["prefix"] // bs  # block ids read and written
        return {"bytes": 4 * (B * T + 3 * B + 2 * fresh), "flops": 0}
    e = DTYPES[case["dtype"]].itemsize
    B, NH, hs, P = case["B"], case["NH"], case["hs"], case["P"]
    mine = B * case["own_max"] / 2  # own cached positions, in the mean
    return {"bytes": NH * hs * e * (2 * P + 2 * mine + 6 * B), "flops": 4 * NH * hs * (B * P + mine + B)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    if case["op"] == "attention":
        B, NH, hs, P, bs = case["B"], case["NH"], case["hs"], case["P"], case["block"]
        flat = s["pool"].transpose(2, 3).reshape(2, -1, NH, hs)  # a row for each slot
        out = torch.empty(B, NH * hs, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["pos"][b])
            p = torch.arange(n, device="cuda")
            row = s["table"][b].long()[p // bs] * bs + p % bs
            q, k1, v1 = s["qkv"][b].double().view(3, NH, hs)
            k, v = torch.cat([flat[0, row].double(), k1[None]]), torch.cat([flat[1, row].double(), v1[None]])
            w = torch.softmax(torch.einsum("hd,jhd->hj", q, k) / hs ** 0.5, dim=1)
            out[b] = torch.einsum("hj,jhd->hd", w, v).reshape(-1)
        return dict(out=out, pool=None)
    x = s["logits"][:, :case["V"]].double()
    if case["op"] == "logprobs":
        logp = torch.log_softmax(x, 1)
        p = logp.exp()
        t = s["targets"].long()
        lp = logp[torch.arange(case["N"], device="cuda"), t.clamp(min=0)].masked_fill(t < 0, 0.0)
        out = dict(logprob=lp, entropy=torch.special.entr(p).sum(1), lse=torch.logsumexp(x, 1))
        if case["K"]:
            out.update(top_ids=None, top_logprobs=torch.topk(logp, case["K"], dim=1).values)
        return out
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    ent = torch.special.entr(p).sum(1, keepdim=True)
    t = s["targets"].long()
    g = s["dlogprob"].double().masked_fill(t < 0, 0.0)[:, None]
    d = -g * p - s["dentropy"].double()[:, None] * (p * ent - torch.special.entr(p))
    rows = torch.arange(case["N"], device="cuda")
    d[rows, t.clamp(min=0)] += g[:, 0]
    full = torch.zeros(case["N"], case["Vp"], dtype=torch.float64, device="cuda")
    full[:, :case["V"]] = d
    return dict(dlogits=full)
