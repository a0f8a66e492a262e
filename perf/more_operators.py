"""Cases and plain forms of the operators that verify drafted tokens: attention
of a tree of drafted tokens over a paged cache, penalties with biases and
grammar masks on logits, and the acceptance of a tree's path with its cache rows
moved together.

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
        # one user's sequence, four tokens in a row from a draft model behind the last one
        dict(name="tree-one", op="attention", B=1, N=5, tree="chain", NH=12, hs=64, cached=1000, block=16, dtype="fp16"),
        # the decode batch of 32 sequences, trees of 16 nodes
        dict(name="tree-decode", op="attention", B=32, N=16, tree="random", NH=12, hs=64, cached=960, block=16,
             dtype="fp16"),
        # long documents, the largest trees
        dict(name="tree-long", op="attention", B=16, N=64, tree="random", NH=16, hs=64, cached=16384, block=64,
             dtype="bf16"),
        # fp32 cache, a head of 32 dimensions, odd sizes
        dict(name="tree-fp32", op="attention", B=6, N=23, tree="random", NH=8, hs=32, cached=2001, block=32,
             dtype="fp32"),
        # one user's next token: penalties over the conversation, a few biases, a grammar
        dict(name="adjust-one", op="adjust", B=1, N=1, tree="chain", V=50257, Vp=50304, H=200, M=20, masks=1,
             dtype="fp32"),
        # the decode batch's trees: penalties alone
        dict(name="adjust-tree", op="adjust", B=32, N=16, tree="random", V=50257, Vp=50304, H=1000, M=0, masks=0,
             dtype="fp32"),
        # an odd number of sequences and tokens, one token each, all under grammars
        dict(name="adjust-grammar", op="adjust", B=777, N=1, tree="chain", V=32003, Vp=32008, H=333, M=7, masks=40,
             dtype="bf16"),
        # many sequences with the largest trees, everything on
        dict(name="adjust-large", op="adjust", B=64, N=64, tree="random", V=50257, Vp=50304, H=1024, M=50, masks=64,
             dtype="fp32"),
        # the end of one user's step
        dict(name="accept-one", op="accept", B=1, N=5, tree="chain", L=12, NH=12, hs=64, block=16, dtype="fp16"),
        # the end of a large batch's step
        dict(name="accept-batch", op="accept", B=64, N=64, tree="random", L=24, NH=16, hs=64, block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "adjust", "adjust", "accept"])
    N = _log(rng, 1, 64)
    case = dict(op=op, N=N, tree=rng.choice(["chain", "random", "random", "wide"]), dtype=rng.choice(sorted(DTYPES)))
    if op == "attention":
        NH, cached = rng.choice([4, 8, 12, 16]), _log(rng, 16, 16384)
        B = _log(rng, 1, max(1, min(256, (16 * 16 * 16384) // (NH * cached), (16 * 16 * 16384 * 64) // (NH * cached * N))))
        if case["dtype"] == "fp32":
            B = max(1, B // 4)
        block = rng.choice([b for b in (1, 8, 16, 32, 64, 128) if (cached + N) // b + 1 <= 1024])
        return dict(case, B=B, NH=NH, hs=rng.choice([16, 32, 64, 64]), cached=cached, block=block)
    if op == "adjust":
        V = _log(rng, 1000, 50257)
        return dict(case, B=_log(rng, 1, max(1, 4096 // N)), V=V, Vp=(V + rng.randint(0, 40) + 7) // 8 * 8,
                    H=_log(rng, 1, 4000), M=rng.choice([0, 0, 1, 17, 200]), masks=rng.choice([0, 0, 1, 13]))
    return dict(case, B=_log(rng, 1, 64), L=rng.choice([6, 12, 24]), NH=rng.choice([4, 12, 16]),
                hs=rng.choice([16, 32, 64]), block=rng.choice([8, 16, 32]))


# ----------------------------------------------------------------- the inputs
def _trees(case, g):
    """parent [B, N]: node 0 the last known token, some trees with fewer nodes
    than N (-2 behind them)."""
    B, N = case["B"], case["N"]
    i = torch.arange(N, device="cuda")
    if case["tree"] == "chain":
        parent = (i - 1).expand(B, N).clone()
    else:
        r = torch.rand(B, N, generator=g, device="cuda")
        if case["tree"] == "wide":
            r = r * r * r  # most children near the root
        parent = torch.minimum((r * i).long(), i - 1)
    nodes = torch.where(torch.rand(B, generator=g, device="cuda") < 0.25,
                        torch.randint(1, N + 1, (B,), generator=g, device="cuda"), N)
    nodes[0] = N
    return torch.where(i < nodes[:, None], parent, torch.full_like(parent, -2)).int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(generator=g, device="cuda")
    B, N = case["B"], case["N"]
    parent = _trees(case, g)
    if case["op"] == "adjust":
        V, Vp, H, M = case["V"], case["Vp"], case["H"], case["M"]
        logits = (torch.randn(B * N, Vp, **dev) * 2.5 - 1.0).to(DTYPES[case["dtype"]])
        # a text repeats few tokens often
        text = lambda *shape: (torch.rand(*shape, **dev) ** 4 * V).int().clamp(max=V - 1)  # noqa: E731
        s = dict(case=case, parent=parent, logits=logits, tok=text(B, N), history=text(B, H),
                 history_len=torch.randint((H + 1) // 2, H + 1, (B,), dtype=torch.int32, **dev),
                 repetition=1.0 + torch.rand(B, **dev) * 0.3, presence=torch.rand(B, **dev),
                 frequency=torch.rand(B, **dev) * 0.5)
        s["prompt_len"] = (s["history_len"] * torch.rand(B, **dev)).int()
        if M:  # distinct tokens, a few places unused
            ids = torch.rand(B, V, **dev).topk(M, dim=1).indices.int()
            s["bias_ids"] = torch.where(torch.rand(B, M, **dev) < 0.1, torch.full_like(ids, -1), ids).contiguous()
            s["bias_values"] = torch.randn(B, M, **dev) * 4
        if case["masks"]:  # 32 tokens a word, a grammar leaves some tokens here and there
            words = (V + 31) // 32
            r = torch.randint(-2**31, 2**31, (2, case["masks"], words), dtype=torch.int64, **dev)
            s["masks"] = (r[0] & r[1]).int()
            s["masks"][0, words // 3:] = 0  # one that rules most out
            s["mask_rows"] = torch.randint(-1, case["masks"], (B * N,), dtype=torch.int32, **dev)
        return s
    bs, NH, hs, dtype = case["block"], case["NH"], case["hs"], DTYPES[case["dtype"]]
    if case["op"] == "attention":
        cached = case["cached"]
        pos = torch.randint(cached // 4, cached + 1, (B,), dtype=torch.int32, **dev)
        if B >= 8:
            pos[torch.rand(B, **dev) < 0.05] = -1  # sequences that wait in this step
        row = (cached + N) // bs + 1
        num_blocks = B * row + 5
        table = torch.randperm(num_blocks, **dev)[:B * row].int().view(B, row).contiguous()
        pool = torch.randn(2, num_blocks, NH, bs, hs, **dev).to(dtype)
        qkv = torch.randn(B * N, 3 * NH * hs, **dev)
        qkv[:, :NH * hs] *= 2.0
        return dict(case=case, parent=parent, pos=pos, table=table, pool=pool, qkv=qkv.to(dtype), num_blocks=num_blocks)
    # the blocks that hold the drafted tokens; what lies before is not touched
    pos = torch.randint(0, 200, (B,), dtype=torch.int32, **dev)
    row, mine = (200 + N) // bs + 1, (bs - 1 + N) // bs + 1
    num_blocks = B * mine + 3
    ids = torch.randperm(num_blocks, **dev)[:B * mine].int().view(B, mine)
    at = torch.arange(row, device="cuda") - pos[:, None] // bs
    table = torch.where((at >= 0) & (at < mine), ids.gather(1, at.clamp(0, mine - 1)), torch.full_like(at, -1).int())
    pool = torch.randn(case["L"], 2, num_blocks, NH, bs, hs, **dev).to(dtype)
    tok = torch.randint(0, 50257, (B, N), dtype=torch.int32, **dev)
    # the model agrees with one of a node's children in most cases
    pick = (torch.randint(0, 1 << 20, (B, N), **dev) << 6) + torch.arange(N, device="cuda")
    pick = torch.where(parent >= 0, pick, torch.full_like(pick, -1))
    child = torch.full((B, N), -1, device="cuda").scatter_reduce_(1, parent.long().clamp(min=0), pick, "amax")
    agree = (child >= 0) & (torch.rand(B, N, **dev) < 0.8)
    chosen = torch.where(agree, tok.gather(1, child.clamp(min=0) & 63),
                         torch.randint(0, 50257, (B, N), dtype=torch.int32, **dev))
    return dict(case=case, parent=parent, pos=pos, table=table.contiguous(), pool=pool, tok=tok, chosen=chosen.contiguous(),
                num_blocks=num_blocks)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _ancestors(parent):
    """[B, N, N]: node i's row holds the nodes on its path, itself among them."""
    B, N = parent.shape
    p = parent.long()
    up = torch.zeros(B, N, N + 1, device=p.device).scatter_(2, torch.where(p < 0, N, p)[:, :, None], 1.0)[:, :, :N]
    m = (up + torch.eye(N, device=p.device)).clamp(max=1)
    m = (m @ m).clamp(max=1)  # paths of up to 2, 4, .. 64 steps
    m = (m @ m).clamp(max=1)
    m = (m @ m).clamp(max=1)
    m = (m @ m).clamp(max=1)
    m = (m @ m).clamp(max=1)
    m = (m @ m).clamp(max=1)
    return (m > 0) & (p >= -1)[:, :, None]


def _plain_attention(s):
    c = s["case"]
    B, N, NH, hs, bs = c["B"], c["N"], c["NH"], c["hs"], c["block"]
    pool, table, pos = s["pool"], s["table"].long(), s["pos"].long()
    anc = _ancestors(s["parent"]) & (pos >= 0)[:, None, None]
    node = (s["parent"] >= -1) & (pos >= 0)[:, None]
    q, k, v = (t.reshape(B, N, NH, hs) for t in s["qkv"].split(NH * hs, 1))
    # the drafted tokens' keys and values go to positions pos + i
    at = (pos.clamp(min=0)[:, None] + torch.arange(N, device=pos.device))
    blk, off = table.gather(1, at // bs)[node], (at % bs)[node]
    pool[0, blk, :, off] = k[node]
    pool[1, blk, :, off] = v[node]
    j = torch.arange(c["cached"], device=pos.device)
    cached = pool[:, table[:, j // bs], :, j % bs].float()  # [B, L, 2, NH, hs]
    kk = torch.cat([cached[:, :, 0].transpose(1, 2), k.float().transpose(1, 2)], 2)  # [B, NH, L + N, hs]
    vv = torch.cat([cached[:, :, 1].transpose(1, 2), v.float().transpose(1, 2)], 2)
    seen = torch.cat([(j < pos[:, None])[:, None].expand(B, N, -1) & node[:, :, None], anc], 2)[:, None]
    sc = torch.matmul(q.float().transpose(1, 2), kk.transpose(2, 3)) / math.sqrt(hs)
    sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(3, keepdim=True)
    e = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(3, keepdim=True)
    o = torch.matmul(e, vv) / torch.where(z > 0, z, torch.ones_like(z))
    return dict(out=o.transpose(1, 2).reshape(B * N, NH * hs).to(pool.dtype), pool=pool)


def _plain_adjust(s):
    c = s["case"]
    B, N, V, H = c["B"], c["N"], c["V"], c["H"]
    x = s["logits"][:, :V].float().view(B, N, V)
    anc = _ancestors(s["parent"])
    t = torch.arange(H, device=x.device)
    said = (t < s["history_len"][:, None]) & (t >= s["prompt_len"][:, None])
    asked = t < s["prompt_len"][:, None]
    hist = s["history"].long()
    count = torch.zeros(B, V, device=x.device).scatter_add_(1, hist, said.float())
    prompt = torch.zeros(B, V, device=x.device).scatter_add_(1, hist, asked.float())
    count = count[:, None].repeat(1, N, 1)
    count.scatter_add_(2, s["tok"].long()[:, None].expand(B, N, N), anc.float())
    rep = s["repetition"][:, None, None]
    x = torch.where((count > 0) | (prompt > 0)[:, None], torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None, None] * count - torch.where(count > 0, s["presence"][:, None, None], 0.0)
    if c["M"]:
        ids = s["bias_ids"].long()
        bias = torch.zeros(B, V + 1, device=x.device).scatter_(1, torch.where(ids < 0, V, ids), s["bias_values"])
        x = x + bias[:, None, :V]
    x = x.reshape(B * N, V)
    if c["masks"]:
        v = torch.arange(V, device=x.device)
        allowed = (s["masks"][:, v // 32] >> (v % 32)) & 1
        rows = s["mask_rows"].long()
        x = torch.where((allowed[rows.clamp(min=0)] == 1) | (rows < 0)[:, None], x, torch.full_like(x, -math.inf))
    node = (s["parent"] >= -1).view(-1)
    out = torch.full_like(s["logits"], -math.inf)
    out[:, :V] = x.to(out.dtype)
    return dict(out=torch.where(node[:, None], out, torch.zeros_like(out)))


def _plain_accept(s):
    c = s["case"]
    B, N, bs = c["B"], c["N"], c["block"]
    parent, tok, chosen, pos, table = (s[k].long() for k in ("parent", "tok", "chosen", "pos", "table"))
    i = torch.arange(N, device=pos.device)
    match = (parent >= 0) & (tok == chosen.gather(1, parent.clamp(min=0)))
    twin = match[:, None] & match[:, :, None] & (parent[:, None] == parent[:, :, None]) & (i[None] < i[:, None])
    good = (match & ~twin.any(2)) | (i == 0)
    anc = _ancestors(s["parent"])
    good = ~(anc & ~good[:, None]).any(2) & (parent >= -1)
    depth = anc.sum(2) - 1
    path = torch.full((B, N + 1), -1, device=pos.device)
    path.scatter_(1, torch.where(good, depth, N), i.expand(B, N))
    path = path[:, :N]
    count = good.sum(1)
    last = chosen.gather(1, path.gather(1, (count - 1)[:, None]))[:, 0]
    after = torch.cat([path[:, 1:], torch.full_like(path[:, :1], -1)], 1)
    emitted = torch.where(after >= 0, tok.gather(1, after.clamp(min=0)), torch.full_like(path, -1))
    emitted = torch.where(i == (count - 1)[:, None], last[:, None], emitted)
    # the path's rows to positions pos + 0, 1, ..
    pool, taken = s["pool"], path >= 0
    src, dst = (pos[:, None] + path)[taken], (pos[:, None] + i)[taken]
    row = torch.arange(B, device=pos.device)[:, None].expand(B, N)[taken]
    moved = pool[:, :, table[row, src // bs], :, src % bs]
    pool[:, :, table[row, dst // bs], :, dst % bs] = moved
    return dict(path=path.int(), count=count.int(), emitted=emitted.int(), next_tok=last.int(),
                next_pos=(pos + count).int(), pool=pool)


_plain = dict(attention=_plain_attention, adjust=_plain_adjust, accept=_plain_accept)


# ----------------------------------------- the framework's calls (own = True)
def _kept(s, name, make):
    """A buffer that a program keeps beside its inputs, made at its first use."""
    if name not in s:
        s[name] = make()
    return s[name]


def _binding():
    from gpt_transformer_forward_gb300 import binding
    return binding


def _kv(s):
    ab, c = _binding(), s["case"]
    return _kept(s, "kv", lambda: ab.paged_kv(s["pool"], s["table"], s["num_blocks"], c["block"], s["table"].shape[1]))


def _own_attention(s):
    ab, c = _binding(), s["case"]
    B, N, NH, C = c["B"], c["N"], c["NH"], c["NH"] * c["hs"]
    precision = ab.PRECISIONS[c["dtype"]]
    nbytes = _kept(s, "ws_bytes", lambda: ab.attention_tree_workspace_size(B, N, C, NH, precision))
    ws = _kept(s, "workspace", lambda: torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda"))
    out = _kept(s, "out", lambda: torch.empty(B * N, C, dtype=s["pool"].dtype, device="cuda"))
    ab.attention_tree(out, s["qkv"], _kv(s), s["pos"], s["parent"], B, N, C, NH, precision, ws, nbytes)
    return dict(out=out, pool=s["pool"])


def _own_adjust(s):
    ab, c = _binding(), s["case"]
    # rows of places without a node are left as they are
    out = _kept(s, "out", lambda: torch.zeros_like(s["logits"]))
    rules = _kept(s, "rules", lambda: ab.logit_rules(
        history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"], history_stride=c["H"],
        repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_ids=s.get("bias_ids"),
        bias_values=s.get("bias_values"), num_bias=c["M"], masks=s.get("masks"), mask_rows=s.get("mask_rows"),
        num_masks=c["masks"]))
    ab.logits_adjust(out, s["logits"], ab.element_type(s["logits"]), rules, s["tok"], s["parent"], c["B"], c["N"],
                     c["V"], c["Vp"])
    return dict(out=out)


def _own_accept(s):
    ab, c = _binding(), s["case"]
    B, N = c["B"], c["N"]
    path, emitted, count, tok, pos = _kept(s, "outputs", lambda: [
        torch.empty(*shape, dtype=torch.int32, device="cuda") for shape in ((B, N), (B, N), (B,), (B,), (B,))])
    cfg = _kept(s, "cfg", lambda: ab.GPT2Config(1024, 50257, 50304, c["L"], c["NH"], c["NH"] * c["hs"]))
    ab.gpt2_accept_tree(path, count, emitted, tok, pos, cfg, _kv(s), s["tok"], s["parent"], s["chosen"], s["pos"], B, N,
                        ab.PRECISIONS[c["dtype"]])
    return dict(path=path, count=count, emitted=emitted, next_tok=tok, next_pos=pos, pool=s["pool"])


_own = dict(attention=_own_attention, adjust=_own_adjust, accept=_own_accept)


# ------------------------------------------------------- work and exact values
def work(case):
    e = DTYPES[case["dtype"]].itemsize
    B, N = case["B"], case["N"]
    if case["op"] == "attention":
        C, n = case["NH"] * case["hs"], case["cached"] * 5 / 8  # cached positions, in the mean
        return {"bytes": C * e * B * (2 * n + 6 * N), "flops": 4 * C * B * N * (n + (N + 1) / 2)}
    if case["op"] == "adjust":
        V = case["V"]
        mask = (V + 31) // 32 * 4 * min(case["masks"], B * N)
        return {"bytes": B * N * e * (V + case["Vp"]) + mask + B * (3 * case["H"] + 8 * case["M"] + 8 * N + 20),
                "flops": 0}
    depth = 3 if case["tree"] != "chain" else (N + 1) / 2  # about what is accepted
    moved = 0 if case["tree"] == "chain" else min(depth, N - 1) / 2
    return {"bytes": B * (12 * N + 8 * N + 12 + 2 * 2 * moved * case["L"] * case["NH"] * case["hs"] * e), "flops": 0}


def exact(case, seed):
    def _path(parent, i):
        nodes = []
        while i >= 0:
            nodes.append(i)
            i = parent[i]
        return nodes

    s = prepare(case, seed)
    B, N = case["B"], case["N"]
    parent = s["parent"].tolist()
    if case["op"] == "attention":
        NH, hs, bs = case["NH"], case["hs"], case["block"]
        flat = s["pool"].transpose(2, 3).reshape(2, -1, NH, hs)  # a row for each slot
        out = torch.zeros(B, N, NH, hs, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["pos"][b])
            if n < 0:
                continue
            p = torch.arange(n, device="cuda")
            row = s["table"][b].long()[p // bs] * bs + p % bs
            q, k1, v1 = s["qkv"].view(B, N, 3, NH, hs)[b].double().unbind(1)
            k, v = torch.cat([flat[0, row].double(), k1]), torch.cat([flat[1, row].double(), v1])
            hide = torch.full((N, n + N), -math.inf, dtype=torch.float64)
            live = [i for i in range(N) if parent[b][i] >= -1]
            for i in live:
                hide[i, :n] = 0
                hide[i, [n + a for a in _path(parent[b], i)]] = 0
            hide = hide.cuda()[live]
            w = torch.softmax(torch.einsum("ihd,jhd->hij", q[live], k) / hs ** 0.5 + hide, dim=2)
            out[b, live] = torch.einsum("hij,jhd->ihd", w, v)
        return dict(out=out.view(B * N, NH * hs), pool=None)
    if case["op"] == "adjust":
        V = case["V"]
        out = torch.zeros(B * N, case["Vp"], dtype=torch.float64)
        x = s["logits"][:, :V].double().cpu()
        hist, tok = s["history"].long().cpu(), s["tok"].tolist()
        v = torch.arange(V)
        allowed = ((s["masks"].cpu()[:, v // 32] >> (v % 32)) & 1).bool() if case["masks"] else None
        for b in range(B):
            n, m = int(s["history_len"][b]), int(s["prompt_len"][b])
            said, asked = torch.bincount(hist[b, m:n], minlength=V), torch.bincount(hist[b, :m], minlength=V)
            r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
            for i in range(N):
                if parent[b][i] < -1:
                    continue
                mine = said.clone()
                for a in _path(parent[b], i):
                    mine[tok[b][a]] += 1
                y = x[b * N + i].clone()
                hit = torch.nonzero(mine + asked)[:, 0]
                z = y[hit]
                y[hit] = torch.where(z > 0, z / r, z * r) - f * mine[hit] - p * (mine[hit] > 0)
                if case["M"]:
                    ids = s["bias_ids"][b].long().cpu()
                    y[ids[ids >= 0]] += s["bias_values"][b].double().cpu()[ids >= 0]
                g = int(s["mask_rows"][b * N + i]) if case["masks"] else -1
                if g >= 0:
                    y[~allowed[g]] = -math.inf
                out[b * N + i, :V] = y
                out[b * N + i, V:] = -math.inf
        return dict(out=out)
    bs, flat = case["block"], s["pool"].double()
    tok, chosen, table, start = (s[k].tolist() for k in ("tok", "chosen", "table", "pos"))
    for b in range(B):
        path, at = [0], 0
        while True:
            nxt = [i for i in range(N) if parent[b][i] == at and tok[b][i] == chosen[b][at]]
            if not nxt:
                break
            at = nxt[0]
            path.append(at)
        slot = [(table[b][(start[b] + i) // bs], (start[b] + i) % bs) for i in range(N)]
        old = [flat[:, :, slot[i][0], :, slot[i][1]].clone() for i in path]
        for k, rows in enumerate(old):
            flat[:, :, slot[k][0], :, slot[k][1]] = rows
    return dict(path=None, count=None, emitted=None, next_tok=None, next_pos=None, pool=flat)
