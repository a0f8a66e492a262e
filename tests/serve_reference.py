"""Plain 64-bit CPU forms of the serving operators, for the tests."""
import numpy as np


def tables(table, cached, new, free, taken, prefix_blocks, prefix_len, T, num_blocks, bs):
    """(table, slots, next_len, taken, bits): request by request."""
    table, B, cap = table.copy(), len(cached), table.shape[1] * bs
    slots, nxt, bits = np.full((B, T), -1, np.int64), np.array(cached, np.int64), 0
    left = len(free) - taken if 0 <= taken <= len(free) else 0
    end, given = 0, 0
    for b in range(B):
        n, add = int(cached[b]), int(new[b]) if new is not None else min(T, 1)
        if n < 0 or add < 0 or add > T or n > cap or n + add > cap or n < prefix_len:
            bits |= 4
            continue
        have, need = -(-n // bs), -(-(n + add) // bs)
        end += need - have
        if need > have and end > left:
            continue
        start = end - (need - have)
        if need > have:
            given = end
        table[b, :prefix_len // bs] = prefix_blocks[:prefix_len // bs] if prefix_len else []
        table[b, have:need] = free[taken + start:taken + end] if need > have else []
        for t in range(add):
            blk = int(table[b, (n + t) // bs])
            if 0 <= blk < num_blocks:
                slots[b, t] = blk * bs + (n + t) % bs
            else:
                bits |= 8
        nxt[b] = n + add
    return table, slots, nxt, taken + given, bits


def logprobs(x, targets, K):
    """x [N, V] float64 (the logits' exact values): dict of arrays."""
    N, V = x.shape
    out = {k: np.zeros(N) for k in ("lse", "entropy", "logprob")}
    out["top_ids"] = np.full((N, K), -1, np.int64)
    out["top_logprobs"] = np.full((N, K), -np.inf)
    for n in range(N):
        r = x[n]
        if np.isnan(r).any() or (r == np.inf).any():
            out["lse"][n] = out["entropy"][n] = np.nan
            out["logprob"][n] = np.nan
            out["top_logprobs"][n] = np.nan
        elif (r == -np.inf).all():
            out["lse"][n] = out["logprob"][n] = -np.inf
        else:
            m = r.max()
            with np.errstate(under="ignore", over="ignore"):
                e = np.exp(r - m)
            s = e.sum()
            logp = (r - m) - np.log(s)  # l - lse without the rounding of a large lse
            some = e > 0
            out["lse"][n] = m + np.log(s)
            out["entropy"][n] = -(e[some] / s * logp[some]).sum()
            if targets is not None:
                out["logprob"][n] = logp[max(0, targets[n])]
            order = np.lexsort((np.arange(V), -r))[:K]
            order = order[r[order] > -np.inf]
            out["top_ids"][n, :len(order)] = order
            out["top_logprobs"][n, :len(order)] = logp[order]
        if targets is None or not 0 <= targets[n] < V:
            out["logprob"][n] = 0.0
    return out


def logprobs_grad(x, targets, entropy, g, h):
    """The formula's dlogits [N, V] in 64 bits."""
    N, V = x.shape
    d = np.zeros((N, V))
    for n in range(N):
        gn = 0.0 if g is None or not 0 <= targets[n] < V else float(g[n])
        hn = 0.0 if h is None else float(h[n])
        m = x[n].max()
        if m == -np.inf:
            continue
        with np.errstate(under="ignore", invalid="ignore", over="ignore"):
            lp = (x[n] - m) - np.log(np.exp(x[n] - m).sum())
            p = np.exp(lp)
            d[n] = -p * gn
            if hn:
                d[n] -= np.where(p == 0, 0.0, hn * p * (np.where(p == 0, 0.0, lp) + entropy[n]))
        if gn:
            d[n, targets[n]] += gn
    return d


def shared_attention(q, k_new, v_new, pool, table, pos, prefix_len, bs):
    """q, k_new, v_new [B, NH, hs], pool [2, blocks, NH, bs, hs], float64:
    (out [B, NH, hs], the largest |k.q| sum / sqrt(hs) of each row [B, NH],
    the largest |v| of each row [B, NH])."""
    B, NH, hs = q.shape
    out, sabs, vmax = np.zeros((B, NH, hs)), np.zeros((B, NH)), np.zeros((B, NH))
    for b in range(B):
        j = np.arange(pos[b])
        rows = np.where(j < prefix_len, 0, b)
        blk, off = table[rows, j // bs], j % bs
        k = np.concatenate([pool[0, blk, :, off], k_new[b][None]])  # [n, NH, hs]
        v = np.concatenate([pool[1, blk, :, off], v_new[b][None]])
        s = np.einsum("hd,jhd->hj", q[b], k) / np.sqrt(hs)
        sabs[b] = np.einsum("hd,jhd->hj", np.abs(q[b]), np.abs(k)).max(1) / np.sqrt(hs)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[b] = np.einsum("hj,jhd->hd", p, v)
        vmax[b] = np.abs(v).max((0, 2))
    return out, sabs, vmax
