"""Plain 64-bit CPU forms of the operators that verify drafted tokens, for the
tests, and the trees they run on."""
import numpy as np


def paths(parent, live=64):
    """Each node's path, itself last ([] for a missing node), of one tree;
    `live`: nodes from there on are missing.  (paths, bits: 16 for a bad parent,
    4 for a present node past `live`)."""
    out, bits = [], 0
    for i, p in enumerate(parent):
        p = int(p)
        if p < -2 or p >= i:
            bits |= 16
            out.append([])
        elif p == -2:
            out.append([])
        elif i >= live:
            bits |= 4
            out.append([])
        elif p == -1:
            out.append([i])
        else:
            out.append(out[p] + [i] if out[p] else [])
    return out, bits


def chain(B, N):
    return np.tile(np.arange(N) - 1, (B, 1)).astype(np.int32)


def trees(B, N, seed, missing=True, roots=False):
    """Random trees: node 0 behind the cache, sometimes further ones, sometimes
    fewer nodes than N, and missing ones in the middle."""
    rng = np.random.default_rng(seed)
    p = np.full((B, N), -1, np.int32)
    for b in range(B):
        kind = rng.integers(4)
        for i in range(1, N):
            p[b, i] = i - 1 if kind == 0 else 0 if kind == 1 else rng.integers(0, i)
            if roots and rng.random() < 0.1:
                p[b, i] = -1
            if missing and rng.random() < 0.05:
                p[b, i] = -2
        if missing and rng.random() < 0.4:
            p[b, rng.integers(0, N):] = -2
    return p


def tree_attention(q, k_new, v_new, pool, table, pos, parent, bs, capacity):
    """q, k_new, v_new [B, N, NH, hs], pool [2, blocks, NH, bs, hs], float64:
    (out [B, N, NH, hs], the largest |k.q| sum / sqrt(hs) and the largest |v| of
    each row [B, N, NH], the positions seen [B, N], who is there)."""
    B, N, NH, hs = q.shape
    out, sabs, vmax = np.zeros((B, N, NH, hs)), np.zeros((B, N, NH)), np.zeros((B, N, NH))
    n_seen, there = np.zeros((B, N)), np.zeros((B, N), bool)
    for b in range(B):
        n = int(pos[b])
        if not 0 <= n < capacity:
            continue
        j = np.arange(n)
        blk, off = table[b, j // bs], j % bs
        blk = np.where((blk < 0) | (blk >= pool.shape[1]), 0, blk)
        old = pool[:, blk, :, off].transpose(1, 0, 2, 3) if n else np.zeros((2, 0, NH, hs))
        for i, path in enumerate(paths(parent[b], capacity - n)[0]):
            if not path:
                continue
            there[b, i] = True
            k, v = np.concatenate([old[0], k_new[b, path]]), np.concatenate([old[1], v_new[b, path]])
            n_seen[b, i] = len(k)
            s = np.einsum("hd,jhd->hj", q[b, i], k) / np.sqrt(hs)
            sabs[b, i] = np.einsum("hd,jhd->hj", np.abs(q[b, i]), np.abs(k)).max(1) / np.sqrt(hs)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[b, i] = np.einsum("hj,jhd->hd", p, v)
            vmax[b, i] = np.abs(v).max((0, 2))
    return out, sabs, vmax, n_seen, there


def adjust(x, V, history, history_len, prompt_len, repetition, presence, frequency, bias_ids, bias_values, masks,
           mask_rows, tok, parent):
    """x [B, N, V] float64: (the adjusted rows, the largest absolute value met on
    the way to each, who is there).  Everything but x may be None."""
    B, N, _ = x.shape
    y, size = x.copy(), np.abs(np.where(np.isfinite(x), x, 0))
    there = np.zeros((B, N), bool)
    for b in range(B):
        said, asked = np.zeros(V), np.zeros(V)
        if history is not None:
            H = history.shape[1]
            n = H if history_len is None else int(np.clip(history_len[b], 0, H))
            m = 0 if prompt_len is None else int(np.clip(prompt_len[b], 0, n))
            for t, where in [(t, asked if k < m else said) for k, t in enumerate(history[b, :n])]:
                if 0 <= t < V:
                    where[t] += 1
        for i, path in enumerate(paths(parent[b])[0]):
            if not path:
                continue
            there[b, i] = True
            count = said.copy()
            for a in path if tok is not None else []:
                if 0 <= tok[b, a] < V:
                    count[tok[b, a]] += 1
            r = y[b, i]

            def met(v):
                size[b, i, v] = max(size[b, i, v], abs(r[v]) if np.isfinite(r[v]) else 0)

            for v in np.nonzero(count + asked)[0]:
                if repetition is not None:
                    r[v] = r[v] / float(repetition[b]) if r[v] > 0 else r[v] * float(repetition[b])
                met(v)
                if count[v]:
                    f = 0.0 if frequency is None else float(frequency[b])
                    r[v] -= f * count[v]
                    size[b, i, v] += abs(f * count[v])
                    met(v)
                    r[v] -= 0.0 if presence is None else float(presence[b])
                    met(v)
            if bias_ids is not None:
                last = {int(t): float(w) for t, w in zip(bias_ids[b], bias_values[b]) if 0 <= t < V}
                for v, w in last.items():
                    r[v] += w
                    met(v)
            g = -1 if masks is None else int(mask_rows[b * N + i])
            if g != -1:
                v = np.arange(V)
                ok = (masks[g, v // 32].astype(np.int64) >> (v % 32)) & 1 if 0 <= g < len(masks) else np.zeros(V)
                r[ok == 0] = -np.inf
    return y, size, there


def accept(tok, parent, chosen, pos, capacity=1 << 30):
    """(path, emitted [B, N], count, next_tok, next_pos [B]): step by step."""
    B, N = tok.shape
    path, emitted = np.full((B, N), -1), np.full((B, N), -1)
    count, last, nxt = np.zeros(B, int), np.full(B, -1), np.array(pos, int)
    for b in range(B):
        if not 0 <= pos[b] < capacity:
            continue
        there = [bool(p) for p in paths(parent[b], capacity - int(pos[b]))[0]]
        if not there[0]:
            continue
        at, k = 0, 0
        while True:
            path[b, k] = at
            emitted[b, k] = chosen[b, at]
            k += 1
            kids = [i for i in range(N) if parent[b, i] == at and there[i] and tok[b, i] == chosen[b, at]]
            if not kids:
                break
            at = kids[0]
        count[b], last[b], nxt[b] = k, chosen[b, at], pos[b] + k
    return path, emitted, count, last, nxt


def moved(pool, table, path, pos, bs):
    """pool [L, 2, blocks, NH, bs, hs] (any array that copies) with the rows of
    each path at consecutive positions; a row through an entry outside the pool
    stays."""
    out, n_blocks = pool.copy(), pool.shape[2]
    for b in range(len(pos)):
        for k, i in enumerate(path[b]):
            if i < 0 or i == k:
                continue
            s, d = int(pos[b]) + int(i), int(pos[b]) + k
            sb, db = table[b, s // bs], table[b, d // bs]
            if 0 <= sb < n_blocks and 0 <= db < n_blocks:
                out[:, :, db, :, d % bs] = pool[:, :, sb, :, s % bs]
    return out
