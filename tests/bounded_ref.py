"""Plain 64-bit implementations (numpy) of linear attention with one decay per head and of the
eviction from the paged cache, for the parity tests. Written from the formulas; no code is shared
with the library."""
import numpy as np

import serving_ref as ref

PAGE = 64


def decay_steps(q, k, v, g, state):
    """One sequence token by token: q, k, v [T, H, d], g [T, H], state [H, d, d]. Returns S^T q per
    token and every state."""
    o, states = np.zeros_like(v), []
    s = state.copy()
    for t in range(q.shape[0]):
        s = s * np.exp(g[t])[:, None, None] + k[t][:, :, None] * v[t][:, None, :]
        o[t] = np.einsum("hk,hkv->hv", q[t], s)
        states.append(s)
    return o, states


def decay_prefill(q, k, v, g, cu, init, scale):
    """q, k [T, Hk, d], v [T, H, d], g [T, H], init [n, H, d, d]. Returns o, final states, and for
    both the same sums with every term's absolute value (what rounding errors are relative to)."""
    H, Hk = v.shape[1], q.shape[1]
    q, k = (np.repeat(x, H // Hk, 1) for x in (q, k))
    o, oa = np.zeros_like(v), np.zeros_like(v)
    fin, fa = init.copy(), np.abs(init)
    for s in range(len(cu) - 1):
        a, b = int(cu[s]), int(cu[s + 1])
        if b <= a:
            continue
        x, st = decay_steps(q[a:b], k[a:b], v[a:b], g[a:b], init[s])
        o[a:b], fin[s] = x * scale, st[-1]
        with np.errstate(invalid="ignore"):
            x, st = decay_steps(*(np.abs(y[a:b]) for y in (q, k, v)), g[a:b], np.abs(init[s]))
        oa[a:b], fa[s] = x * abs(scale), st[-1]
    return o, fin, oa, fa


def weigh(q, start, lens, table, kval, kscale, weights, scale, keep, batch):
    """In place on weights [n_pages, H, 64]; q [batch * W, Hq, d]. Returns for each entry the sum over
    queries of p times the sum of absolute products behind its score (what errors are relative
    to), and which entries were written."""
    W = q.shape[0] // batch
    n_pages, Hkv = kval.shape[:2]
    G = q.shape[1] // Hkv
    size, written = np.zeros_like(weights), np.zeros(weights.shape, dtype=bool)
    for b in range(batch):
        n = W if lens is None else max(0, min(W, int(lens[b])))
        if start[b] < 0 or n == 0:
            continue
        k, there = ref.gather(kval, kscale, table[b], int(start[b]) + n, n_pages)
        for t in np.nonzero(there)[0]:
            page, at = table[b][t // PAGE], t % PAGE
            written[page, :, at] = True
            old = weights[page, :, at]
            weights[page, :, at] = keep * old if t < start[b] and keep != 0 else 0.0
        for j in range(n):
            seen = np.nonzero(there[:int(start[b]) + j + 1])[0]
            if not seen.size:
                continue
            page, at = np.asarray(table[b])[seen // PAGE], seen % PAGE
            for h in range(q.shape[1]):
                kh, x = k[seen, h // G], q[b * W + j, h]
                s = scale * (kh @ x)
                p = np.exp(s - s.max())
                p /= p.sum()
                top = (abs(scale) * (np.abs(kh) @ np.abs(x))).max()
                weights[page, h // G, at] += p
                size[page, h // G, at] += p * top
    return size, written


def evict(length, table, new_table, sides, weights, budget, sinks, recent):
    """In place on sides = [(code values [n_pages, H, 64, d], scales [n_pages, H])] and weights.
    Returns new_length, kept."""
    n_pages, H = weights.shape[:2]
    n = len(length)
    count, kept = np.zeros(n, np.int64), np.full((n, H, budget), -1, np.int64)
    for b in range(n):
        if length[b] < 0:
            count[b] = length[b]
            continue
        end = min(int(length[b]), len(table[b]) * PAGE)
        there = [t for t in range(end) if 0 <= table[b][t // PAGE] < n_pages]
        count[b] = min(len(there), budget)
        for h in range(H):
            def rank(t):
                if t < sinks or t >= end - recent:
                    return (0, 0.0, t)
                w = weights[table[b][t // PAGE], h, t % PAGE]
                return (2, 0.0, t) if np.isnan(w) else (1, -w, t)
            keep = sorted(sorted(there, key=rank)[:count[b]])
            kept[b, h, :len(keep)] = keep
            for i in range(0, len(keep), PAGE):
                dst, part = new_table[b][i // PAGE], keep[i:i + PAGE]
                if not 0 <= dst < n_pages:
                    continue
                src = [(table[b][t // PAGE], t % PAGE) for t in part]
                for val, scale in sides:
                    s = max(scale[p, h] for p, _ in src)
                    for r, (p, at) in enumerate(src):
                        val[dst, h, r] = ref.round_e4m3(val[p, h, at] * (scale[p, h] / s))
                    scale[dst, h] = s
                w = [weights[p, h, at] for p, at in src]
                weights[dst, h] = 0
                weights[dst, h, :len(w)] = w
    return count, kept
