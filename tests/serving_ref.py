"""Plain 64-bit implementations (numpy) of the serving operators next to the recurrence, for the
parity tests. Written from the formulas; no code is shared with the library."""
import math

import numpy as np
import torch

PAGE = 64
_CODE = None


def code_values():
    """The 256 values of the 8-bit format: 1 sign, 4 exponent (bias 7), 3 mantissa bits; the
    all-ones pattern is NaN."""
    global _CODE
    if _CODE is None:
        v = np.zeros(256)
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
        _CODE = v
    return _CODE


def values(codes):
    """float64 values of a code tensor."""
    return code_values()[codes.view(torch.uint8).cpu().numpy()]


def round_e4m3(x):
    """Nearest value of the format, ties to even, saturated at +-448; NaN stays."""
    x = np.clip(np.asarray(x, dtype=np.float64), -448, 448)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.clip(np.round(x / step) * step, -448, 448)


def pow2_scale(m):
    """Smallest power of two s >= 2^-100 with m <= 448 s."""
    s = 2.0 ** -100
    while m > 448 * s:
        s *= 2
    return s


def head_norm(x, w, eps, l2, table, pos, interleaved):
    """x float64 [T, H, d] -> [T, H, d]; table [n_pos, rot] float64 or None."""
    d = x.shape[2]
    ss = (x * x).sum(-1, keepdims=True)
    y = x / np.sqrt((ss if l2 else ss / d) + eps)
    if w is not None:
        y = y * w
    if table is None or table.shape[1] == 0:
        return y
    h = table.shape[1] // 2
    out = y.copy()
    for t in range(x.shape[0]):
        if not 0 <= pos[t] < table.shape[0]:
            continue
        c, s = table[pos[t], :h], table[pos[t], h:]
        ia, ib = (np.arange(h) * 2, np.arange(h) * 2 + 1) if interleaved else \
            (np.arange(h), np.arange(h) + h)
        a, b = y[t][:, ia], y[t][:, ib]
        out[t][:, ia] = a * c - b * s
        out[t][:, ib] = b * c + a * s
    return out


def cache_write(x, val, scale, cu, start, lens, table, n_pages):
    """In place on val [n_pages, H, 64, d] (code values, float64) and scale [n_pages, H]."""
    H = x.shape[1]
    for s in range(len(start)):
        n = cu[s + 1] - cu[s]
        if lens is not None:
            n = min(n, max(int(lens[s]), 0))
        if start[s] < 0:
            continue
        i = 0
        while i < n:
            pos = start[s] + i
            blk, off = pos // PAGE, pos % PAGE
            take = min(PAGE - off, n - i)
            page = table[s][blk] if blk < len(table[s]) else -1
            if 0 <= page < n_pages:
                for h in range(H):
                    new = x[cu[s] + i:cu[s] + i + take, h]
                    fin = np.abs(new[np.isfinite(new)])
                    sc = pow2_scale(fin.max() if fin.size else 0.0)
                    if off:
                        sc = max(sc, scale[page, h])
                        val[page, h, :off] = round_e4m3(val[page, h, :off] * (scale[page, h] / sc))
                    val[page, h, off:off + take] = round_e4m3(new / sc)
                    scale[page, h] = sc
            i += take


def gather(val, scale, table_row, n, n_pages):
    """Values [n, H, d] of positions 0 .. n-1 of one row, and which of them are present."""
    H, d = val.shape[1], val.shape[3]
    out, there = np.zeros((n, H, d)), np.zeros(n, dtype=bool)
    for t0 in range(0, n, PAGE):
        blk = t0 // PAGE
        page = table_row[blk] if blk < len(table_row) else -1
        m = min(PAGE, n - t0)
        if 0 <= page < n_pages:
            there[t0:t0 + m] = True
            out[t0:t0 + m] = (val[page, :, :m] * scale[page][:, None, None]).transpose(1, 0, 2)
    return out, there


def attention(q, start, lens, table, kval, kscale, vval, vscale, scale, batch):
    """q float64 [batch * W, Hq, d]; returns o of the same shape."""
    W = q.shape[0] // batch
    Hkv = kval.shape[1]
    G = q.shape[1] // Hkv
    o = np.zeros_like(q)
    for b in range(batch):
        if start[b] < 0:
            continue
        k, there = gather(kval, kscale, table[b], int(start[b]) + W, kval.shape[0])
        v, _ = gather(vval, vscale, table[b], int(start[b]) + W, vval.shape[0])
        for j in range(W if lens is None else min(W, int(lens[b]))):
            n = int(start[b]) + j + 1
            seen = np.nonzero(there[:n])[0]
            if not seen.size:
                continue
            for h in range(q.shape[1]):
                s = scale * (k[seen, h // G] @ q[b * W + j, h])
                p = np.exp(s - s.max())
                o[b * W + j, h] = (p / p.sum()) @ v[seen, h // G]
    return o


def verify(target, draft, drafts, lens, ua, us, slots):
    """Plain Python, integers for the weights. target/draft float32 arrays."""
    B, W1, V = target.shape
    W = W1 - 1
    tokens, count, resume = np.full((B, W1), -1, np.int64), np.zeros(B, np.int64), []
    for b in range(B):
        n_len = W if lens is None else min(W, int(lens[b]))
        if n_len < 0:
            resume.append(-1)
            continue
        n, bad = 0, False
        while n < n_len:
            x = int(drafts[b, n])
            bad = not 0 <= x < V
            if bad:
                break
            q = np.float32(1) if draft is None else draft[b, n, x]
            if not np.float32(ua[b, n]) * q < target[b, n, x]:
                break
            tokens[b, n] = x
            n += 1
        y = target[b, n].astype(np.float32).copy()
        if n < n_len and not bad:
            if draft is None:
                y[int(drafts[b, n])] = 0
            else:
                y = y - draft[b, n]
        for z in (y, target[b, n]):
            z = np.where(np.isnan(z), np.float32(0), z)
            w = np.floor(np.clip(z, 0, 1).astype(np.float64) * 2.0 ** 40).astype(np.int64)
            total = int(w.sum())
            if total:
                break
        if total:
            r = total * int(math.floor(float(us[b]) * 2 ** 24)) // 2 ** 24
            tokens[b, n] = int(np.searchsorted(np.cumsum(w), r, side="right"))
        count[b] = n
        resume.append(-1 if slots is None else int(slots[b, n]))
    return count, tokens, np.array(resume)
