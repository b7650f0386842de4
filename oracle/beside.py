"""fp64 CPU oracle of the operators beside the experts: the router with its balance loss
and gradient, 4-bit weights with group scales, the quantised cache.

Plain NumPy from the formulas, token by token and block by block; shares no code with
the GPU path. Arrays come in as float64 (the exact values of their 16- or 32-bit
elements) or as raw bytes, and results go out as float64, unrounded, or as bytes.
"""

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


# ------------------------------------------------------------------ the router

def scores(z, score):
    """Scores of one token's logits; -inf: 0."""
    if score == "sigmoid":
        return np.array([0.0 if v == -np.inf else 1 / (1 + np.exp(-v)) if v > 0 else np.exp(v) / (1 + np.exp(v))
                         for v in z])
    on = z[z > -np.inf]
    if on.size == 0:
        return np.zeros_like(z)
    e = np.exp(z - on.max())
    return e / e.sum()


def shares(z, score):
    s = scores(z, score)
    return s / s.sum() if s.sum() > 0 else s


def moe_gate(logits, k, score="softmax", bias=None, renorm=True, scale=1.0):
    T, E = logits.shape
    ids, w = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        s = scores(logits[t], score)
        key = logits[t] if bias is None else s + bias
        on = [e for e in range(E) if logits[t, e] > -np.inf]
        chosen = sorted(on, key=lambda e: (-key[e], e))[:k]
        ids[t, :len(chosen)] = chosen
        total = sum(s[e] for e in chosen) if renorm else 1.0
        for j, e in enumerate(chosen):
            w[t, j] = scale * s[e] / total if total > 0 else 0.0
    return ids, w


def moe_balance(logits, ids, seq_off=None, score="softmax", coef=1.0):
    """(loss [S], counts [S, E])."""
    T, E = logits.shape
    k = ids.shape[1]
    seq_off = [0, T] if seq_off is None else seq_off
    S = len(seq_off) - 1
    loss, counts = np.zeros(S), np.zeros((S, E), np.int64)
    for q in range(S):
        a, b = seq_off[q], seq_off[q + 1]
        p = np.zeros(E)
        for t in range(a, b):
            p += shares(logits[t], score)
            for e in ids[t]:
                if 0 <= e < E:
                    counts[q, e] += 1
        if b > a:
            loss[q] = coef * E / (k * (b - a) ** 2) * (counts[q] * p).sum()
    return loss, counts


def moe_gate_grad(logits, ids, d_w=None, counts=None, d_loss=None, seq_off=None, score="softmax", renorm=True,
                  scale=1.0, coef=1.0):
    """(d_logits, the sum of the magnitudes of what each is a sum of)."""
    T, E = logits.shape
    k = ids.shape[1]
    seq_off = [0, T] if seq_off is None else seq_off
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s, p = scores(logits[t], score), shares(logits[t], score)
        slots = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        d, m = np.zeros(E), np.zeros(E)             # for the scores, and its parts' magnitudes
        if d_w is not None:
            total = sum(s[e] for _, e in slots) if renorm else 1.0
            if total > 0:
                mean = sum(s[e] * d_w[t, j] for j, e in slots) / total if renorm else 0.0
                most = sum(s[e] * abs(d_w[t, j]) for j, e in slots) / total if renorm else 0.0
                for j, e in slots:
                    d[e] += scale * (d_w[t, j] - mean) / total
                    m[e] += scale * (abs(d_w[t, j]) + most) / total
        b, c = np.zeros(E), np.zeros(E)             # for the shares
        for q in range(len(seq_off) - 1):
            if counts is not None and seq_off[q] <= t < seq_off[q + 1]:
                n = seq_off[q + 1] - seq_off[q]
                b = coef * E / (k * n * n) * d_loss[q] * counts[q]
        c = p * (np.abs(b) + (p * np.abs(b)).sum())
        b = p * (b - (p * b).sum())
        if score == "sigmoid":
            out[t] = (1 - s) * (s * d + b)
            size[t] = (1 - s) * (s * m + c)
        else:
            # the renormalised weights give the sum nothing
            out[t] = s * (d - (0.0 if renorm else (s * d).sum())) + b
            size[t] = s * (m + (0.0 if renorm else (s * m).sum())) + c
    return out, size


# ------------------------------------------------------------------ 4-bit weights

def nibbles(w):
    out = np.empty((w.shape[0], 2 * w.shape[1]), np.int64)
    out[:, 0::2], out[:, 1::2] = w & 15, w >> 4
    return out


def e8m0(b):
    return np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))


def w4_weights(w, scales, zeros=None):
    """(values [N, K], the magnitudes that enter the products: code and zero point apart)."""
    code = nibbles(w)
    group = code.shape[1] // scales.shape[1]
    if scales.dtype == np.uint8:
        s = np.repeat(e8m0(scales), group, 1)
        v = np.where(code < 8, 1, -1) * E2M1[code & 7] * s
        return v, np.abs(v)
    s = np.repeat(scales, group, 1)
    z = np.full(code.shape, 8) if zeros is None else np.repeat(zeros.astype(np.int64), group, 1)
    return (code - z) * s, (code + z) * np.abs(s)


# ------------------------------------------------------------------ the cache

def _grid(fmt):
    """Non-negative element values, code by code."""
    if fmt == "mxfp4":
        return E2M1
    v = [f * 2.0 ** -9 for f in range(8)]
    return np.array((v + [(1 + f / 8) * 2.0 ** (e - 7) for e in range(1, 16) for f in range(8)])[:127])


def quantize_rows(x, fmt):
    """(codes, scales) bytes of float64 rows: each block of 32 by itself, each value to the nearest of the grid."""
    grid, emax = _grid(fmt), 2 if fmt == "mxfp4" else 8
    sign_bit = 8 if fmt == "mxfp4" else 128
    R, W = x.shape
    codes, scales = np.zeros((R, W), np.int64), np.zeros((R, W // 32), np.uint8)
    mid = (grid[1:] + grid[:-1]) / 2
    for r in range(R):
        for b in range(W // 32):
            v = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                continue
            amax = np.abs(v).max()
            byte = 0 if amax == 0 else max(int(np.frexp(amax)[1]) - 1 - emax + 127, 0)
            scales[r, b] = byte
            a = np.abs(v) * 2.0 ** (127 - byte)
            i = np.searchsorted(mid, a)                       # mid[i - 1] < a <= mid[i]
            tie = (i < len(mid)) & (a == mid[np.minimum(i, len(mid) - 1)])
            i = np.where(tie & (i % 2 == 1), i + 1, i)        # of two the even code
            codes[r, 32 * b:32 * b + 32] = i + np.where(np.signbit(v), sign_bit, 0)
    if fmt == "mxfp4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return codes.astype(np.uint8), scales


def dequantize_rows(codes, scales, fmt):
    if fmt == "mxfp4":
        c = nibbles(codes)
        v = E2M1[c & 7] * np.where(c < 8, 1, -1)
    else:
        c = codes.astype(np.int64)
        v = np.append(_grid(fmt), np.nan)[c & 127] * np.where(c < 128, 1, -1)
    return v * np.repeat(e8m0(scales), 32, 1)


def cache_write(x, slots, codes, scales, fmt):
    """Copies of codes and scales [pages, page_size, ..] with the rows written."""
    c, s = codes.reshape(-1, codes.shape[2]).copy(), scales.reshape(-1, scales.shape[2]).copy()
    qc, qs = quantize_rows(x, fmt)
    for t, i in enumerate(slots):
        if 0 <= i < c.shape[0]:
            c[i], s[i] = qc[t], qs[t]
    return c.reshape(codes.shape), s.reshape(scales.shape)


def cache_read(codes, scales, table, seq_off, out, fmt):
    """A copy of float64 out with the sequences' rows."""
    out = out.copy()
    pages, page_size = codes.shape[:2]
    for b in range(len(seq_off) - 1):
        for r in range(seq_off[b], min(seq_off[b + 1], out.shape[0])):
            i = r - seq_off[b]
            page = table[b, i // page_size] if i // page_size < table.shape[1] else -1
            out[r] = 0.0
            if 0 <= page < pages:
                out[r] = dequantize_rows(codes[page, i % page_size][None], scales[page, i % page_size][None], fmt)[0]
    return out
