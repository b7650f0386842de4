"""fp64 CPU oracle of the operators around the experts: rows to the experts and back
with the gradient, the norms around a block, low-rank adapters.

Plain NumPy from the formulas, row by row and slot by slot; shares no code with the
GPU path. Arrays come in as float64 (the exact values of their 16- or 32-bit
elements) and results go out as float64, unrounded.
"""

import numpy as np


def moe_sort(ids, E):
    """(expert_off [E+1], row_slot [P], slot_row [T, k]) of ids [T, k]; -1 where there is none."""
    flat = [int(v) for v in np.asarray(ids).reshape(-1)]
    off, row_slot = [0], []
    for e in range(E):
        row_slot += [p for p, v in enumerate(flat) if v == e]
        off.append(len(row_slot))
    slot_row = np.full(len(flat), -1, np.int64)
    for r, p in enumerate(row_slot):
        slot_row[p] = r
    row_slot = np.array(row_slot + [-1] * (len(flat) - len(row_slot)), np.int64)
    return np.array(off, np.int64), row_slot, slot_row.reshape(np.asarray(ids).shape)


def moe_permute(x, slot_row, xs):
    """xs with row slot_row[t, j] = x[t]; the other rows as they are."""
    xs = xs.copy()
    for t in range(slot_row.shape[0]):
        for r in slot_row[t]:
            if 0 <= r < xs.shape[0]:
                xs[r] = x[t]
    return xs


def moe_unpermute(ys, slot_row, w=None):
    T, k = slot_row.shape
    y = np.zeros((T, ys.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < ys.shape[0]:
                y[t] += ys[r] * (1.0 if w is None else w[t, j])
    return y


def moe_unpermute_grad(dy, ys, slot_row, w, dys):
    dys, dw = dys.copy(), np.zeros(slot_row.shape)
    for t in range(slot_row.shape[0]):
        for j in range(slot_row.shape[1]):
            r = slot_row[t, j]
            if 0 <= r < ys.shape[0]:
                dys[r] = w[t, j] * dy[t]
                dw[t, j] = dy[t] @ ys[r]
    return dys, dw


def _rms(v, eps):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def block_norm(residual, w_pre=None, y=None, w_post=None, gate=None, res_scale=1.0, eps=1e-6):
    """(normed or None, residual_out)."""
    r = residual
    if y is not None:
        u = y if w_post is None else y / _rms(y, eps) * w_post
        r = residual + res_scale * (u if gate is None else gate * u)
    return (None if w_pre is None else r / _rms(r, eps) * w_pre), r


def _norm_grad(v, w, dn, eps):
    """Gradient of v / rms(v) * w for v, and v / rms(v)."""
    s = _rms(v, eps)
    h = v / s
    return (dn * w - h * (dn * w * h).mean(axis=1, keepdims=True)) / s, h


def block_norm_grad(r, w_pre=None, dn=None, dr_out=None, y=None, w_post=None, gate=None, res_scale=1.0, eps=1e-6):
    """dict of d_residual, dw_pre, d_y, dw_post, d_gate (what there is of them) at the stored sum r."""
    g = {"d_residual": np.zeros_like(r) if dr_out is None else dr_out.copy()}
    if w_pre is not None:
        d, h = _norm_grad(r, w_pre, dn, eps)
        g["d_residual"] = g["d_residual"] + d
        g["dw_pre"] = (dn * h).sum(axis=0)
    if y is not None:
        df = res_scale * g["d_residual"]              # of gate * u
        du = df if gate is None else df * gate
        u = y
        g["d_y"] = du
        if w_post is not None:
            g["d_y"], h = _norm_grad(y, w_post, du, eps)
            g["dw_post"] = (du * h).sum(axis=0)
            u = h * w_post
        if gate is not None:
            d = df * u
            g["d_gate"] = d.sum(axis=0) if gate.ndim == 1 else d.sum(axis=1, keepdims=True) \
                if gate.shape[1] == 1 else d
    return g


def lora_add(y, x, a, b, adapter, scale=None):
    """y + scale (x A^T) B^T, each token with its adapter's; adapter outside [0, n): y."""
    y = y.copy()
    for t, i in enumerate(np.asarray(adapter).reshape(-1)):
        if 0 <= i < a.shape[0]:
            y[t] += (1.0 if scale is None else scale[i]) * (b[i] @ (a[i] @ x[t]))
    return y
