"""mx_block_norm and mx_block_norm_grad against the fp64 oracle, within bounds of their fp32 arithmetic."""

import itertools

import numpy as np
import pytest
import torch

from around_util import DTYPES, U, depth, f64, pair, rounded, within
from oracle import around

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def _inputs(T, H, name, res_name, gate, post, seed=0, size=3.0):
    rng = np.random.default_rng(seed + T * 10 + H)
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    d = {"y": pair(rng.standard_normal((T, H)), name), "residual": pair(size * rng.standard_normal((T, H)), res_name),
         "w_pre": pair(1 + 0.3 * rng.standard_normal(H), name),
         "w_post": pair(1 + 0.3 * rng.standard_normal(H), name) if post else (None, None),
         "gate": (None, None) if shape is None else pair(rng.uniform(-1, 1, shape), name),
         "dn": pair(rng.standard_normal((T, H)), name), "dro": pair(rng.standard_normal((T, H)), res_name)}
    return {k: v[0] for k, v in d.items()}, {k: v[1] for k, v in d.items()}


def _rms(v):
    return np.sqrt((v * v).mean(1, keepdims=True) + EPS)


def _bounds(h, s):
    """Bounds of the fp32 parts of (residual_out, normed) of the forward pass.
    A row's mean square: a sum of positive terms, off by depth * U of itself, halved by the root; the
    reciprocal root and the few products around it: 8 U together."""
    H = h["residual"].shape[1]
    rel = depth(H) * U / 2 + 8 * U
    n, r = around.block_norm(h["residual"], h["w_pre"], h["y"], h["w_post"], h["gate"], s, EPS)
    add = r - h["residual"]
    er = np.abs(add) * rel + 2 * U * (np.abs(r) + np.abs(h["residual"]))
    en = None
    if h["w_pre"] is not None:
        spread = np.sqrt((er * er).sum(1, keepdims=True) / (r * r).sum(1, keepdims=True))
        en = np.abs(n) * (rel + spread) + er / _rms(r) * np.abs(h["w_pre"])
    return n, r, en, er


def _forward(mx, T, H, name, res_name, gate, post, s=0.7):
    t, h = _inputs(T, H, name, res_name, gate, post)
    normed, res = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=s,
                                eps=EPS)
    n, r, en, er = _bounds(h, s)
    assert normed.dtype == DTYPES[name] and res.dtype == DTYPES[res_name]
    within(res, r, 1.02 * (er + rounded(r, res_name)), "residual_out")
    within(normed, n, 1.02 * (en + rounded(n, name)), "normed")


WIDTHS = [1, 7, 8, 64, 100, 264, 511, 512, 1000, 2048, 2056, 4104, 7168, 8192, 9000, 16384, 16383]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("name,res_name", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                           ("fp32", "fp32")])
def test_forward_widths(mx, H, name, res_name):
    _forward(mx, 5, H, name, res_name, "channel", True)


@pytest.mark.parametrize("gate,post", itertools.product(["none", "channel", "token", "full"], [False, True]))
@pytest.mark.parametrize("T,H", [(1, 264), (1, 7168), (33, 137), (3000, 72), (1100, 1160)])
def test_forward_gates(mx, T, H, gate, post):
    _forward(mx, T, H, "bf16", "bf16" if T % 2 else "fp32", gate, post)


def test_forward_parts(mx):
    """Only the norm of the residual; only the addition; in place."""
    t, h = _inputs(20, 520, "bf16", "fp32", "token", True)
    n, res = mx.block_norm(t["residual"], t["w_pre"], eps=EPS)
    assert res is t["residual"]
    ref, _ = around.block_norm(h["residual"], h["w_pre"], eps=EPS)
    within(n, ref, 1.02 * (np.abs(ref) * (depth(520) * U / 2 + 8 * U) + rounded(ref, "bf16")))
    none, added = mx.block_norm(t["residual"], None, y=t["y"], gate=t["gate"])
    assert none is None
    r = h["residual"] + h["y"] * h["gate"]
    within(added, r, 4 * U * (np.abs(r) + np.abs(h["residual"])))
    both = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    keep_r, keep_y = t["residual"].clone(), t["y"].clone()
    n2, r2 = mx.block_norm(keep_r, t["w_pre"], y=keep_y, w_post=t["w_post"], gate=t["gate"], eps=EPS,
                           residual_out=keep_r, normed=keep_y)
    assert n2 is keep_y and r2 is keep_r
    assert torch.equal(n2, both[0]) and torch.equal(r2, both[1])


def test_rows_do_not_touch_each_other(mx):
    """A row of NaN, one of infinities, one of zeros and one of tiny values; eps 0 on an ordinary row."""
    t, h = _inputs(70, 264, "bf16", "fp32", "full", True)
    base = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    t["y"][3], t["residual"][9], t["y"][11], t["residual"][11] = float("nan"), float("inf"), 0.0, 0.0
    t["y"][12], t["residual"][12] = 1e-38, 1e-38
    got = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    rest = [i for i in range(70) if i not in (3, 9, 11, 12)]
    for a, b in zip(base, got):
        assert torch.equal(a[rest], b[rest])
        assert not a[rest].isnan().any() and not b[11].any() and b[12].isfinite().all() and b[3].isnan().all()
    n, _ = mx.block_norm(t["residual"][:2], t["w_pre"], eps=0.0)
    r = h["residual"][:2]
    ref = r / np.sqrt((r * r).mean(1, keepdims=True)) * h["w_pre"]
    within(n, ref, 1.02 * (np.abs(ref) * (depth(264) * U / 2 + 8 * U) + rounded(ref, "bf16")))


# ---------------------------------------------------------------- backward

def _grad_bounds(h, r, s, T, H):
    """Reference gradients and bounds of their fp32 parts: every product and sum of the formulas with its
    absolute terms. rel: of 1 / rms; dots: of a row sum relative to the sum of its absolute terms."""
    rel, dots = depth(H) * U / 2 + 8 * U, depth(H) * U
    cols = (T + 32) * U                                # a column's sum over the rows
    g = around.block_norm_grad(r, h["w_pre"], h["dn"], h["dro"], h["y"], h["w_post"], h["gate"], s, EPS)
    e = {}
    dr = np.zeros_like(r) if h["dro"] is None else np.abs(h["dro"])
    edr = 2 * U * np.abs(g["d_residual"])
    if h["w_pre"] is not None:
        fr = 1 / _rms(r)
        rh, d = np.abs(r) * fr, np.abs(h["dn"] * h["w_pre"])
        m = (d * rh).mean(1, keepdims=True)
        edr = edr + fr * d * (rel + 4 * U) + fr * rh * m * (3 * rel + dots + 8 * U) + 4 * U * dr
        mass = (np.abs(h["dn"]) * rh).sum(0)
        e["dw_pre"] = mass * (rel + cols + 4 * U)
    e["d_residual"] = edr
    if h["y"] is not None:
        y = np.abs(h["y"])
        gate = 1.0 if h["gate"] is None else np.abs(h["gate"])
        adr = np.abs(g["d_residual"])
        du, edu = abs(s) * gate * adr, abs(s) * gate * (edr + 4 * U * adr)
        yh, w = y, 1.0
        if h["w_post"] is not None:
            fy = 1 / _rms(h["y"])
            yh, w = y * fy, np.abs(h["w_post"])
            d, ed = du * w, edu * w + 2 * U * du * w
            m = (d * yh).mean(1, keepdims=True)
            em = (ed * yh).mean(1, keepdims=True) + m * (2 * rel + dots + 8 * U)
            e["d_y"] = fy * (ed + d * (rel + 4 * U)) + fy * yh * (em + m * (2 * rel + 6 * U))
            e["dw_post"] = (yh * edu + du * yh * (rel + 6 * U)).sum(0) + cols * (du * yh).sum(0)
        else:
            e["d_y"] = edu
        if h["gate"] is not None:
            a = abs(s) * adr * yh * w
            ea = abs(s) * edr * yh * w + a * (rel + 8 * U)
            e["d_gate"] = ea.sum(0) + cols * a.sum(0) if h["gate"].ndim == 1 else \
                ea.sum(1, keepdims=True) + dots * a.sum(1, keepdims=True) if h["gate"].shape[1] == 1 else ea
    return g, e


def _grad(mx, t, h, name, res_name, s=0.7, **kw):
    T, H = h["residual"].shape
    out = dict(zip(("d_residual", "dw_pre", "d_y", "dw_post", "d_gate"),
                   mx.block_norm_grad(t["residual"], t["w_pre"], t["dn"], d_residual_out=t["dro"], y=t["y"],
                                      w_post=t["w_post"], gate=t["gate"], res_scale=s, eps=EPS, **kw)))
    ref, e = _grad_bounds(h, h["residual"], s, T, H)
    for key, got in out.items():
        if key not in ref:
            assert got is None, key
            continue
        full = key == "d_gate" and h["gate"].shape == (T, H)
        kind = res_name if key == "d_residual" else name if key == "d_y" or full else "fp32"
        assert got.dtype == DTYPES[kind], key
        within(got, ref[key], 1.02 * (e[key] + rounded(ref[key], kind)), key)
    return out


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("name,res_name", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                           ("fp32", "fp32")])
def test_grad_widths(mx, H, name, res_name):
    t, h = _inputs(5, H, name, res_name, "channel", True)
    _grad(mx, t, h, name, res_name)


@pytest.mark.parametrize("gate,post", itertools.product(["none", "channel", "token", "full"], [False, True]))
@pytest.mark.parametrize("T,H", [(1, 264), (1, 7168), (33, 137), (3000, 72), (1100, 1160)])
def test_grad_gates(mx, T, H, gate, post):
    name, res_name = ("bf16", "fp32") if T % 2 else ("fp32", "fp32")
    t, h = _inputs(T, H, name, res_name, gate, post)
    _grad(mx, t, h, name, res_name)


def test_grad_parts(mx):
    """Without the block, without the next norm, without a gradient from behind; in place."""
    t, h = _inputs(40, 1000, "fp16", "fp32", "channel", True)

    def cut(*names):
        return {k: None if k in names else v for k, v in t.items()}, {k: None if k in names else v for k, v in h.items()}
    _grad(mx, *cut("y", "w_post", "gate"), "fp16", "fp32")
    _grad(mx, *cut("w_pre", "dn"), "fp16", "fp32")
    _grad(mx, *cut("dro"), "fp16", "fp32")
    _grad(mx, *cut("y", "w_post", "gate", "dro"), "fp16", "fp32")
    ref = _grad(mx, t, h, "fp16", "fp32")
    t2 = {k: v.clone() if v is not None else None for k, v in t.items()}
    got = _grad(mx, t2, h, "fp16", "fp32", d_residual=t2["dro"], d_y=t2["dn"])
    assert got["d_residual"] is t2["dro"] and got["d_y"] is t2["dn"]
    for key in ref:
        assert torch.equal(ref[key], got[key]), key


def test_grad_without_rows_is_zero(mx):
    z = torch.empty((0, 40), device="cuda")
    w = torch.ones(40, device="cuda")
    dr, dw_pre, dy, dw_post, dg = mx.block_norm_grad(z, w, z, d_residual_out=z, y=z, w_post=w, gate=w)
    assert dr.shape == dy.shape == (0, 40)
    assert not dw_pre.any() and not dw_post.any() and not dg.any()
    n, r = mx.block_norm(z, w, y=z, w_post=w, gate=w)
    assert n.shape == r.shape == (0, 40)


def test_grad_is_the_gradient_of_the_forward_pass(mx):
    """Differences of the forward kernel itself in fp32: for f = sum(normed dn + residual_out dro), the change
    along a direction is the gradient's product with it."""
    t, h = _inputs(6, 96, "fp32", "fp32", "full", True, size=1.0)
    rng = np.random.default_rng(1)

    def f(v):
        n, r = mx.block_norm(v["residual"], v["w_pre"], y=v["y"], w_post=v["w_post"], gate=v["gate"], res_scale=0.7,
                             eps=EPS)
        return float((n.double() * t["dn"].double()).sum() + (r.double() * t["dro"].double()).sum()), r
    _, r = f(t)
    out = mx.block_norm_grad(r, t["w_pre"], t["dn"], d_residual_out=t["dro"], y=t["y"], w_post=t["w_post"],
                             gate=t["gate"], res_scale=0.7, eps=EPS)
    step = 2.0 ** -8
    for key, g in zip(("residual", "w_pre", "y", "w_post", "gate"), out):
        d = torch.from_numpy(rng.standard_normal(g.shape)).float().cuda()
        up, down = ({**t, key: t[key] + sign * step * d} for sign in (1, -1))
        slope = (f(up)[0] - f(down)[0]) / (2 * step)
        # central difference: third-order term of order step^2 of the function's scale, and the rounding of the
        # 2 * 576 outputs of size below 16, U each, over 2 * step
        scale = float(torch.linalg.vector_norm(g) * torch.linalg.vector_norm(d))
        assert abs(slope - float((g * d).sum())) <= 64 * step ** 2 * max(scale, 1.0) + 2 * 576 * 16 * U / (2 * step), key


def test_grad_is_the_same_every_time(mx):
    t, h = _inputs(2500, 264, "bf16", "bf16", "channel", True)
    first = _grad(mx, t, h, "bf16", "bf16")
    for _ in range(3):
        again = _grad(mx, t, h, "bf16", "bf16")
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("H", [9, 12, 15, 70, 1001, 4099, 8189, 8200, 12347])
@pytest.mark.parametrize("name,res_name", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_rows_that_start_anywhere(mx, H, name, res_name, gate):
    """Widths that are no whole number of 16-byte pieces, more rows than workgroups hold at once."""
    T = 300 if H < 2000 else 5
    _forward(mx, T, H, name, res_name, gate, True)
    t, h = _inputs(T, H, name, res_name, gate, True)
    _grad(mx, t, h, name, res_name)


@pytest.mark.parametrize("shift", [1, 2, 5])
def test_views_at_any_alignment(mx, shift):
    """Buffers off 16 bytes give the bits of aligned ones, and nothing around them is written."""
    t, _ = _inputs(37, 520, "bf16", "fp32", "full", True)

    def off(v):
        buf = torch.full((v.numel() + 16,), 7.0, dtype=v.dtype, device="cuda")
        view = buf[shift:shift + v.numel()].view(v.shape)
        view.copy_(v)
        return buf, view
    want = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    grad = mx.block_norm_grad(want[1], t["w_pre"], t["dn"], d_residual_out=t["dro"], y=t["y"], w_post=t["w_post"],
                              gate=t["gate"], eps=EPS)
    u = {k: off(v)[1] for k, v in t.items()}
    outs = [off(torch.zeros_like(v)) for v in (want[0], want[1], grad[0], grad[2])]
    mx.block_norm(u["residual"], u["w_pre"], y=u["y"], w_post=u["w_post"], gate=u["gate"], eps=EPS,
                  normed=outs[0][1], residual_out=outs[1][1])
    g = mx.block_norm_grad(outs[1][1], u["w_pre"], u["dn"], d_residual_out=u["dro"], y=u["y"], w_post=u["w_post"],
                           gate=u["gate"], eps=EPS, d_residual=outs[2][1], d_y=outs[3][1])
    for (buf, view), ref in zip(outs, (want[0], want[1], grad[0], grad[2])):
        assert torch.equal(view, ref)
        assert (buf[:shift] == 7).all() and (buf[shift + view.numel():] == 7).all()
    assert all(torch.equal(g[i], grad[i]) for i in (1, 3, 4))


def test_more_than_2_to_the_31_elements(mx):
    """Offsets past 32 bits: the last rows of 300,001 x 7168 as the same rows alone give them."""
    T, H, n = 300001, 7168, 5
    t, _ = _inputs(n, H, "bf16", "bf16", "token", True)
    big = {}
    for k in ("y", "residual", "dn", "dro"):
        big[k] = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        big[k][-n:] = t[k]
    gate = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    gate[-n:] = t["gate"]
    a = mx.block_norm(big["residual"], t["w_pre"], y=big["y"], w_post=t["w_post"], gate=gate, eps=EPS)
    b = mx.block_norm(t["residual"], t["w_pre"], y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    assert all(torch.equal(x[-n:], y) and not x[:-n].any() for x, y in zip(a, b))
    g = mx.block_norm_grad(a[1], t["w_pre"], big["dn"], d_residual_out=big["dro"], y=big["y"], w_post=t["w_post"],
                           gate=gate, eps=EPS)
    r = mx.block_norm_grad(b[1], t["w_pre"], t["dn"], d_residual_out=t["dro"], y=t["y"], w_post=t["w_post"],
                           gate=t["gate"], eps=EPS)
    assert all(torch.equal(g[i][-n:], r[i]) and not g[i][:-n].any() for i in (0, 2, 4))
    # the column sums: the same five terms among zeros, joined in another order: two sums of five, each off by at
    # most four halves of a step of the sum of the terms' sizes
    rh = np.abs(f64(b[1])) / _rms(f64(b[1]))
    yh = np.abs(f64(t["y"])) / _rms(f64(t["y"]))
    du = np.abs(f64(t["gate"]) * f64(r[0]))
    for i, mass in ((1, np.abs(f64(t["dn"])) * rh), (3, du * yh)):
        within(g[i], f64(r[i]), 1.02 * 8 * U * mass.sum(0))


# rows of more than one piece per thread (beyond 8192 elements, in fp32 4096), more of them than workgroups: every
# workgroup goes through its sums' LDS and its one row buffer several times
LONG = [(300, 8200, "bf16", "bf16"), (530, 16384, "bf16", "fp32"), (300, 12345, "fp16", "fp16"), (530, 16383, "fp16", "fp32"),
        (530, 4100, "fp32", "fp32"), (300, 8192, "fp32", "fp32"), (270, 16384, "fp32", "fp32"), (300, 9001, "fp32", "fp32")]
KINDS = [("none", False), ("channel", True), ("token", True), ("token", False), ("full", True)]
LONG = [shape + KINDS[(i + j) % 5] for i, shape in enumerate(LONG) for j in (0, 2)]      # each shape with two kinds


@pytest.mark.parametrize("T,H,name,res_name,gate,post", LONG)
def test_forward_of_many_long_rows(mx, T, H, name, res_name, gate, post):
    _forward(mx, T, H, name, res_name, gate, post)


@pytest.mark.parametrize("T,H,name,res_name,gate,post", LONG)
def test_grad_of_many_long_rows(mx, T, H, name, res_name, gate, post):
    t, h = _inputs(T, H, name, res_name, gate, post)
    _grad(mx, t, h, name, res_name)


@pytest.mark.parametrize("T,H", [(530, 8200), (300, 16384)])
def test_parts_of_many_long_rows(mx, T, H):
    """Without the block, without the next norm: one sum a row, or none, and a barrier that stands for the other."""
    t, h = _inputs(T, H, "bf16", "bf16", "channel", True)
    n, _ = mx.block_norm(t["residual"], t["w_pre"], eps=EPS)
    ref, _ = around.block_norm(h["residual"], h["w_pre"], eps=EPS)
    within(n, ref, 1.02 * (np.abs(ref) * (depth(H) * U / 2 + 8 * U) + rounded(ref, "bf16")))
    none, added = mx.block_norm(t["residual"], None, y=t["y"], w_post=t["w_post"], gate=t["gate"], eps=EPS)
    assert none is None
    _, r, _, er = _bounds({**h, "w_pre": None}, 1.0)
    within(added, r, 1.02 * (er + rounded(r, "bf16")))

    def cut(*names):
        return {k: None if k in names else v for k, v in t.items()}, {k: None if k in names else v for k, v in h.items()}
    _grad(mx, *cut("y", "w_post", "gate"), "bf16", "bf16")
    _grad(mx, *cut("w_pre", "dn"), "bf16", "bf16")
