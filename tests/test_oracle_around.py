"""The fp64 oracle of the operators around the experts: its sort against a plain one, its gradients against
differences of its own forward functions."""

import numpy as np
import pytest

from oracle import around

STEP = 2.0 ** -16


def _slope(f, v, d):
    return (f(v + STEP * d) - f(v - STEP * d)) / (2 * STEP)


def _close(slope, exact, scale):
    # central difference of a smooth function in float64: STEP^2 of its scale, and 2^-52 of it over STEP
    assert abs(slope - exact) <= 1e3 * scale * STEP ** 2 + 1e3 * scale * 2.0 ** -52 / STEP, (slope, exact)


def test_sort():
    rng = np.random.default_rng(0)
    ids = rng.integers(-2, 9, size=(40, 3))
    off, row_slot, slot_row = around.moe_sort(ids, 7)
    flat = ids.reshape(-1)
    assert off[-1] == ((flat >= 0) & (flat < 7)).sum() and off[0] == 0
    for e in range(7):
        mine = row_slot[off[e]:off[e + 1]]
        assert (flat[mine] == e).all() and (np.diff(mine) > 0).all()
    assert (row_slot[off[-1]:] == -1).all()
    for p, r in enumerate(slot_row.reshape(-1)):
        assert (r == -1) == (not 0 <= flat[p] < 7) and (r < 0 or row_slot[r] == p)


def test_unpermute_gradients():
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, 6, size=(20, 3))
    _, _, sr = around.moe_sort(ids, 5)
    ys, w, g = rng.standard_normal((60, 8)), rng.standard_normal((20, 3)), rng.standard_normal((20, 8))
    f = lambda ys, w: (around.moe_unpermute(ys, sr, w) * g).sum()
    dys, dw = around.moe_unpermute_grad(g, ys, sr, w, np.zeros_like(ys))
    for v, grad, fun in ((ys, dys, lambda v: f(v, w)), (w, dw, lambda v: f(ys, v))):
        d = rng.standard_normal(v.shape)
        _close(_slope(fun, v, d), (grad * d).sum(), 100.0)
    x, gx = rng.standard_normal((20, 8)), rng.standard_normal((60, 8))
    kept = np.zeros((60, 8))
    d = rng.standard_normal(x.shape)
    back = around.moe_unpermute(gx, sr)                       # of the permute
    _close(_slope(lambda v: (around.moe_permute(v, sr, kept) * gx).sum(), x, d), (back * d).sum(), 100.0)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradients(gate, post):
    rng = np.random.default_rng(2)
    T, H = 5, 12
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    v = {"residual": rng.standard_normal((T, H)), "w_pre": rng.standard_normal(H), "y": rng.standard_normal((T, H)),
         "w_post": rng.standard_normal(H) if post else None,
         "gate": None if shape is None else rng.standard_normal(shape)}
    dn, dro = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def f(v):
        n, r = around.block_norm(v["residual"], v["w_pre"], v["y"], v["w_post"], v["gate"], 0.7, 1e-3)
        return (n * dn).sum() + (r * dro).sum()
    _, r = around.block_norm(v["residual"], v["w_pre"], v["y"], v["w_post"], v["gate"], 0.7, 1e-3)
    g = around.block_norm_grad(r, v["w_pre"], dn, dro, v["y"], v["w_post"], v["gate"], 0.7, 1e-3)
    for key, name in (("residual", "d_residual"), ("w_pre", "dw_pre"), ("y", "d_y"), ("w_post", "dw_post"),
                      ("gate", "d_gate")):
        if v[key] is None:
            assert name not in g
            continue
        d = rng.standard_normal(v[key].shape)
        _close(_slope(lambda u: f({**v, key: u}), v[key], d), (g[name] * d).sum(), 100.0)


def test_lora_is_the_sum_over_adapters():
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((9, 6)), rng.standard_normal((9, 4))
    a, b, s = rng.standard_normal((3, 2, 6)), rng.standard_normal((3, 4, 2)), rng.standard_normal(3)
    adapter = np.array([0, -1, 2, 1, 1, 3, 0, 2, -5])
    ref = y.copy()
    for i in range(3):
        ref += s[i] * (adapter == i)[:, None] * (x @ a[i].T @ b[i].T)
    assert np.allclose(around.lora_add(y, x, a, b, adapter, s), ref, rtol=0, atol=1e-13)
