"""The oracle of the operators beside the experts: its gradients against differences, its formats against the
quantiser oracle and hand-worked values."""

import numpy as np
import pytest

from oracle import beside as o
from oracle import mx_oracle


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("what", ["weights", "loss", "both"])
def test_gate_gradient_against_differences(score, renorm, what):
    rng = np.random.default_rng(3)
    T, E, k, scale, coef = 6, 7, 3, 2.5, 0.3
    z = rng.standard_normal((T, E))
    z[1, 2] = -np.inf
    seq_off = [0, 2, 2, 5]                        # an empty sequence, a token behind the last
    ids, _ = o.moe_gate(z, k, score)
    ids[4] = [1, 1, -1]                           # the same expert twice, a slot without one
    _, counts = o.moe_balance(z, ids, seq_off, score, coef)
    d_w, d_loss = rng.standard_normal((T, k)), rng.standard_normal(3)

    def value(z):
        total = 0.0
        if what != "loss":
            for t in range(T):
                s = o.scores(z[t], score)
                w = np.array([s[e] if e >= 0 else 0.0 for e in ids[t]])
                total += (scale * (w / w.sum() if renorm else w) * d_w[t]).sum()
        if what != "weights":
            for q in range(3):
                a, b = seq_off[q], seq_off[q + 1]
                if b > a:
                    p = sum(o.shares(z[t], score) for t in range(a, b))
                    total += d_loss[q] * coef * E / (k * (b - a) ** 2) * (counts[q] * p).sum()
        return total
    kw = {}
    if what != "loss":
        kw["d_w"] = d_w
    if what != "weights":
        kw.update(counts=counts, d_loss=d_loss)
    got, size = o.moe_gate_grad(z, ids, seq_off=seq_off, score=score, renorm=renorm, scale=scale, coef=coef, **kw)
    assert (np.abs(got) <= size * (1 + 1e-12)).all()
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if z[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((value(up) - value(down)) / (2 * h) - got[t, e]) < 1e-7, (t, e)


def test_gate_order_and_what_is_off():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [-np.inf] * 5, [-np.inf, 0.5, -np.inf, -np.inf, 0.25]])
    ids, w = o.moe_gate(z, 3, renorm=True)
    assert ids.tolist() == [[1, 2, 4], [-1, -1, -1], [1, 4, -1]]
    assert np.allclose(w.sum(1), [1, 0, 1]) and w[2, 2] == 0
    ids, _ = o.moe_gate(z, 2, "sigmoid", bias=np.array([9.0, 0, 0, 99, 0]))
    assert ids.tolist() == [[0, 1], [-1, -1], [1, 4]]


def test_balance_of_even_load_is_its_coefficient():
    E, k = 6, 2
    ids = np.array([[0, 1], [2, 3], [4, 5]])
    for score in ("softmax", "sigmoid"):
        loss, counts = o.moe_balance(np.zeros((3, E)), ids, score=score, coef=0.25)
        assert np.allclose(loss, 0.25) and (counts == 1).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_rows_quantise_as_the_quantiser_does(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)) * np.exp(4 * rng.standard_normal((40, 1)))
    x[3] = 0
    x[5, 7] = np.inf
    x[6] = rng.choice([0.25, -0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 64)
    x[7, :8] = -1e-39
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)      # bf16 by cutting off
    exact = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    codes, scales = o.quantize_rows(exact, fmt)
    ref = mx_oracle.mxfp4_quantize(bits) if fmt == "mxfp4" else mx_oracle.mxfp8_quantize(bits)
    assert (scales == ref[1]).all() and (codes == ref[0]).all()
    back = o.dequantize_rows(codes, scales, fmt)
    again = o.quantize_rows(back[[i for i in range(40) if i != 5]], fmt)
    assert np.array_equal(o.dequantize_rows(*again, fmt), back[[i for i in range(40) if i != 5]])


def test_w4_values():
    w = np.array([[0x10, 0x98, 0xF7, 0x2A]], np.uint8)
    v, _ = o.w4_weights(np.tile(w, (1, 4)), np.array([[128]], np.uint8))
    assert v[0, :8].tolist() == [0, 1, -0.0, -1, 12, -12, -2, 2]
    v, m = o.w4_weights(np.tile(w, (1, 4)), np.array([[0.5]]), np.array([[3]], np.uint8))
    assert v[0, :8].tolist() == [-1.5, -1, 2.5, 3, 2, 6, 3.5, -0.5]
    assert m[0, :8].tolist() == [1.5, 2, 5.5, 6, 5, 9, 6.5, 2.5]
    v, _ = o.w4_weights(np.tile(w, (1, 4)), np.array([[2.0]]))
    assert v[0, :8].tolist() == [-16, -14, 0, 2, -2, 14, 4, -12]


def test_cache_reads_what_was_written():
    rng = np.random.default_rng(2)
    for fmt, wide in (("mxfp8", 64), ("mxfp4", 32)):
        codes, scales = np.full((4, 3, wide), 7, np.uint8), np.full((4, 3, 2), 9, np.uint8)
        x = rng.standard_normal((5, 64))
        c, s = o.cache_write(x, [11, 3, -1, 12, 0], codes, scales, fmt)
        assert (c.reshape(12, wide)[[1, 2, 4, 5, 6, 7, 8, 9, 10]] == 7).all() and not (c.reshape(12, wide)[11] == 7).all()
        out = np.full((6, 64), 5.0)
        got = o.cache_read(c, s, np.array([[3], [1]]), [1, 4, 5], out, fmt)
        assert (got[[0, 5]] == 5).all()
        rows = o.dequantize_rows(*o.quantize_rows(x, fmt), fmt)
        assert np.array_equal(got[3], rows[0]) and np.array_equal(got[4], rows[1])
        assert (o.cache_read(c, s, np.array([[9], [-1]]), [0, 4, 5], out, fmt)[:5] == 0).all()
