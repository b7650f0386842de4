"""Linear layers of unquantised activations with 4-bit weights on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

from around_util import DTYPES, U, f64, half_step, pair, within
from oracle import beside as o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def weights(rng, N, K, fmt, group, name, zeros, lo=118, hi=126):
    """(device arguments w, w_s, zeros; values and magnitudes in 64 bits)."""
    w = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
    z = rng.integers(0, 16, size=(N, K // group)).astype(np.uint8) if zeros else None
    if fmt == "mxfp4":
        s = rng.integers(lo, hi, size=(N, K // group)).astype(np.uint8)
        sd, sr = torch.from_numpy(s).cuda(), s
    else:
        sd, sr = pair(0.01 * (1 + rng.random((N, K // group))) * rng.choice([-1, 1], (N, K // group)), name)
    v, m = o.w4_weights(w, sr, z)
    return (torch.from_numpy(w).cuda(), sd, None if z is None else torch.from_numpy(z).cuda()), v, m


def bound(xr, m, ref, name):
    """The matrix cores' sums: 32 products, then the groups', every add off by at most a whole step (2 U) of the sum of
    the magnitudes so far, the scale's product and the splits of K by as much again; one rounding."""
    K = xr.shape[1]
    depth = 32 + K / 32 + 40
    return 2 * U * depth * (np.abs(xr) @ m.T) + half_step(name) * np.abs(ref) * (1 + 2 ** -7) + 2.0 ** -25


FORMS = [("mxfp4", 32, False), ("int4", 32, True), ("int4", 64, False), ("int4", 128, True), ("int4", 128, False)]


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 16, 256), (2, 17, 384), (3, 96, 1024), (4, 1000, 512), (5, 33, 128),
                                   (8, 256, 7168), (15, 100, 640), (16, 64, 2048), (17, 65, 256), (31, 48, 896), (33, 130, 1152),
                                   (48, 31, 512), (64, 200, 1024), (65, 128, 384), (100, 257, 640), (129, 96, 256),
                                   (200, 300, 1408), (257, 513, 384), (300, 128, 256), (512, 260, 768)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_sizes(mx, M, N, K, name):
    rng = np.random.default_rng(M * 7 + N)
    x, xr = pair(rng.standard_normal((M, K)), name)
    for fmt, group, zeros in FORMS:
        (w, s, z), v, m = weights(rng, N, K, fmt, group, name, zeros)
        y = mx.w4_linear(x, w, s, z)
        ref = xr @ v.T
        assert y.shape == (M, N) and y.dtype == DTYPES[name]
        within(y, ref, bound(xr, m, ref, name), (fmt, group, zeros))


@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 288, 2080, 4128])
@pytest.mark.parametrize("M", [1, 7, 20, 70, 300])
def test_short_last_steps(mx, M, K):
    """Widths that are no multiple of 128: what stands behind a row (the next row, or nothing) has no part."""
    rng = np.random.default_rng(K + M)
    x, xr = pair(rng.standard_normal((M, K)), "bf16")
    for fmt, group in (("mxfp4", 32), ("int4", 32), ("int4", 64)):
        if K % group:
            continue
        (w, s, z), v, m = weights(rng, 50, K, fmt, group, "bf16", fmt == "int4")
        if fmt == "mxfp4":
            sn = s.clone()
            sn[1::2] = 255                             # the rows between are NaN
            y = mx.w4_linear(x, w, sn)
            assert torch.isnan(y[:, 1::2]).all()
            ref = xr @ v[::2].T
            within(y[:, ::2].contiguous(), ref, bound(xr, m[::2], ref, "bf16"))
        y = mx.w4_linear(x, w, s, z)
        ref = xr @ v.T
        within(y, ref, bound(xr, m, ref, "bf16"), fmt)


@pytest.mark.parametrize("M", [1, 6, 40, 130, 400])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_strides(mx, M, name):
    """x and y as column ranges, of one matrix too; what stands beside them stays."""
    rng = np.random.default_rng(M)
    K, N = 256, 41
    wide, wr = pair(rng.standard_normal((M, 800)), name)
    (w, s, z), v, m = weights(rng, N, K, "int4", 64, name, True)
    xr = wr[:, 80:80 + K]
    ref = xr @ v.T
    for at in (400, 401, 759):
        y = wide.clone()
        got = mx.w4_linear(y[:, 80:80 + K], w, s, z, out=y[:, at:at + N])
        assert got.data_ptr() == y[:, at:].data_ptr()
        within(y[:, at:at + N].contiguous(), ref, bound(xr, m, ref, name))
        rest = [c for c in range(800) if not at <= c < at + N]
        assert torch.equal(y[:, rest], wide[:, rest])
    with pytest.raises(mx.MxError, match="multiple of 8"):
        y = torch.zeros((M + 1, 260 + 1), dtype=DTYPES[name], device="cuda")
        mx.w4_linear(y[:, :K], w, s, z)


@pytest.mark.parametrize("M", [1, 5, 64, 300])
def test_scales_of_the_whole_range(mx, M):
    """E8M0 scales from 2^-127 to 2^127, far outside fp16: the fp32 sums carry them."""
    K, N = 128, 256
    rng = np.random.default_rng(1)
    w = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
    s = np.zeros((N, 4), np.uint8)
    s[:, 0] = np.arange(N)
    s[:, 1:] = np.arange(N)[:, None]
    for name, small in (("bf16", 2.0 ** -60), ("fp16", 2.0 ** -10)):
        x, xr = pair(small * rng.standard_normal((M, K)), name)
        v, m = o.w4_weights(w, s)
        with np.errstate(all="ignore"):
            ref = xr @ v.T
        y = f64(mx.w4_linear(x, torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()))
        assert np.isnan(y[:, 255]).all()
        top = torch.finfo(DTYPES[name]).max
        inside = np.abs(ref) < top * 0.99
        inside[:, 255] = False
        tiny = 2.0 ** -132 if name == "bf16" else 2.0 ** -24     # below the smallest normal: a step of the subnormals
        tol = 2 * U * 80 * (np.abs(xr) @ np.nan_to_num(m).T) + half_step(name) * np.abs(ref) * 1.01 + tiny
        assert (np.abs(y - ref)[inside] <= tol[inside]).all()
        far = np.abs(ref) > top * 1.01
        far[:, 255] = False
        assert (np.isinf(y[far]) & (np.sign(y[far]) == np.sign(ref[far]))).all()


@pytest.mark.parametrize("M", [1, 6, 14, 30, 64, 300])
@pytest.mark.parametrize("size", [-60, 40, 120])
def test_scales_that_are_bf16_numbers(mx, M, size):
    """Bytes of up to 252, whose products with codes bf16 holds, and no other: from subnormal weights with large
    activations to the largest."""
    K, N = 256, 253
    rng = np.random.default_rng(2)
    w = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
    s = np.tile(np.arange(N)[:, None], (1, K // 32)).astype(np.uint8)
    x, xr = pair(2.0 ** size * rng.standard_normal((M, K)), "bf16")
    v, m = o.w4_weights(w, s)
    y = f64(mx.w4_linear(x, torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda()))
    ref, most = xr @ v.T, np.abs(xr) @ m.T
    inside = most < torch.finfo(torch.float32).max / 2
    tol = 2 * U * 80 * most + half_step("bf16") * np.abs(ref) * 1.01 + 2.0 ** -132
    assert inside.sum() > 100 * M and (np.abs(y - ref)[inside] <= tol[inside]).all()


@pytest.mark.parametrize("M", [1, 12, 70, 300])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_activations_that_are_not_finite(mx, M, bad):
    rng = np.random.default_rng(2)
    xr = rng.standard_normal((M, 384))
    xr[M // 2, 200] = bad
    for name in ("bf16", "fp16"):
        x, _ = pair(xr, name)
        for fmt, group, zeros in FORMS:
            (w, s, z), v, m = weights(rng, 70, 384, fmt, group, name, zeros)
            y = mx.w4_linear(x, w, s, z)
            hit = torch.zeros(M, dtype=torch.bool, device="cuda")
            hit[M // 2] = True
            assert not torch.isfinite(y[hit]).any() and torch.isfinite(y[~hit]).all(), (fmt, group)


def test_unit_rows_give_the_weights(mx):
    """x = the unit vectors: y is the weights themselves, each code, scale and zero point."""
    rng = np.random.default_rng(3)
    K, N = 256, 48
    for name in ("bf16", "fp16"):
        x = torch.eye(K, dtype=DTYPES[name], device="cuda")
        for fmt, group, zeros in FORMS:
            (w, s, z), v, _ = weights(rng, N, K, fmt, group, name, zeros)
            want = torch.from_numpy(v.T.copy()).to(DTYPES[name])
            for rows in (slice(0, 1), slice(3, 7), slice(0, 60), slice(0, K)):
                assert torch.equal(mx.w4_linear(x[rows], w, s, z).cpu(), want[rows]), (name, fmt, group)


def test_no_tokens(mx):
    w, s = torch.zeros((8, 32), dtype=torch.uint8, device="cuda"), torch.ones((8, 2), dtype=torch.bfloat16, device="cuda")
    assert mx.w4_linear(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, s).shape == (0, 8)


def test_many_tokens_run_to_run(mx):
    """A prompt's size: the same bits twice, the oracle's on a sample of rows and columns."""
    rng = np.random.default_rng(9)
    M, N, K = 1111, 2064, 1952
    x, xr = pair(rng.standard_normal((M, K)), "bf16")
    for fmt, group in (("mxfp4", 32), ("int4", 32)):
        (w, s, z), v, m = weights(rng, N, K, fmt, group, "bf16", False)
        y = mx.w4_linear(x, w, s, z)
        for _ in range(2):
            assert torch.equal(y, mx.w4_linear(x, w, s, z))
        ref = xr @ v.T
        within(y, ref, bound(xr, m, ref, "bf16"))


def test_past_2_to_the_31(mx):
    """Rows of x and y whose elements lie beyond 2^31."""
    rng = np.random.default_rng(4)
    M, K, N = 3, 256, 64
    stride = (1 << 30)
    big = torch.empty((M, stride), dtype=torch.bfloat16, device="cuda")
    x, xr = pair(rng.standard_normal((M, K)), "bf16")
    big[:, 512:512 + K] = x
    (w, s, z), v, m = weights(rng, N, K, "mxfp4", 32, "bf16", False)
    y = mx.w4_linear(big[:, 512:512 + K], w, s, out=big[:, :N])
    ref = xr @ v.T
    within(y.contiguous(), ref, bound(xr, m, ref, "bf16"))


@pytest.mark.parametrize("M", [3, 11, 20, 70, 140])
@pytest.mark.parametrize("K", [40032, 33024])
def test_long_rows(mx, M, K):
    """More columns than a workgroup has the scales of at a time; rows of scales at odd addresses (K 40032) and not."""
    rng = np.random.default_rng(M)
    N = 37
    x, xr = pair(rng.standard_normal((M, K)), "bf16")
    for fmt, group, zeros in (("mxfp4", 32, False), ("int4", 32, True), ("int4", 64, False), ("int4", 128, True)):
        if K % group:
            continue
        (w, s, z), v, m = weights(rng, N, K, fmt, group, "bf16", zeros)
        y = mx.w4_linear(x, w, s, z)
        ref = xr @ v.T
        within(y, ref, bound(xr, m, ref, "bf16"), (fmt, group))


@pytest.mark.parametrize("M", [4, 30, 90])
def test_scales_and_zeros_at_odd_addresses(mx, M):
    """Scales that start one element, zero points and E8M0 bytes that start one byte behind a multiple of 4."""
    rng = np.random.default_rng(M)
    K, N = 1024, 50
    x, xr = pair(rng.standard_normal((M, K)), "fp16")
    for fmt, group, zeros in (("mxfp4", 32, False), ("int4", 32, True), ("int4", 128, True)):
        (w, s, z), v, m = weights(rng, N, K, fmt, group, "fp16", zeros)
        def odd(a):
            r = torch.empty(a.numel() + 1, dtype=a.dtype, device="cuda")[1:].view(a.shape)
            return r.copy_(a)
        y = mx.w4_linear(x, w, odd(s), None if z is None else odd(z))
        ref = xr @ v.T
        within(y, ref, bound(xr, m, ref, "fp16"), (fmt, group))


def test_tokens_far_apart(mx):
    """More than 2^24 elements from token to token, more than 16 tokens."""
    rng = np.random.default_rng(6)
    M, K, N = 18, 512, 64
    big = torch.empty((M, (1 << 24) + 8), dtype=torch.bfloat16, device="cuda")
    x, xr = pair(rng.standard_normal((M, K)), "bf16")
    big[:, 64:64 + K] = x
    (w, s, z), v, m = weights(rng, N, K, "int4", 64, "bf16", True)
    y = mx.w4_linear(big[:, 64:64 + K], w, s, z)
    ref = xr @ v.T
    within(y, ref, bound(xr, m, ref, "bf16"))
