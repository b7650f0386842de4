"""mx_lora_add against the fp64 oracle."""

import numpy as np
import pytest
import torch

from around_util import U, f64, half_step, pair, rounded, within
from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def _plan(mx, adapter, n):
    off, row_token, _ = mx.moe_sort(torch.from_numpy(adapter.astype(np.int32).reshape(-1, 1)).cuda(), n)
    return off, row_token


def _bound(y, x, a, b, adapter, scale, name):
    """v = A x: K products and additions in fp32; its two 16-bit halves keep 2^-17 of it (2^-21 in fp16, where
    the halves of the row's smallest values may be subnormal: 2^-23 of the row's largest). Then 2 R more."""
    tol = np.zeros_like(y)
    K, R = a.shape[2], a.shape[1]
    keep = 2.0 ** -17 if name == "bf16" else 2.0 ** -21
    for t, i in enumerate(adapter):
        if 0 <= i < a.shape[0]:
            s = 1.0 if scale is None else abs(scale[i])
            v = np.abs(a[i] @ x[t])
            ev = (K + 8) * U * (np.abs(a[i]) @ np.abs(x[t]))
            ev = ev + keep * (v + ev) + (2.0 ** -23 * (v + ev).max() if name == "fp16" else 0.0)
            tol[t] = s * (np.abs(b[i]) @ (ev + (2 * R + 8) * U * v)) + 4 * U * np.abs(y[t])
    return tol


def _case(mx, M, K, N, R, n, adapter, name, seed, scaled=True, keep_scale=1.0):
    rng = np.random.default_rng(seed)
    x, x64 = pair(rng.standard_normal((M, K)), name)
    y, y64 = pair(rng.standard_normal((M, N)), name)
    a, a64 = pair(rng.standard_normal((n, R, K)) * K ** -0.5, name)
    b, b64 = pair(rng.standard_normal((n, N, R)) * R ** -0.5, name)
    s, s64 = pair(rng.uniform(-2, 2, n), "fp32") if scaled else (None, None)
    got = mx.lora_add(y, x, a, b, *_plan(mx, adapter, n), scale=s)
    assert got is y
    ref = around.lora_add(y64, x64, a64, b64, adapter, s64)
    tol = _bound(y64, x64, a64, b64, adapter, s64, name)
    within(got, ref, 1.01 * (tol * (1 + half_step(name)) + rounded(ref, name)))
    bare = (adapter < 0) | (adapter >= n)
    assert np.array_equal(f64(got)[bare], y64[bare])


@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("M,K,N,R,n", [(1, 8, 8, 8, 1), (1, 256, 128, 64, 4), (3, 40, 72, 24, 2), (16, 128, 64, 16, 16),
                                       (17, 136, 200, 32, 3), (33, 512, 264, 128, 5), (64, 264, 128, 40, 64),
                                       (130, 104, 520, 72, 2), (200, 256, 136, 8, 1), (257, 64, 64, 96, 7)])
def test_lora(mx, M, K, N, R, n, name):
    rng = np.random.default_rng(M)
    _case(mx, M, K, N, R, n, rng.integers(-1, n + 1, size=M), name, M + K)


def test_without_scale_and_without_tokens(mx):
    _case(mx, 20, 64, 64, 16, 3, np.arange(20) % 4, "bf16", 1, scaled=False)
    _case(mx, 20, 64, 64, 16, 3, np.full(20, -1), "bf16", 2)            # no token has an adapter
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    a = torch.empty((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    y = mx.lora_add(x.clone(), x, a, torch.empty((2, 64, 8), dtype=torch.bfloat16, device="cuda"),
                    *_plan(mx, np.empty(0), 2))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("M,K,N,R,n", [(1, 7168, 1536, 64, 4), (64, 7168, 7168, 16, 32), (700, 7168, 1536, 128, 3),
                                       (300, 1536, 7168, 40, 100), (2100, 520, 1000, 24, 6),
                                       (2500, 256, 264, 128, 3), (2304, 1032, 64, 72, 4), (2100, 40, 72, 16, 2),
                                       (4500, 128, 64, 8, 512), (5000, 64, 136, 56, 1)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_whole_numbers_come_out_exactly(mx, M, K, N, R, n, name):
    """Small whole numbers keep every sum exact in fp32 and every v exact in its halves, so that the output is
    the exact sum, rounded once; real sizes, many requests."""
    rng = np.random.default_rng(R)
    x, x64 = pair(rng.integers(-2, 3, size=(M, K)), name)
    y, y64 = pair(rng.integers(-8, 9, size=(M, N)), name)
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), name)
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)) * 0.5, name)
    s, s64 = pair(2.0 ** rng.integers(-3, 1, size=n), "fp32")
    adapter = np.sort(rng.integers(-1, n, size=M))
    rng.shuffle(adapter[:M // 2])
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n), scale=s)
    ref = y64.copy()
    for i in range(n):
        t = np.nonzero(adapter == i)[0]
        ref[t] += s64[i] * ((x64[t] @ a64[i].T) @ b64[i].T)
    expect = torch.from_numpy(ref).to(y.dtype)
    assert torch.equal(y.cpu(), expect)


def test_column_ranges_of_wider_matrices(mx):
    """x a slice of columns; y one half of a stacked gate-and-up output, also inside the matrix that holds x."""
    rng = np.random.default_rng(9)
    M, K, N, R, n = 37, 72, 96, 16, 3
    adapter = rng.integers(-1, n, size=M)
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), "bf16")
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)), "bf16")
    wide, w64 = pair(rng.integers(-2, 3, size=(M, K + 2 * N + 16)), "bf16")
    x, y = wide[:, 8:8 + K], wide[:, K + 8 + N:K + 8 + 2 * N]
    ref = w64.copy()
    ref[:, K + 8 + N:K + 8 + 2 * N] = around.lora_add(w64[:, K + 8 + N:K + 8 + 2 * N], w64[:, 8:8 + K], a64, b64, adapter)
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    assert torch.equal(wide.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
    with pytest.raises(mx.MxError, match="overlaps x"):
        mx.lora_add(wide[:, 16:16 + N], x, a, b, *_plan(mx, adapter, n))


@pytest.mark.parametrize("name,big", [("bf16", 1e30), ("fp16", 60000.0)])
def test_large_and_non_finite_values_stay_in_their_rows(mx, name, big):
    """v beyond fp16's range, and NaN and infinities of one token, leave the other tokens alone."""
    rng = np.random.default_rng(2)
    M, K, N, R, n = 24, 64, 64, 16, 2
    adapter = np.arange(M) % n
    xv = rng.integers(-2, 3, size=(M, K)).astype(np.float64)
    xv[5] = big
    x, x64 = pair(xv, name)
    xn = x.clone()
    xn[6, 3], xn[7, 9] = float("nan"), float("inf")
    # |A| <= 2^-14: the product of a large x with it stays in range of y
    a, a64 = pair(rng.integers(0, 2, size=(n, R, K)), name)
    b, b64 = pair(rng.integers(0, 2, size=(n, N, R)) * 2.0 ** -14, name)
    y0, y64 = pair(np.zeros((M, N)), name)
    plan = _plan(mx, adapter, n)
    clean = mx.lora_add(y0.clone(), x, a, b, *plan)
    dirty = mx.lora_add(y0.clone(), xn, a, b, *plan)
    ref = around.lora_add(y64, x64, a64, b64, adapter)
    tol = _bound(y64, x64, a64, b64, adapter, None, name)
    within(clean, ref, 1.01 * (tol * (1 + half_step(name)) + rounded(ref, name)))
    others = [t for t in range(M) if t not in (6, 7)]
    assert torch.equal(clean[others], dirty[others])
    assert not torch.isfinite(dirty[6]).all() and not torch.isfinite(dirty[7]).all()
    assert torch.isnan(dirty[6][b[0].sum(1) > 0]).any()


def test_more_than_2_to_the_31_elements(mx):
    """Offsets past 32 bits in x and y, whole numbers, only the last tokens with adapters."""
    M, K, N, R, n = 300001, 7168, 7200, 16, 2
    rng = np.random.default_rng(4)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    xt, x64 = pair(rng.integers(-2, 3, size=(40, K)), "bf16")
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), "bf16")
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)), "bf16")
    x[-40:] = xt
    adapter = np.full(M, -1)
    adapter[-40:] = np.arange(40) % 3 - 1
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    ref = around.lora_add(np.zeros((40, N)), x64, a64, b64, adapter[-40:])
    assert torch.equal(y[-40:].cpu(), torch.from_numpy(ref).to(torch.bfloat16)) and not y[:-40].any()


@pytest.mark.parametrize("M,busy", [(1, 0), (40, 1), (4100, 5), (4100, 3000), (4100, 0)])
def test_adapters_of_few_of_the_tokens(mx, M, busy):
    """Most tokens without an adapter, most adapters without a token, all of an adapter's tokens in one place."""
    K, N, R, n = 192, 136, 24, 300
    rng = np.random.default_rng(busy)
    x, x64 = pair(rng.integers(-2, 3, size=(M, K)), "fp16")
    y, y64 = pair(rng.integers(-8, 9, size=(M, N)), "fp16")
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), "fp16")
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)), "fp16")
    adapter = np.full(M, -1)
    adapter[M - busy:] = 297
    adapter[:min(busy, 2)] = (0, 299)[:min(busy, 2)]
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    ref = around.lora_add(y64, x64, a64, b64, adapter)
    assert torch.equal(y.cpu(), torch.from_numpy(ref).to(torch.float16))


@pytest.mark.parametrize("M,K,N,R,n", [(2100, 7176, 824, 24, 6), (2500, 256, 6480, 128, 3), (2304, 1032, 6256, 72, 4),
                                       (2100, 40, 7960, 16, 2), (4500, 128, 3608, 8, 70), (5000, 64, 3296, 56, 1),
                                       (70000, 136, 104, 40, 5)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_prompts_of_wide_rows(mx, M, K, N, R, n, name):
    """M (K + N) of 2^24 and more: the large tiles, at ranks, widths and shares that do not fill them."""
    test_whole_numbers_come_out_exactly(mx, M, K, N, R, n, name)


@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_prompts_of_wide_rows_in_ordinary_numbers(mx, name):
    rng = np.random.default_rng(12)
    _case(mx, 2100, 4104, 4000, 88, 3, rng.integers(-1, 4, size=2100), name, 13)


@pytest.mark.parametrize("busy", [0, 5, 63, 64, 65, 3000])
def test_prompts_with_adapters_of_few_of_the_tokens(mx, busy):
    """As test_adapters_of_few_of_the_tokens, in large tiles: one filled partly, exactly, and one row over."""
    M, K, N, R, n = 4100, 2056, 2048, 24, 60
    rng = np.random.default_rng(busy)
    x, x64 = pair(rng.integers(-2, 3, size=(M, K)), "bf16")
    y, y64 = pair(rng.integers(-8, 9, size=(M, N)), "bf16")
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), "bf16")
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)), "bf16")
    adapter = np.full(M, -1)
    adapter[M - busy:] = 57
    adapter[:min(busy, 2)] = (0, 59)[:min(busy, 2)]
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    ref = around.lora_add(y64, x64, a64, b64, adapter)
    assert torch.equal(y.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


@pytest.mark.parametrize("M,K,N,R,n", [(9000, 64, 2056, 16, 8), (21000, 32, 1096, 8, 4), (36000, 16, 520, 72, 2),
                                       (1500, 64, 5000, 8, 90)])
def test_more_tiles_than_one_round_of_workgroups(mx, M, K, N, R, n):
    test_whole_numbers_come_out_exactly(mx, M, K, N, R, n, "bf16")


@pytest.mark.parametrize("M,N,R,n", [(1, 72, 8, 1), (40, 136, 24, 3), (70, 264, 128, 2), (150, 64, 56, 1),
                                     (2100, 8000, 24, 3), (2050, 8200, 64, 2), (2200, 7800, 128, 2)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_where_the_adapter_cancels_the_projection(mx, M, N, R, n, name):
    """The inner product's low bits count: each column takes one rank, y holds that product rounded to its type
    with the other sign, and what is left is exact. v is a whole number of up to 22 bits times 2^-s, s up to 14 from
    rank to rank, so that fp16's pieces reach its smallest subnormals (2^22 2^-s next to 1)."""
    K = 8
    rng = np.random.default_rng(M + R)
    xv = np.zeros((M, K))
    for i, size in enumerate((1.0, 2.0 ** 7, 2.0 ** 15)):
        xv[:, i] = size * rng.choice([-1, 1], size=M)
    step = 2.0 ** -rng.integers(0, 15, size=(n, R, 1))
    x, x64 = pair(xv, name)
    a, a64 = pair(rng.integers(-127, 128, size=(n, R, K)) * step, name)
    bv = np.zeros((n, N, R))
    bv[:, np.arange(N), np.arange(N) % R] = rng.choice([-1, 1], size=(n, N))
    b, b64 = pair(bv, name)
    adapter = rng.integers(0, n, size=M)
    scale, s64 = pair(np.full(n, 2.0 ** -8), "fp32")
    delta = np.zeros((M, N))
    for i in range(n):
        t = adapter == i
        delta[t] = 2.0 ** -8 * ((x64[t] @ a64[i].T) @ b64[i].T)          # exact in 64 bits
    y, y64 = pair(-delta, name)
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n), scale=scale)
    left = torch.from_numpy(y64 + delta)
    assert (left != 0).any()
    assert torch.equal(y.cpu(), left.to(y.dtype))


@pytest.mark.parametrize("M,N,R,n", [(1, 72, 8, 1), (40, 136, 24, 3), (70, 264, 128, 2), (150, 64, 56, 1),
                                     (2100, 8000, 24, 3), (2050, 8200, 64, 2), (2200, 7800, 128, 2)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_where_two_ranks_cancel(mx, M, N, R, n, name):
    """Each column takes the difference of two ranks' v, whole numbers of up to 22 bits times 2^-s that differ in the
    last 8 only: the difference fits either type and comes out exactly."""
    K = 8
    rng = np.random.default_rng(M + R + 1)
    xv = np.zeros((M, K))
    for i, size in enumerate((1.0, 2.0 ** 7, 2.0 ** 15)):
        xv[:, i] = size * rng.choice([-1, 1], size=M)
    av = rng.integers(-127, 128, size=(n, R, K)).astype(np.float64)
    av[:, 1::2, 1:] = av[:, 0::2, 1:]
    av *= np.repeat(2.0 ** -rng.integers(0, 15, size=(n, R // 2, 1)), 2, axis=1)
    x, x64 = pair(xv, name)
    a, a64 = pair(av, name)
    bv = np.zeros((n, N, R))
    at = 2 * (np.arange(N) % (R // 2))
    bv[:, np.arange(N), at], bv[:, np.arange(N), at + 1] = 1, -1
    b, b64 = pair(bv, name)
    adapter = rng.integers(0, n, size=M)
    y, y64 = pair(np.zeros((M, N)), name)
    for i in range(n):
        t = adapter == i
        y64[t] = (x64[t] @ a64[i].T) @ b64[i].T                           # exact in 64 bits
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    assert (y64 != 0).any()
    assert np.array_equal(f64(y), y64)


@pytest.mark.parametrize("M,N,R", [(1, 72, 8), (40, 136, 24), (70, 264, 56), (90, 80, 72), (2100, 7992, 16),
                                   (2050, 8200, 64), (2200, 7800, 128)])
@pytest.mark.parametrize("name", ["bf16", "fp16"])
@pytest.mark.parametrize("where", ["A", "B"])
def test_infinite_weights(mx, M, N, R, name, where):
    """Infinities and NaN in A or in B, next to v of one and of more pieces, zeros and large values: +-inf and NaN where
    the formula has them, the rest the exact sum rounded once."""
    K, n = 64, 3
    rng = np.random.default_rng(R)
    xv = rng.integers(-2, 3, size=(M, K)).astype(np.float64)
    xv[::3] *= 2.0 ** rng.integers(-6, 7, size=K)           # v of many bits
    xv[1::5] = 0.0                                          # v = 0: 0 * inf is NaN
    xv[:, 7], xv[:, 8] = 1.0, 2.0 ** 6
    av, bv = rng.integers(-1, 2, size=(n, R, K)).astype(np.float64), rng.integers(-1, 2, size=(n, N, R)) * 0.25
    av[:, :, 7] = 0.0
    if where == "A":
        # an adapter with an infinite and a large v, of which the columns take some, and one with v that is NaN
        av[1, 2, 7], av[1, 3, 7] = -np.inf, 2.0 ** (15 if name == "fp16" else 100)
        av[1, 3, 8], av[2, 4, 9] = av[1, 3, 7], np.nan
    else:
        bv[1, 3, 5], bv[1, 11, 0], bv[1, 11, 1], bv[1, 20, 2] = np.inf, -np.inf, np.inf, np.nan
        bv[1, N - 1], bv[1, N - 2, R - 1] = np.inf, -np.inf
    x = pair(xv, name)[0]
    a = pair(av, name)[0]
    b = pair(bv, name)[0]
    y = pair(rng.integers(-4, 5, size=(M, N)), name)[0]
    adapter = (np.arange(M) // 2 + 1) % n
    ref, xd, ad, bd = y.double(), x.double(), a.double(), b.double()      # product by product: 0 * inf is NaN
    for i in range(n):
        t = torch.from_numpy(np.nonzero(adapter == i)[0]).cuda()
        v = sum(xd[t, k, None] * ad[i, :, k] for k in range(K))
        ref[t] += sum(v[:, r, None] * bd[i, :, r] for r in range(R))
    ref = ref.to(y.dtype)
    mx.lora_add(y, x, a, b, *_plan(mx, adapter, n))
    assert torch.isinf(ref).any() and torch.isnan(ref).any()
    assert torch.equal(y.isnan(), ref.isnan())
    assert torch.equal(y[~ref.isnan()], ref[~ref.isnan()])
