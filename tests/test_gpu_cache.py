"""The quantised cache on the GPU against the fp64 oracle: bytes as written, values as read."""

import numpy as np
import pytest
import torch

from around_util import DTYPES, pair
from oracle import beside as o

pytestmark = pytest.mark.gpu
FORMATS = ["mxfp8", "mxfp4"]


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def cache(rng, pages, page, width, fmt):
    codes = rng.integers(0, 256, size=(pages, page, width if fmt == "mxfp8" else width // 2)).astype(np.uint8)
    scales = rng.integers(100, 150, size=(pages, page, width // 32)).astype(np.uint8)
    return codes, scales


def same(got, ref, name):
    """Equal to ref rounded once to the type; a NaN where ref has one."""
    want = torch.from_numpy(ref).to(DTYPES[name])
    g = got.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan) and torch.equal(g[~nan], want[~nan])


@pytest.mark.parametrize("T,width,pages,page", [(1, 32, 1, 1), (1, 576, 3, 16), (5, 64, 4, 3), (33, 96, 9, 16), (64, 1024, 2, 64),
                                                (100, 160, 30, 7), (3, 8192, 2, 5)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
def test_write(mx, T, width, pages, page, fmt, name):
    rng = np.random.default_rng(T + width)
    codes, scales = cache(rng, pages, page, width, fmt)
    x, xr = pair(rng.standard_normal((T, width)) * np.exp(3 * rng.standard_normal((T, 1))), name)
    slots = rng.permutation(pages * page)[:T]
    slots = np.concatenate([slots, np.full(T - len(slots), -1)])      # more tokens than slots: padding
    rng.shuffle(slots)
    if T > 4:
        slots[2], slots[3] = -5, pages * page                         # neither is a slot
    c, s = dev(codes, torch.uint8), dev(scales, torch.uint8)
    got = mx.cache_write(fmt, x, dev(slots), c, s)
    assert got[0] is c and got[1] is s
    rc, rs = o.cache_write(xr, slots, codes, scales, fmt)
    assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
def test_every_value_is_rounded_as_said(mx, fmt, name):
    """Blocks that start with a value fixing the scale, then every value next to a border of the grid and its
    neighbours in the type, both signs, at scales up and down the range; zeros, subnormals, infinities and NaN."""
    dt = DTYPES[name]
    grid = o._grid(fmt)
    mid = (grid[1:] + grid[:-1]) / 2
    near = torch.tensor(np.concatenate([grid, mid])).to(dt)
    bits = torch.int32 if dt == torch.float32 else torch.int16
    around = torch.cat([near, (near.view(bits) + 1).view(dt), (near.view(bits) - 1).clamp(min=0).view(dt)]).to(torch.float64)
    lo, hi = {"bf16": (-126, 110), "fp16": (-14, 5), "fp32": (-126, 110)}[name]
    rows = []
    for e in [lo, lo + 1, lo + 7, 0, 1, -3, hi]:
        v = around.numpy() * 2.0 ** e
        v = v[v <= grid[-1] * 1.1 * 2.0 ** e]
        for sign in (1, -1):
            for i in range(0, len(v), 31):
                rows.append(np.concatenate([[grid[-1] * 2.0 ** e], sign * v[i:i + 31]]))
    block = np.zeros((len(rows) + 8, 32))
    for i, r in enumerate(rows):
        block[i, :len(r)] = r
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    block[-8, :] = -0.0
    block[-7, 3] = tiny
    block[-6, 4] = -tiny
    block[-5, 5] = np.inf
    block[-4, 6] = -np.inf
    block[-3, 7] = np.nan
    block[-2, :] = torch.finfo(dt).max
    block[-1, :] = -torch.finfo(dt).smallest_normal
    x, xr = pair(block, name)
    n = len(block)
    codes, scales = np.full((1, n, 32 if fmt == "mxfp8" else 16), 0x55, np.uint8), np.zeros((1, n, 1), np.uint8)
    c, s = dev(codes, torch.uint8), dev(scales, torch.uint8)
    mx.cache_write(fmt, x, dev(np.arange(n)), c, s)
    rc, rs = o.cache_write(xr, np.arange(n), codes, scales, fmt)
    assert np.array_equal(s.cpu().numpy(), rs)
    bad = np.argwhere(c.cpu().numpy() != rc)
    assert bad.size == 0, (bad[:5], xr[bad[0][1]])
    for out in DTYPES:
        got = mx.cache_read(fmt, c, s, dev([[0]]), dev([0, n]), rows=n, dtype=DTYPES[out])
        with np.errstate(all="ignore"):
            same(got, o.dequantize_rows(rc[0], rs[0], fmt), out)


def test_write_as_the_quantiser_does(mx):
    rng = np.random.default_rng(8)
    x, _ = pair(rng.standard_normal((50, 256)), "bf16")
    for fmt in FORMATS:
        qc, qs = mx.quantize_act(fmt, x)
        c, s = torch.zeros((10, 5, qc.shape[1]), dtype=torch.uint8, device="cuda"), torch.zeros((10, 5, 8), dtype=torch.uint8, device="cuda")
        mx.cache_write(fmt, x, torch.arange(50, dtype=torch.int32, device="cuda"), c, s)
        assert torch.equal(c.view(50, -1), qc) and torch.equal(s.view(50, -1), qs)


@pytest.mark.parametrize("lengths,width,page", [([1], 32, 1), ([0], 64, 4), ([0, 5, 0, 0, 17, 1], 96, 4), ([100], 576, 16),
                                                ([33, 31, 32, 64, 65], 160, 32), ([1] * 70, 64, 2), ([300, 3], 1024, 7)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
def test_read(mx, lengths, width, page, fmt, name):
    rng = np.random.default_rng(sum(lengths) + width)
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    codes, scales = cache(rng, pages, page, width, fmt)
    table = np.full((len(lengths), max(need) + 1), -1)
    order, k = rng.permutation(pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[k:k + n]
        k += n
    for lead, behind in ((0, 0), (3, 40)):
        off = lead + np.concatenate([[0], np.cumsum(lengths)])
        rows = int(off[-1]) + behind
        start, sr = pair(rng.standard_normal((rows, width)), name)
        got = mx.cache_read(fmt, dev(codes, torch.uint8), dev(scales, torch.uint8), dev(table), dev(off), out=start)
        assert got is start
        with np.errstate(all="ignore"):
            same(got, o.cache_read(codes, scales, table, off, sr, fmt), name)


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_pages_read_as_zeros(mx, fmt):
    rng = np.random.default_rng(4)
    codes, scales = cache(rng, 5, 8, 64, fmt)
    table = np.array([[0, 5, 4], [-1, 1, 2 ** 31 - 1], [3, -2 ** 31, 2]])
    off = np.array([0, 24, 60, 70])                   # the second is longer than its table
    c, s = dev(codes, torch.uint8), dev(scales, torch.uint8)
    got = mx.cache_read(fmt, c, s, dev(table), dev(off), rows=70)
    ref = o.cache_read(codes, scales, table, off, np.zeros((70, 64)), fmt)
    assert (ref[8:16] == 0).all() and (ref[48:60] == 0).all() and (ref[24:32] == 0).all()
    same(got, ref, "bf16")
    # no pages at all, no table
    none = mx.cache_read(fmt, c[:0], s[:0], dev(table), dev(off), rows=70)
    assert (none == 0).all()
    none = mx.cache_read(fmt, c, s, dev(table)[:, :0].contiguous(), dev(off), rows=70)
    assert (none == 0).all()
    keep = torch.full((70, 64), 3.0, device="cuda")
    assert (mx.cache_read(fmt, c, s, dev(table)[:0], dev(off)[:1], out=keep) == 3).all()


def test_fewer_rows_than_the_sequences_have(mx):
    rng = np.random.default_rng(5)
    codes, scales = cache(rng, 4, 16, 96, "mxfp8")
    got = mx.cache_read("mxfp8", dev(codes, torch.uint8), dev(scales, torch.uint8), dev([[0, 1], [2, 3]]), dev([0, 30, 62]),
                        rows=41)
    with np.errstate(all="ignore"):
        same(got, o.cache_read(codes, scales, np.array([[0, 1], [2, 3]]), [0, 30, 62], np.zeros((41, 96)), "mxfp8"), "bf16")


@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_rows_of_a_wider_matrix(mx, name):
    """Keys and values as column ranges of one projection's output."""
    rng = np.random.default_rng(6)
    qkv, r = pair(rng.standard_normal((20, 448)), name)
    for fmt in FORMATS:
        for lo in (0, 128, 288):
            codes, scales = cache(rng, 2, 16, 160, fmt)
            c, s = dev(codes, torch.uint8), dev(scales, torch.uint8)
            mx.cache_write(fmt, qkv[:, lo:lo + 160], dev(np.arange(20)), c, s)
            rc, rs = o.cache_write(r[:, lo:lo + 160], np.arange(20), codes, scales, fmt)
            assert np.array_equal(c.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    with pytest.raises(mx.MxError, match="x is not 16-byte aligned"):
        mx.cache_write("mxfp4", qkv[:, 1:161], dev(np.arange(20)), c, s)


def test_no_tokens_and_no_rows(mx):
    c, s = torch.zeros((2, 4, 64), dtype=torch.uint8, device="cuda"), torch.zeros((2, 4, 2), dtype=torch.uint8, device="cuda")
    mx.cache_write("mxfp8", torch.empty((0, 64), device="cuda"), dev(np.zeros(0)), c, s)
    assert mx.cache_read("mxfp8", c, s, dev([[0]]), dev([0, 0]), rows=0).shape == (0, 64)
    assert (c == 0).all()


def test_a_long_cache(mx):
    """Rows whose bytes lie past 2^32 in the cache, and past 2^31 elements in the output."""
    width, page = 8192, 128
    pages = (5 << 30) // (width * page)
    c = torch.zeros((pages, page, width), dtype=torch.uint8, device="cuda")
    s = torch.full((pages, page, width // 32), 127, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    x, xr = pair(rng.standard_normal((3, width)), "bf16")
    slots = np.array([pages * page - 1, pages * page // 2 + 77, 5])
    mx.cache_write("mxfp8", x, dev(slots), c, s)
    n = (1 << 31) // width + 40                        # as many rows as fit 2^31 elements, and some
    table = torch.full((1, -(-n // page)), -1, dtype=torch.int32, device="cuda")
    for i, sl in enumerate(slots):
        table[0, -1 - i] = int(sl) // page
    out = mx.cache_read("mxfp8", c, s, table, dev([0, n]), rows=n)
    want = o.dequantize_rows(*o.quantize_rows(xr, "mxfp8"), "mxfp8")
    first = (n - 1) // page
    for i, sl in enumerate(slots):
        r = (first - i) * page + int(sl) % page
        if r < n:
            assert np.array_equal(out[r].float().cpu().numpy(), want[i].astype(np.float32))
    assert int((out != 0).any(1).sum()) == sum((first - i) * page + int(sl) % page < n for i, sl in enumerate(slots))
