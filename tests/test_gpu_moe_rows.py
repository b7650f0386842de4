"""mx_moe_sort, mx_moe_permute, mx_moe_unpermute and mx_moe_unpermute_grad against the fp64 oracle:
the maps exactly, copied rows bit for bit, sums within the bound of their fp32 arithmetic."""

import numpy as np
import pytest
import torch

from around_util import DTYPES, U, depth, f64, pair, rounded, routing, within
from oracle import around

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def _host(*ts):
    return [t.cpu().numpy().astype(np.int64) for t in ts]


def _check_sort(mx, ids, E):
    off, row_slot, slot_row = _host(*mx.moe_sort(torch.from_numpy(ids).cuda(), E))
    flat = ids.reshape(-1).astype(np.int64)
    local = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(local, flat, E), kind="stable")
    n = int(local.sum())
    assert np.array_equal(off, np.searchsorted(flat[order][:n], np.arange(E + 1)) if n else np.zeros(E + 1))
    assert np.array_equal(row_slot, np.where(np.arange(flat.size) < n, order, -1))
    inv = np.full(flat.size, -1)
    inv[order[:n]] = np.arange(n)
    assert np.array_equal(slot_row.reshape(-1), inv)
    return off, row_slot, slot_row


@pytest.mark.parametrize("T,k,E", [(0, 3, 5), (1, 1, 1), (1, 8, 48), (8, 8, 48), (63, 1, 7), (64, 1, 512), (65, 3, 33),
                                   (127, 8, 512), (128, 8, 64), (171, 6, 384), (512, 8, 48), (513, 8, 48),
                                   (1025, 1, 2), (4096, 1, 1), (4097, 1, 3), (1000, 5, 512)])
def test_sort(mx, T, k, E):
    """One workgroup and several, chunk borders, one expert to 512, ids of other ranks on both sides."""
    rng = np.random.default_rng(T * 1000 + k * 10 + E)
    ids = rng.integers(-E // 4 - 1, E + E // 4 + 2, size=(T, k)).astype(np.int32)
    got = _check_sort(mx, ids, E)
    if T and T <= 200:
        for a, b in zip(got, around.moe_sort(ids, E)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("T,k,E", [(33, 4, 8), (3000, 4, 8)])
def test_sort_extremes(mx, T, k, E):
    """No local pair at all; every pair on one expert; ids at the ends of int32."""
    for fill in (-1, E, 2 ** 31 - 1, -2 ** 31, 0, E - 1):
        _check_sort(mx, np.full((T, k), fill, np.int32), E)


def test_sort_many_chunks(mx):
    """300,000 pairs over 293 chunks."""
    rng = np.random.default_rng(0)
    _check_sort(mx, rng.integers(-1, 200, size=(100000, 3)).astype(np.int32), 200)


def _maps(mx, rng, T, k, E, total):
    ids = routing(rng, T, k, E, total) - (total - E) // 2
    _, _, slot_row = mx.moe_sort(torch.from_numpy(np.ascontiguousarray(ids)).cuda(), E)
    return slot_row, slot_row.cpu().numpy()


SHAPES = [(1, 1, 1, 1, 8), (1, 8, 48, 48, 7168), (5, 3, 4, 4, 1), (7, 2, 6, 6, 33), (9, 9, 16, 16, 100),
          (33, 6, 8, 64, 1000), (64, 4, 8, 8, 2049), (130, 17, 32, 32, 264),
          (20, 3, 5, 9, 5), (20, 3, 5, 9, 9), (20, 3, 5, 9, 14), (6, 2, 4, 4, 4099)]


@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,total,H", SHAPES)
def test_permute(mx, T, k, E, total, H, name):
    rng = np.random.default_rng(T + H)
    slot_row, sr = _maps(mx, rng, T, k, E, total)
    x, _ = pair(rng.standard_normal((T, H)), name)
    out = torch.full((T * k, H), -7.0, dtype=DTYPES[name], device="cuda")
    got = mx.moe_permute(x, slot_row, out=out)
    assert got is out
    assert np.array_equal(f64(got), around.moe_permute(f64(x), sr, np.full((T * k, H), -7.0)))


def test_permute_keeps_bits_and_skips_rows_past_the_buffer(mx):
    """NaN payloads are copied as they are; a buffer with fewer rows takes those it has."""
    rng = np.random.default_rng(3)
    slot_row, sr = _maps(mx, rng, 40, 3, 5, 5)
    bits = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, size=(40, 56)).astype(np.int16)).cuda()
    out = torch.zeros((60, 56), dtype=torch.bfloat16, device="cuda")
    mx.moe_permute(bits.view(torch.bfloat16), slot_row, out=out)
    ref = around.moe_permute(bits.cpu().numpy(), sr, np.zeros((60, 56), np.int16))
    assert np.array_equal(out.view(torch.int16).cpu().numpy(), ref)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,total,H", SHAPES)
def test_unpermute(mx, T, k, E, total, H, name, weighted):
    rng = np.random.default_rng(T + H + 1)
    slot_row, sr = _maps(mx, rng, T, k, E, total)
    ys, ys64 = pair(rng.standard_normal((T * k, H)), name)
    w, w64 = pair(rng.standard_normal((T, k)), "fp32") if weighted else (None, None)
    got = mx.moe_unpermute(ys, slot_row, topk_w=w)
    ref = around.moe_unpermute(ys64, sr, w64)
    mass = around.moe_unpermute(np.abs(ys64), sr, None if w64 is None else np.abs(w64))
    # k fused multiply-adds, each off by half a step of a partial sum of at most `mass`
    within(got, ref, 1.01 * (rounded(ref, name) + k * U * mass))


def test_unpermute_ignores_what_skipped_slots_hold(mx):
    """NaN and infinite rows and weights that no routed slot uses change nothing; a token without any
    routed slot gets zeros; rows past the buffer are skipped."""
    sr = torch.tensor([[0, -1, 2], [-1, -1, -1], [9, 1, -1]], dtype=torch.int32, device="cuda")
    ys = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    ys[3] = float("nan")
    w = torch.tensor([[2.0, float("nan"), 3.0], [float("inf")] * 3, [float("nan"), 0.5, float("nan")]], device="cuda")
    y = f64(mx.moe_unpermute(ys, sr, topk_w=w))
    assert np.array_equal(y, np.array([[5.0] * 16, [0.0] * 16, [0.5] * 16]))
    dys, dw = mx.moe_unpermute_grad(torch.ones((3, 16), dtype=torch.bfloat16, device="cuda"), ys, sr, w)
    assert np.array_equal(f64(dys), np.array([[2.0] * 16, [0.5] * 16, [3.0] * 16, [0.0] * 16]))
    assert np.array_equal(f64(dw), np.array([[16.0, 0, 16.0], [0, 0, 0], [0, 16.0, 0]]))


@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,total,H", SHAPES)
def test_unpermute_grad(mx, T, k, E, total, H, name):
    rng = np.random.default_rng(T + H + 2)
    slot_row, sr = _maps(mx, rng, T, k, E, total)
    ys, ys64 = pair(rng.standard_normal((T * k, H)), name)
    dy, dy64 = pair(rng.standard_normal((T, H)), name)
    w, w64 = pair(rng.standard_normal((T, k)), "fp32")
    keep, keep64 = pair(rng.standard_normal((T * k, H)), name)
    dys, dw = mx.moe_unpermute_grad(dy, ys, slot_row, w, d_ys=keep)
    rdys, rdw = around.moe_unpermute_grad(dy64, ys64, sr, w64, keep64)
    _, mass = around.moe_unpermute_grad(np.abs(dy64), np.abs(ys64), sr, np.abs(w64), keep64)
    within(dys, rdys, 1.01 * (rounded(rdys, name) + U * np.abs(rdys)), "dys")
    within(dw, rdw, 1.01 * depth(H) * U * mass, "dw")


def test_gradients_of_a_round_trip(mx):
    """Permute, a weight per expert, unpermute, and back through the gradients, in fp32, against torch's
    differentiation of the same function in float64."""
    rng = np.random.default_rng(11)
    T, k, E, H = 50, 3, 6, 96
    ids = routing(rng, T, k, E + 2)                       # some slots on other ranks
    off, row_slot, slot_row = mx.moe_sort(torch.from_numpy(ids).cuda(), E)
    x, x64 = pair(rng.standard_normal((T, H)), "fp32")
    w, w64 = pair(rng.standard_normal((T, k)), "fp32")
    m, m64 = pair(rng.standard_normal((E, H)), "fp32")
    g, g64 = pair(rng.standard_normal((T, H)), "fp32")
    n = int(off[-1])
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), (off[1:] - off[:-1]).long())
    xs = mx.moe_permute(x, slot_row, out=torch.zeros((T * k, H), device="cuda"))
    ys = torch.zeros_like(xs)
    ys[:n] = xs[:n] * m[expert]
    y = mx.moe_unpermute(ys, slot_row, topk_w=w)
    dys, dw = mx.moe_unpermute_grad(g, ys, slot_row, w)
    dxs = torch.zeros_like(dys)
    dxs[:n] = dys[:n] * m[expert]
    dx = mx.moe_unpermute(dxs, slot_row)
    tx, tw, tm = (torch.tensor(v, requires_grad=True) for v in (x64, w64, m64))
    loc = torch.from_numpy((ids < E).astype(np.float64))
    ty = (tx[:, None, :] * tm[torch.from_numpy(np.minimum(ids, E - 1)).long()] * (tw * loc)[:, :, None]).sum(1)
    ty.backward(torch.from_numpy(g64))
    # products of three fp32 numbers, sums of at most depth(H) terms of size below 64
    tol = 64 * depth(H) * U
    for a, b in ((y, ty.detach()), (dx, tx.grad), (dw, tw.grad)):
        within(a, b.numpy(), tol * np.maximum(1.0, np.abs(b.numpy())))


def test_views_at_any_alignment(mx):
    """Rows that start off 16 bytes take the narrower accesses, with the same results."""
    rng = np.random.default_rng(5)
    slot_row, sr = _maps(mx, rng, 20, 2, 4, 4)
    buf = torch.from_numpy(rng.standard_normal(20 * 64 + 8)).to(torch.bfloat16).cuda()
    for shift in (1, 2, 4):
        x = buf[shift:shift + 20 * 64].view(20, 64)
        xs = mx.moe_permute(x, slot_row)
        assert np.array_equal(f64(xs), around.moe_permute(f64(x), sr, np.zeros((40, 64))))
        ob = torch.empty(20 * 64 + 8, dtype=torch.bfloat16, device="cuda")
        y = mx.moe_unpermute(xs, slot_row, out=ob[shift:shift + 20 * 64].view(20, 64))
        assert np.array_equal(f64(y), 2 * f64(x))


def test_more_than_2_to_the_31_elements(mx):
    """Offsets past 32 bits: the last rows of a 5.4 GB buffer."""
    H, rows = 7168, 380000
    xs = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    slot_row = torch.tensor([[rows - 1, 0], [rows - 2, 1]], dtype=torch.int32, device="cuda")
    x = torch.arange(2 * H, device="cuda").remainder(251).to(torch.bfloat16).view(2, H)
    mx.moe_permute(x, slot_row, out=xs)
    assert torch.equal(xs[rows - 1], x[0]) and torch.equal(xs[rows - 2], x[1]) and not xs[2:rows - 2].any()
    assert torch.equal(mx.moe_unpermute(xs, slot_row), x + x)
    w = torch.ones((2, 2), device="cuda")
    dys = torch.zeros_like(xs)
    _, dw = mx.moe_unpermute_grad(x, xs, slot_row, w, d_ys=dys)
    assert torch.equal(dys[rows - 1], x[0]) and torch.equal(dys[1], x[1])
    ref = (f64(x) ** 2).sum(1, keepdims=True).repeat(2, 1)
    within(dw, ref, depth(H) * U * ref)


@pytest.mark.parametrize("P,k,E", [(512 * 1024 - 1, 1, 200), (512 * 1024, 4, 512), (512 * 1024 + 1, 1, 1),
                                   (513 * 1024, 8, 200), (600 * 1024 + 300, 1, 512), (1 << 20, 8, 48)])
def test_sort_past_the_chunks_that_scan_themselves(mx, P, k, E):
    """Up to 512 chunks every scatter workgroup sums the histograms itself, beyond a kernel of its own does: both sides
    of the border, the last chunk whole and not, ids outside the experts on both sides."""
    assert P % k == 0
    rng = np.random.default_rng(P + E)
    _check_sort(mx, rng.integers(-E // 4 - 1, E + E // 4 + 2, size=(P // k, k)).astype(np.int32), E)


@pytest.mark.parametrize("P", [512 * 1024, 512 * 1024 + 1024])
def test_sort_of_many_slots_on_one_expert_or_none(mx, P):
    for fill in (-1, 6, 7):
        _check_sort(mx, np.full((P, 1), fill, np.int32), 7)
