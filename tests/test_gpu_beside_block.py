"""The router, the 4-bit linears and the quantised cache run together, as a layer of a model would run them, and the ways
they are called: through autograd, captured into graphs, on streams, at once."""

import numpy as np
import pytest
import torch

import workloads as W
from around_util import DTYPES, U, f64, pair, rounded, within
from gpu_util import assert_mlp_close, bits, t
from oracle import beside as o
from test_gpu_router import score_error
from test_gpu_w4 import bound, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def _pages(rng, lengths, page):
    """(page table, offsets, the slot of every row), pages in no order."""
    need = [-(-n // page) for n in lengths]
    order, k = rng.permutation(sum(need) + 2), 0
    table = np.full((len(lengths), max(need)), -1)
    for b, n in enumerate(need):
        table[b, :n] = order[k:k + n]
        k += n
    off = np.concatenate([[0], np.cumsum(lengths)])
    slots = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(lengths)])
    return table.astype(np.int32), off.astype(np.int32), slots.astype(np.int32), sum(need) + 2


@pytest.mark.parametrize("lengths", [[1, 1, 1], [40, 1, 75]])
def test_a_layer(mx, lengths):
    """A narrow projection into the cache and back, the router's logits, the choice, the experts. Each step against the
    oracle on what the step before gave; the experts also by sort, gather, single experts and combine."""
    T, H, I, E, k, page, width = sum(lengths), 256, 128, 5, 2, 16, 160
    rng = np.random.default_rng(T)
    x, xr = pair(rng.standard_normal((T, H)), "bf16")
    (w, s, _), v, m = weights(rng, width, H, "mxfp4", 32, "bf16", False)
    latent = mx.w4_linear(x, w, s)
    ref = xr @ v.T
    within(latent, ref, bound(xr, m, ref, "bf16"), "latent")

    table, off, slots, pages = _pages(rng, lengths, page)
    for fmt, wide in (("mxfp8", width), ("mxfp4", width // 2)):
        codes = torch.zeros((pages, page, wide), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((pages, page, width // 32), dtype=torch.uint8, device="cuda")
        mx.cache_write(fmt, latent, t(slots), codes, scales)
        back = mx.cache_read(fmt, codes, scales, t(table), t(off), rows=T)
        want = o.dequantize_rows(*o.quantize_rows(f64(latent), fmt), fmt)
        assert torch.equal(back.cpu(), torch.from_numpy(want).to(torch.bfloat16))

    (w, s, z), v, m = weights(rng, E, H, "int4", 64, "bf16", True)
    logits = mx.w4_linear(x, w, s, z)
    ref = xr @ v.T
    within(logits, ref, bound(xr, m, ref, "bf16"), "logits")
    zr = f64(logits)
    ids, gw = mx.moe_gate(logits, k, scale=2.5)
    ri, rw = o.moe_gate(zr, k, scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), ri)
    within(gw, rw, (2 * score_error(zr, E) + 4 * U) * np.abs(rw), "weights")
    loss, counts = mx.moe_balance(logits, ids, t(off), coef=0.01)
    rl, rc = o.moe_balance(zr, ri, off, coef=0.01)
    assert np.array_equal(counts.cpu().numpy(), rc)
    within(loss, rl, (score_error(zr, E).max() + (T + 40) * U) * rl, "loss")

    d = W.grouped(tokens=T, n_experts=E, k=k, seed=3, hidden=H, inter=I)
    ws = [t(d[n]) for n in ("w1", "w1s", "w3", "w3s", "w2", "w2s")]
    y = mx.grouped_expert_mlp(x, ids, gw, *ws)
    eoff, _, slot_row = mx.moe_sort(ids, E)
    assert np.array_equal(np.diff(eoff.cpu().numpy()), rc.sum(0))
    xs = mx.moe_permute(x, slot_row)
    ys, edges = torch.empty_like(xs), eoff.tolist()
    for e in range(E):
        if edges[e] < edges[e + 1]:
            mx.expert_mlp(xs[edges[e]:edges[e + 1]], *(q[e] for q in ws), out=ys[edges[e]:edges[e + 1]])
    assert_mlp_close(bits(mx.moe_unpermute(ys, slot_row, topk_w=gw)), bits(y))


# ------------------------------------------------------------------ autograd

def _route(mx, k, seq_off, score, renorm, scale, coef):
    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, z):
            z = z.detach()
            ids, w = mx.moe_gate(z, k, score, renorm=renorm, scale=scale)
            loss, counts = mx.moe_balance(z, ids, seq_off, score, coef)
            ctx.save_for_backward(z, ids, counts)
            ctx.mark_non_differentiable(ids)
            return ids, w, loss

        @staticmethod
        def backward(ctx, _, d_w, d_loss):
            z, ids, counts = ctx.saved_tensors
            return mx.moe_gate_grad(z, ids, d_w.contiguous(), counts, d_loss.contiguous(), seq_off, score, renorm, scale, coef)
    return Route.apply


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_through_autograd(mx, score, renorm):
    """Of a loss of the weights and the balance: what autograd finds in 64 bits, and central differences of the
    forward pass in 64 bits along a direction."""
    T, E, k, off, scale, coef = 90, 48, 6, [0, 20, 20, 90], 1.5, 0.1
    rng = np.random.default_rng(1)
    z, zr = pair(2 * rng.standard_normal((T, E)), "fp32")
    a, ar = pair(rng.standard_normal((T, k)), "fp32")
    b, br = pair(1 + rng.random(3), "fp32")
    z.requires_grad_()
    ids, w, loss = _route(mx, k, t(np.array(off, np.int32)), score, renorm, scale, coef)(z)
    ((w * a).sum() + (loss * b).sum()).backward()
    ri, _ = o.moe_gate(zr, k, score)
    assert np.array_equal(ids.cpu().numpy(), ri)
    _, counts = o.moe_balance(zr, ri, off, score)
    c = torch.from_numpy(counts).double()

    def objective(v):
        s = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
        chosen = s.gather(1, torch.from_numpy(ri).long())
        weight = scale * (chosen / chosen.sum(1, keepdim=True) if renorm else chosen)
        p = s / s.sum(1, keepdim=True)
        total = (weight * torch.from_numpy(ar)).sum()
        for q in range(3):
            n = off[q + 1] - off[q]
            if n:
                total = total + br[q] * coef * E / (k * n * n) * (c[q] * p[off[q]:off[q + 1]].sum(0)).sum()
        return total

    v = torch.from_numpy(zr).requires_grad_()
    objective(v).backward()
    _, size = o.moe_gate_grad(zr, ri, ar, counts, br, off, score, renorm, scale, coef)
    tol = (3 * score_error(zr, E) + (k + 30) * U) * size + 2.0 ** -120
    within(z.grad, v.grad.numpy(), tol + rounded(v.grad.numpy(), "fp32"))
    direction, h = torch.from_numpy(rng.standard_normal((T, E))), 1e-5
    with torch.no_grad():
        slope = float(objective(v + h * direction) - objective(v - h * direction)) / (2 * h)
        most = float(objective(v).abs())
    # the third derivative's part (h^2 times scores' products of at most the gradient's size) and the objective's rounding
    room = 1e-8 * float((direction.abs() ** 3 * torch.from_numpy(size)).sum()) + 2.0 ** -50 * (most + 10) / h
    got = float((z.grad.double().cpu() * direction).sum())
    assert abs(got - slope) <= room + float((torch.from_numpy(tol + rounded(v.grad.numpy(), "fp32")) * direction.abs()).sum())


# ------------------------------------------------------------------ graphs and streams

class _Step:
    """Every operator once, over buffers of its own; run() into given outputs and a given workspace, so that it can be
    captured."""

    def __init__(self, mx, T, H, width, seed, name="bf16", ws=None):
        rng = np.random.default_rng(seed)
        self.mx, E, k, page = mx, 40, 4, 8
        i32, u8, f32, dt = torch.int32, torch.uint8, torch.float32, DTYPES[name]
        z = lambda *s, dt: torch.zeros(s, dtype=dt, device="cuda")
        self.x = pair(rng.standard_normal((T, H)), name)[0]
        self.router = weights(rng, E, H, "int4", 32, name, True)[0]
        self.down = weights(rng, width, H, "mxfp4", 32, name, False)[0][:2]
        self.bias = pair(0.1 * rng.standard_normal(E), "fp32")[0]
        self.a, self.b = pair(rng.standard_normal((T, k)), "fp32")[0], pair(rng.standard_normal(3), "fp32")[0]
        cut = np.sort(rng.integers(0, T + 1, size=2)).tolist()
        lengths = np.diff([0, *cut, T])
        need = -(-lengths // page)
        rest = rng.permutation(-(-T // page) + 3)
        self.table, at = t(np.full((3, -(-T // page)), -1, np.int32)), 0
        for q in range(3):
            self.table[q, :need[q]] = t(rest[at:at + need[q]].astype(np.int32))
            at += need[q]
        self.off = t(np.array([0, *cut, T], np.int32))
        tab = self.table.cpu().numpy()
        self.slots = t(np.concatenate([tab[q, np.arange(n) // page] * page + np.arange(n) % page
                                       for q, n in enumerate(lengths)]).astype(np.int32))
        self.logits, self.latent, self.back = z(T, E, dt=dt), z(T, width, dt=dt), z(T, width, dt=dt)
        self.ids, self.gw, self.loss, self.counts = z(T, k, dt=i32), z(T, k, dt=f32), z(3, dt=f32), z(3, E, dt=i32)
        self.dz = z(T, E, dt=dt)
        self.codes, self.scales = z(len(rest), page, width, dt=u8), z(len(rest), page, width // 32, dt=u8)
        need = max(mx.w4_linear_workspace_size(T, H, E), mx.w4_linear_workspace_size(T, H, width),
                   mx.moe_balance_workspace_size(T, E, 3), 256)
        self.ws = torch.empty(need, dtype=u8, device="cuda") if ws is None else ws
        self.ins = [self.x, *self.router, *self.down, self.bias, self.a, self.b, self.table, self.off, self.slots]
        self.outs = [self.logits, self.latent, self.back, self.ids, self.gw, self.loss, self.counts, self.dz, self.codes,
                     self.scales]

    def run(self, stream=None):
        m, s = self.mx, {"stream": stream}
        m.w4_linear(self.x, *self.router, out=self.logits, workspace=self.ws, **s)
        m.moe_gate(self.logits, 4, "sigmoid", self.bias, topk_ids=self.ids, topk_w=self.gw, **s)
        m.moe_balance(self.logits, self.ids, self.off, "sigmoid", loss=self.loss, counts=self.counts, workspace=self.ws, **s)
        m.moe_gate_grad(self.logits, self.ids, self.a, self.counts, self.b, self.off, "sigmoid", d_logits=self.dz, **s)
        m.w4_linear(self.x, *self.down, out=self.latent, workspace=self.ws, **s)
        m.cache_write("mxfp8", self.latent, self.slots, self.codes, self.scales, **s)
        m.cache_read("mxfp8", self.codes, self.scales, self.table, self.off, out=self.back, **s)

    def clear(self):
        for v in self.outs:
            v.zero_()

    def values(self):
        return [v.clone() for v in self.outs]


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


# one token; K in parts; tiles of 256 with scales' tables
SIZES = [(1, 256, 160, "bf16"), (90, 992, 160, "fp16"), (2600, 256, 3840, "bf16")]


@pytest.mark.parametrize("T,H,width,name", SIZES)
def test_captured_and_replayed(mx, T, H, width, name):
    """A graph of every operator: replays with eager work between them, and with new inputs in the old buffers, give
    what eager calls give, bit for bit."""
    st = _Step(mx, T, H, width, 1, name)
    st.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    other = _Step(mx, T, H, width, 2, name)
    for seed in (1, 7, 8):
        fresh = _Step(mx, T, H, width, seed, name)
        for mine, theirs in zip(st.ins, fresh.ins):
            mine.copy_(theirs)
        fresh.run()
        want = fresh.values()
        for _ in range(2):
            st.clear()
            st.ws.fill_(0xFF)                      # whatever a workspace held before
            other.run()                            # the program's own eager work
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert _same(st.values(), want), seed


@pytest.mark.parametrize("T,H,width,name", SIZES[1:])
def test_two_graphs_share_a_workspace(mx, T, H, width, name):
    """Replayed one after the other on a stream."""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    steps = [_Step(mx, T, H, width, s, name, ws=ws) for s in (1, 2)]
    want, graphs = [], []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.values())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.run()
        graphs.append(g)
    for _ in range(3):
        for st in steps:
            st.clear()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(_same(st.values(), w) for st, w in zip(steps, want))


def test_at_once_in_a_graph(mx):
    """Two branches of one graph, each with a workspace of its own."""
    steps = [_Step(mx, 300, 512, 160, s) for s in (1, 2)]
    want = []
    for st in steps:
        st.run()
        want.append(st.values())
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        steps[0].run()
        steps[1].run(stream=side)
        now.wait_stream(side)
    for _ in range(3):
        for st in steps:
            st.clear()
            st.ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert all(_same(st.values(), w) for st, w in zip(steps, want))


def test_on_a_given_stream_and_at_once(mx):
    """Calls on streams of their own, in flight together, each with buffers of its own; and calls that make their
    own outputs and workspaces for a stream that is not the current one."""
    steps = [_Step(mx, 700, 512, 160, s) for s in range(3)]
    want = []
    for st in steps:
        st.run()
        want.append(st.values())
        st.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for st, s in zip(steps, streams):
            st.run(stream=s)
    torch.cuda.synchronize()
    assert all(_same(st.values(), w) for st, w in zip(steps, want))
    s, st = streams[0], steps[0]
    for _ in range(5):
        logits = mx.w4_linear(st.x, *st.router, stream=s)
        ids, gw = mx.moe_gate(logits, 4, "sigmoid", st.bias, stream=s)
        loss, counts = mx.moe_balance(logits, ids, st.off, "sigmoid", stream=s)
        dz = mx.moe_gate_grad(logits, ids, st.a, counts, st.b, st.off, "sigmoid", stream=s)
        latent = mx.w4_linear(st.x, *st.down, stream=s)
        back = mx.cache_read("mxfp8", st.codes, st.scales, st.table, st.off, rows=700, dtype=st.x.dtype, stream=s)
        with torch.cuda.stream(s):
            got = [v.clone() for v in (logits, latent, back, ids, gw, loss, counts, dz)]
        del logits, ids, gw, loss, counts, dz, latent, back
        junk = [torch.full((700, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (40, 160, 4, 8, 40, 160)]
        s.synchronize()
        del junk
        assert _same(got, want[0][:8])
