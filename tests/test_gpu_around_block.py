"""The operators around the experts run together, as a MoE block would run them, and the ways they are called:
captured into graphs, on streams, at once, refused."""

import numpy as np
import pytest
import torch

import workloads as W
from around_util import DTYPES, U, depth, f64, half_step, pair, rounded, routing, within
from gpu_util import assert_mlp_close, bf16_t, bits, t
from oracle import around

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def _norm_tol(n, rel, name="bf16"):
    return 1.02 * (np.abs(n) * rel + rounded(n, name))


@pytest.mark.parametrize("T", [4, 150])
def test_a_moe_block(mx, T):
    """Norm, sort, rows to MXFP4 experts and back, a shared expert beside them, the norms and the gate behind the
    block. Each step against the oracle on what the step before gave; the routed part also against
    mx_grouped_expert_mlp, which does sort, gather and combine itself."""
    E, k, H, I = 5, 2, 256, 128
    names = ("w1", "w1s", "w3", "w3s", "w2", "w2s")
    d = W.grouped(tokens=T, n_experts=E, k=k, seed=3, hidden=H, inter=I)
    w = [t(d[n]) for n in names]
    ids, gw = t(d["ids"]), t(d["w"])
    rng = np.random.default_rng(T)
    res, res64 = pair(3 * rng.standard_normal((T, H)), "fp32")
    w_pre, wpre64 = pair(1 + 0.1 * rng.standard_normal(H), "bf16")
    w_post, wpost64 = pair(1 + 0.1 * rng.standard_normal(H), "bf16")
    w_next, wnext64 = pair(1 + 0.1 * rng.standard_normal(H), "bf16")
    gate, gate64 = pair(rng.uniform(0, 1, (T, 1)), "bf16")
    rel = depth(H) * U / 2 + 8 * U

    x, _ = mx.block_norm(res, w_pre, eps=EPS)
    n, _ = around.block_norm(res64, wpre64, eps=EPS)
    within(x, n, _norm_tol(n, rel), "first norm")

    off, row_slot, slot_row = mx.moe_sort(ids, E)
    xs = mx.moe_permute(x, slot_row)
    ys = torch.empty_like(xs)
    bounds = off.tolist()
    assert bounds[-1] == T * k
    for e in range(E):
        if bounds[e] < bounds[e + 1]:
            mx.expert_mlp(xs[bounds[e]:bounds[e + 1]], *(v[e] for v in w), out=ys[bounds[e]:bounds[e + 1]])
    y = mx.moe_unpermute(ys, slot_row, topk_w=gw)
    sr, gw64, ys64 = slot_row.cpu().numpy(), f64(gw), f64(ys)
    ref = around.moe_unpermute(ys64, sr, gw64)
    within(y, ref, 1.01 * (rounded(ref, "bf16") + k * U * around.moe_unpermute(np.abs(ys64), sr, np.abs(gw64))), "back")
    # the fused path rounds w * y per pair; its experts' kernels are chosen by the whole batch
    assert_mlp_close(bits(y), bits(mx.grouped_expert_mlp(x, ids, gw, *w)))

    y += mx.expert_mlp(x, *(v[0] for v in w))              # a shared expert
    y64 = f64(y)
    nxt, r = mx.block_norm(res, w_next, y=y, w_post=w_post, gate=gate, res_scale=0.5, eps=EPS)
    n64, r64 = around.block_norm(res64, wnext64, y64, wpost64, gate64, 0.5, EPS)
    er = np.abs(r64 - res64) * rel + 2 * U * (np.abs(r64) + np.abs(res64))
    within(r, r64, 1.02 * (er + rounded(r64, "fp32")), "residual")
    rms = np.sqrt((r64 * r64).mean(1, keepdims=True) + EPS)
    spread = np.sqrt((er * er).sum(1, keepdims=True) / (r64 * r64).sum(1, keepdims=True))
    within(nxt, n64, _norm_tol(n64, rel + spread) + 1.02 * er / rms * np.abs(wnext64), "next norm")


def test_adapters_on_quantised_projections(mx):
    """The NVFP4 and the FP8 linear with the adapters of a batch's requests on top, one plan for both; the
    projections themselves are unchanged."""
    M, K, N, R, n = 70, 256, 384, 16, 3
    rng = np.random.default_rng(0)
    x, x64 = pair(rng.integers(-2, 3, size=(M, K)), "bf16")
    a, a64 = pair(rng.integers(-1, 2, size=(n, R, K)), "bf16")
    b, b64 = pair(rng.integers(-1, 2, size=(n, N, R)), "bf16")
    adapter = np.repeat([2, -1, 0, 1, 2], 14)
    off, row_token, _ = mx.moe_sort(t(adapter.astype(np.int32).reshape(-1, 1)), n)
    codes = t(rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8))
    scales = t(np.full((N, K // 16), 0x38, np.uint8))                 # 1.0
    fp8 = t(rng.integers(0, 0x78, size=(N, K)).astype(np.uint8))
    fs = t(np.full((N // 128, K // 128), 120, np.uint8))
    for run in (lambda: mx.nvfp4_linear(x, codes, scales, 0.5, 0.25), lambda: mx.fp8_block_linear(x, fp8, fs)):
        y = run()
        base = f64(y)
        assert mx.lora_add(y, x, a, b, off, row_token) is y
        ref = around.lora_add(base, x64, a64, b64, adapter)
        # whole numbers: the sum is exact in fp32 up to its addition to y
        within(y, ref, 1.01 * (rounded(ref, "bf16") + 2 * U * (np.abs(ref) + np.abs(base))))
        assert torch.equal(run().cpu()[14:28], y.cpu()[14:28])


# ------------------------------------------------------------------ graphs and streams

class _Step:
    """Every operator once, over buffers of its own; run() with `out` buffers and workspaces, so that it can be captured."""

    def __init__(self, mx, T, H, seed, name="bf16", k=3, E=9, R=24, n=4, ws=None):
        rng = np.random.default_rng(seed)
        self.mx = mx
        mk = lambda *s: pair(rng.standard_normal(s), name)[0]
        self.x, self.res, self.y0, self.dn = mk(T, H), mk(T, H), mk(T, H), mk(T, H)
        self.w1, self.w2, self.gate = mk(H), mk(H), mk(H)
        self.ids = t(routing(rng, T, k, E, E + 4))
        self.gw = pair(rng.standard_normal((T, k)), "fp32")[0]
        self.a, self.b = mk(n, R, H), mk(n, H, R)
        self.aid = t(rng.integers(-1, n, size=(T, 1)).astype(np.int32))
        self.E, self.n = E, n
        z = lambda *s, dt=DTYPES[name]: torch.zeros(s, dtype=dt, device="cuda")
        i32 = torch.int32
        self.off, self.rs, self.sr = z(E + 1, dt=i32), z(T * k, dt=i32), z(T, k, dt=i32)
        self.aoff, self.ars, self.asr = z(n + 1, dt=i32), z(T, dt=i32), z(T, 1, dt=i32)
        self.normed, self.ro, self.xs, self.back, self.yl = z(T, H), z(T, H), z(T * k, H), z(T, H), z(T, H)
        self.dys, self.dw = z(T * k, H), z(T, k, dt=torch.float32)
        self.dr, self.dy = z(T, H), z(T, H)
        need = max(mx.moe_sort_workspace_size(T, k, E), mx.moe_sort_workspace_size(T, 1, n),
                   mx.block_norm_grad_workspace_size(T, H), mx.lora_add_workspace_size(T, H, R, n), 256)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda") if ws is None else ws
        self.outs = [self.off, self.rs, self.sr, self.normed, self.ro, self.xs, self.back, self.yl, self.dys, self.dw,
                     self.dr, self.dy]
        self.grads = None

    def run(self, stream=None):
        m, s = self.mx, {"stream": stream}
        m.block_norm(self.res, self.w1, y=self.y0, w_post=self.w2, gate=self.gate, residual_out=self.ro,
                     normed=self.normed, **s)
        m.moe_sort(self.ids, self.E, self.off, self.rs, self.sr, workspace=self.ws, **s)
        m.moe_permute(self.normed, self.sr, out=self.xs, **s)
        m.moe_unpermute(self.xs, self.sr, topk_w=self.gw, out=self.back, **s)
        m.moe_sort(self.aid, self.n, self.aoff, self.ars, self.asr, workspace=self.ws, **s)
        m.lora_add(self.yl, self.x, self.a, self.b, self.aoff, self.ars, workspace=self.ws, **s)
        m.moe_unpermute_grad(self.dn, self.xs, self.sr, self.gw, d_ys=self.dys, d_w=self.dw, **s)
        self.grads = m.block_norm_grad(self.ro, self.w1, self.dn, d_residual_out=self.res, y=self.y0, w_post=self.w2,
                                       gate=self.gate, d_residual=self.dr, d_y=self.dy, workspace=self.ws, **s)

    def clear(self):
        for o in self.outs:
            o.zero_()

    def values(self):
        return [v.clone() for v in self.outs + [self.grads[i] for i in (1, 3, 4)]]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


SIZES = [(1, 256, "bf16"), (130, 1000, "fp16"), (1500, 512, "bf16")]


@pytest.mark.parametrize("T,H,name", SIZES)
def test_captured_and_replayed(mx, T, H, name):
    """A graph of every operator: replays with eager work between them, and with new inputs in the old buffers,
    give what eager calls give, bit for bit."""
    st = _Step(mx, T, H, 1, name)
    st.run()
    torch.cuda.synchronize()
    st.clear()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    captured = st.grads
    other = _Step(mx, T, H, 2, name)
    for seed in (1, 7, 8):
        fresh = _Step(mx, T, H, seed, name)
        for mine, theirs in ((st.x, fresh.x), (st.res, fresh.res), (st.y0, fresh.y0), (st.ids, fresh.ids),
                             (st.gw, fresh.gw), (st.aid, fresh.aid), (st.dn, fresh.dn), (st.a, fresh.a),
                             (st.b, fresh.b), (st.w1, fresh.w1), (st.w2, fresh.w2), (st.gate, fresh.gate)):
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
            st.grads = captured
            assert _same(st.values(), want), seed


def test_two_graphs_share_a_workspace(mx):
    """Replayed one after the other on a stream."""
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    steps = [_Step(mx, 300, 264, s, ws=ws) for s in (1, 2)]
    want, graphs, grads = [], [], []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        want.append(st.values())
        g = torch.cuda.CUDAGraph()
        st.clear()
        with torch.cuda.graph(g):
            st.run()
        graphs.append(g)
        grads.append(st.grads)
    for _ in range(3):
        for st in steps:
            st.clear()
        for g in graphs + graphs[::-1]:
            for st in steps:
                st.yl.zero_()                      # the one output that is added to
            g.replay()
        torch.cuda.synchronize()
        # the adapters' output of the step replayed last; all others of both
        for i, st in enumerate(steps):
            st.grads = grads[i]
            got = st.values()
            if i == 1:
                got[7] = want[i][7]
            assert _same(got, want[i])


def test_on_a_given_stream_and_at_once(mx):
    """Calls on streams of their own, in flight together, each with buffers of its own; and calls that make their
    own outputs and workspaces for a stream that is not the current one."""
    steps = [_Step(mx, 700, 512, s) for s in range(3)]
    want = []
    for st in steps:
        st.run()
        want.append(st.values())
        st.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for st, s in zip(steps, streams):
            st.run(stream=s)
            with torch.cuda.stream(s):
                st.yl.zero_()
    for st, s in zip(steps, streams):
        st.run(stream=s)
    torch.cuda.synchronize()
    assert all(_same(st.values(), w) for st, w in zip(steps, want))
    s = streams[0]
    st = steps[0]
    for _ in range(5):
        off, rs, sr = mx.moe_sort(st.ids, st.E, stream=s)
        n, r = mx.block_norm(st.res, st.w1, y=st.y0, w_post=st.w2, gate=st.gate, stream=s)
        xs = mx.moe_permute(n, sr, stream=s)
        y = mx.moe_unpermute(xs, sr, topk_w=st.gw, stream=s)
        g = mx.block_norm_grad(r, st.w1, st.dn, d_residual_out=st.res, y=st.y0, w_post=st.w2, gate=st.gate, stream=s)
        dys, dw = mx.moe_unpermute_grad(st.dn, xs, sr, st.gw, stream=s)
        with torch.cuda.stream(s):
            got = [y.clone(), g[0].clone(), g[1].clone(), dw.clone(), dys.clone()]
        del off, rs, sr, n, r, xs, y, g, dys, dw
        junk = [torch.full((700 * 3, 512), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        s.synchronize()
        del junk
        assert _same(got, [want[0][6], want[0][10], want[0][12], want[0][9], want[0][8]])


# ------------------------------------------------------------------ refusals

def test_refusals(mx):
    """Wrong types, shapes, strides and overlaps raise, and nothing is written."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    gw = torch.zeros((4, 2), device="cuda")
    ys = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    a, b = x.view(2, 2, 64).repeat(1, 4, 1), torch.zeros((2, 32, 8), dtype=torch.bfloat16, device="cuda")
    y = torch.ones((4, 32), dtype=torch.bfloat16, device="cuda")
    off, tok = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    value = [
        lambda: mx.moe_sort(ids.long(), 4), lambda: mx.moe_sort(ids, 0), lambda: mx.moe_sort(ids, 513),
        lambda: mx.moe_sort(ids.t(), 4), lambda: mx.moe_sort(ids, 4, expert_off=off),
        lambda: mx.moe_permute(x.double(), ids), lambda: mx.moe_permute(x, ids[:3]), lambda: mx.moe_permute(x, ids, out=ys[:, :32]),
        lambda: mx.moe_permute(x[:, ::2], ids), lambda: mx.moe_permute(x, ids.cpu()),
        lambda: mx.moe_unpermute(ys, ids, topk_w=gw.bfloat16()), lambda: mx.moe_unpermute(ys, ids, topk_w=gw[:2]),
        lambda: mx.moe_unpermute_grad(x.float(), ys, ids, gw), lambda: mx.moe_unpermute_grad(x, ys, ids, gw, d_ys=ys[:4]),
        lambda: mx.block_norm(x), lambda: mx.block_norm(x, w.float(), y=x), lambda: mx.block_norm(x, w[:32]),
        lambda: mx.block_norm(x, w, w_post=w), lambda: mx.block_norm(x, w, y=x, gate=x[:2]),
        lambda: mx.block_norm(x, w, y=x.t().contiguous()), lambda: mx.block_norm(x, normed=x, y=x),
        lambda: mx.block_norm_grad(x, w), lambda: mx.block_norm_grad(x, w, x, d_residual_out=x.float()),
        lambda: mx.block_norm_grad(x, y=x), lambda: mx.block_norm_grad(x, w, x, d_y=x),
        lambda: mx.lora_add(y, x[:, :32], a, b, off, tok), lambda: mx.lora_add(y[:, :24], x, a, b, off, tok),
        lambda: mx.lora_add(y, x, a, b, off[:2], tok), lambda: mx.lora_add(y, x, a, b.half(), off, tok),
        lambda: mx.lora_add(y.t(), x[:, ::2], a, b, off, tok),
    ]
    for call in value:
        with pytest.raises(ValueError):
            call()
    library = [
        (lambda: mx.moe_permute(x, ids, out=torch.as_strided(x, (2, 64), (64, 1))), "overlaps"),
        (lambda: mx.moe_unpermute_grad(x, ys, ids, gw, d_ys=ys), "overlaps"),
        (lambda: mx.block_norm(x.half(), w, y=x), "residual type"),
        (lambda: mx.block_norm(x, w, y=x, eps=-1.0), "eps"),
        (lambda: mx.block_norm(x, w, y=ys[:4], normed=x), "overlaps"),
        (lambda: mx.lora_add(y, x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), off, tok), "rank"),
        (lambda: mx.lora_add(y.float(), x.float(), a.float(), b.float(), off, tok), "bf16 or fp16"),
        (lambda: mx.lora_add(y, x, a, b, off, tok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), "workspace"),
    ]
    for call, text in library:
        with pytest.raises(mx.MxError, match=text):
            call()
    torch.cuda.synchronize()
    assert (y == 1).all() and not x.any() and not ys.any()
