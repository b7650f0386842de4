"""The operators beside the experts: host-side validation of the C ABI (nothing here reaches a kernel) and of the
binding's own checks, on the CPU; the same checks again under the host sanitizers."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import test_abi_around as A
from binding_util import BF16, F32, I32, U8, Stream, Tensor, stand_in, t
from test_abi_around import ALIGN, FORMAT, NULL, ROOT, SHAPE, VALUE, WORKSPACE, L, at  # noqa: F401  (L: fixture)

F16_, F32_ = 1, 2


def _call(L, name, good, **over):
    return A._call(L, name, good, list(good), **over)


def _none(good):
    return {k: (None if isinstance(v, int) and v >= at(0) and k != "n" else v) for k, v in good.items()}


GATE = dict(dt=F32_, z=at(0), T=8, E=48, score=0, bias=at(1), k=8, renorm=1, scale=1.0, ids=at(2), w=at(3), s=None)
BAL = dict(dt=F32_, z=at(0), T=8, E=48, score=0, ids=at(1), k=8, off=at(2), S=2, coef=1.0, loss=at(3), counts=at(4),
           ws=at(5), n=1 << 40, s=None)
GRAD = dict(dt=F32_, z=at(0), T=8, E=48, score=1, ids=at(1), k=8, renorm=1, scale=1.0, dw=at(2), counts=at(3), off=at(4),
            S=2, coef=1.0, dloss=at(5), dz=at(6), s=None)
ROUTER = [("mx_moe_gate", GATE), ("mx_moe_balance", BAL), ("mx_moe_gate_grad", GRAD)]


@pytest.mark.parametrize("name,good", ROUTER)
def test_router_values(L, name, good):
    c = lambda **kw: _call(L, name, good, **kw)
    for kw in (dict(T=-1), dict(T=(1 << 26) + 1), dict(E=0), dict(E=513), dict(k=0), dict(k=-1), dict(T=1 << 26, k=33)):
        assert c(**kw) == SHAPE, kw
    for kw in (dict(dt=3), dict(dt=-1), dict(score=2), dict(score=-1), dict(score=-2 ** 31)):
        assert c(**kw) == FORMAT, kw
    scalar = "coef" if "coef" in good else "scale"
    for bad in (float("nan"), float("inf")):
        assert c(**{scalar: bad}) == VALUE
    if "scale" in good:
        assert c(scale=float("-inf")) == VALUE and c(k=65, E=100) == SHAPE
    if "S" in good:
        for kw in (dict(S=0), dict(S=-1), dict(S=(1 << 20) + 1), dict(S=1 << 20, E=300)):
            assert c(**kw) == SHAPE, kw
        assert c(off=None) == NULL


@pytest.mark.parametrize("name,good", ROUTER)
def test_router_pointers(L, name, good):
    c = lambda **kw: _call(L, name, good, **kw)
    for p, v in good.items():
        if not isinstance(v, int) or v < at(0) or p == "n":
            continue
        if p not in ("bias", "ws", "dw"):
            assert c(**{p: None}) == NULL, p
        if p != "ws":
            assert c(**{p: v + 2}) == ALIGN, p
    assert c(dt=0, z=at(9) + 1) == ALIGN
    outs = {"mx_moe_gate": ("ids", "w"), "mx_moe_balance": ("loss", "counts"), "mx_moe_gate_grad": ("dz",)}[name]
    for o in outs:
        for p, v in good.items():
            if isinstance(v, int) and v >= at(0) and p not in (o, "n", "ws"):
                assert c(**{o: v}) == VALUE and "overlaps" in L.mx_last_error().decode(), (o, p)
    if name != "mx_moe_balance":
        assert c(**_none(good) | dict(T=0, off=at(4), counts=at(3), dloss=at(5)) if "off" in good
                 else _none(good) | dict(T=0)) == 0


def test_gate_k(L):
    assert _call(L, "mx_moe_gate", GATE, E=7) == SHAPE
    assert _call(L, "mx_moe_gate_grad", GRAD, dw=None, dloss=None, counts=None) == NULL
    assert _call(L, "mx_moe_gate_grad", GRAD, dloss=None) == NULL
    assert _call(L, "mx_moe_gate_grad", GRAD, counts=None) == NULL


def test_balance_workspace(L):
    size = L.mx_moe_balance_workspace_size
    assert size(8, 48, 1) == 0 and size(0, 48, 4) == 0
    need = size(4096, 384, 1)
    assert need >= 2 * 384 * 8
    assert _call(L, "mx_moe_balance", BAL, T=4096, E=384, S=1, ws=None) == NULL
    assert _call(L, "mx_moe_balance", BAL, T=4096, E=384, S=1, ws=at(5) + 64) == ALIGN
    assert _call(L, "mx_moe_balance", BAL, T=4096, E=384, S=1, n=need - 1) == WORKSPACE
    for p in ("z", "ids", "loss", "counts", "off"):
        assert _call(L, "mx_moe_balance", BAL, T=4096, E=384, S=1, ws=BAL[p]) == VALUE, p
    for bad in ((-1, 48, 1), (8, 0, 1), (8, 513, 1), (8, 48, 0), (8, 512, 1 << 20), ((1 << 26) + 1, 48, 1)):
        assert size(*bad) == 0


W4 = dict(dt=0, x=at(0), ldx=256, M=4, K=256, fmt=4, w=at(1), scales=at(2), zeros=at(3), group=64, N=96, y=at(4), ldy=96,
          ws=at(5), n=1 << 40, s=None)


def test_w4_values(L):
    c = lambda **kw: _call(L, "mx_w4_linear", W4, **kw)
    for kw in (dict(M=-1), dict(M=(1 << 20) + 1), dict(K=0), dict(K=32), dict(K=320), dict(K=(1 << 20) + 64), dict(N=0),
               dict(N=(1 << 20) + 1), dict(group=16), dict(group=0), dict(group=256), dict(group=-32), dict(ldx=248),
               dict(ldx=260), dict(ldy=95), dict(ldx=1 << 31), dict(ldy=1 << 31), dict(fmt=0, zeros=None)):
        assert c(**kw) == SHAPE, kw
    for kw in (dict(dt=F32_), dict(dt=3), dict(dt=-1), dict(fmt=1), dict(fmt=2), dict(fmt=3), dict(fmt=5), dict(fmt=-1)):
        assert c(**kw) == FORMAT, kw
    assert c(fmt=0, group=32) == VALUE and "zeros" in L.mx_last_error().decode()
    assert c(**_none(W4) | dict(M=0)) == 0
    for bad in ((-1, 64, 64), (1, 0, 64), (1, 64, 0), (1 << 21, 64, 64), (1, 1 << 21, 64), (1, 64, 1 << 21)):
        assert L.mx_w4_linear_workspace_size(*bad) == 0


def test_w4_pointers(L):
    c = lambda **kw: _call(L, "mx_w4_linear", W4, **kw)
    for p in ("x", "w", "scales", "y"):
        assert c(**{p: None}) == NULL, p
    for p, off in (("x", 8), ("w", 8), ("scales", 1), ("y", 1)):
        assert c(**{p: at(20) + off}) == ALIGN, p
    for kw in (dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(0)), dict(y=at(0) + 2 * 256), dict(y=at(1) + 96 * 128 - 2),
               dict(ldx=512, ldy=512, y=at(0) + 2 * 250), dict(ldx=512, ldy=512, y=at(0) + 2 * 450)):
        assert c(**kw) == VALUE and "overlaps" in L.mx_last_error().decode(), kw


def test_w4_workspace(L):
    """None up to 16 tokens; for parts of K, and for the scales of tiles of 256, so many bytes, aligned, apart."""
    size = L.mx_w4_linear_workspace_size
    assert size(16, 1 << 20, 1 << 20) == 0 and size(1, 7168, 7168) == 0 and size(0, 64, 64) == 0
    parts, tables = size(64, 7168, 512), size(4096, 256, 4096)
    assert parts >= 2 * 64 * 512 * 4 and tables >= 2 * 8 * 4096 * 4
    for M, K, N, need in ((64, 7168, 512, parts), (4096, 256, 4096, tables)):
        # operands 2^40 apart
        c = lambda **kw: _call(L, "mx_w4_linear", W4, **(dict(M=M, K=K, N=N, ldx=K, ldy=N, x=1 << 40, w=2 << 40, scales=3 << 40,
                                                              zeros=4 << 40, y=5 << 40, ws=6 << 40) | kw))
        assert c(ws=None) == NULL and c(ws=(6 << 40) + 64) == ALIGN and c(n=need - 1) == WORKSPACE
        for p in (1, 2, 3, 4, 5):
            assert c(ws=p << 40) == VALUE and "overlaps" in L.mx_last_error().decode(), p


WRITE = dict(fmt=3, dt=0, x=at(0), ldx=64, T=4, W=64, slots=at(1), pages=8, page=16, codes=at(2), scales=at(3), s=None)
READ = dict(fmt=0, codes=at(0), scales=at(1), pages=8, page=16, W=64, table=at(2), wide=4, off=at(3), B=2, rows=40, dt=0,
            out=at(4), s=None)


@pytest.mark.parametrize("name,good", [("mx_cache_write", WRITE), ("mx_cache_read", READ)])
def test_cache_values(L, name, good):
    c = lambda **kw: _call(L, name, good, **kw)
    for kw in (dict(W=0), dict(W=16), dict(W=-32), dict(W=48), dict(W=(1 << 16) + 32), dict(pages=-1), dict(page=0),
               dict(page=-1), dict(pages=1 << 27, page=16), dict(pages=1 << 62, page=16), dict(page=1 << 31)):
        assert c(**kw) == SHAPE, kw
    for kw in (dict(fmt=1), dict(fmt=2), dict(fmt=4), dict(fmt=-1), dict(dt=3), dict(dt=-1)):
        assert c(**kw) == FORMAT, kw


def test_cache_sizes(L):
    c = lambda **kw: _call(L, "mx_cache_write", WRITE, **kw)
    for kw in (dict(T=-1), dict(T=1 << 31), dict(T=1 << 28), dict(ldx=56), dict(ldx=68), dict(ldx=1 << 31)):
        assert c(**kw) == SHAPE, kw
    assert c(**_none(WRITE) | dict(T=0)) == 0 and c(**_none(WRITE) | dict(pages=0)) == 0
    c = lambda **kw: _call(L, "mx_cache_read", READ, **kw)
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(B=-1), dict(wide=-1), dict(B=1 << 20, wide=1 << 20),
               dict(B=1 << 31, wide=0)):
        assert c(**kw) == SHAPE, kw
    assert c(**_none(READ) | dict(rows=0)) == 0 and c(**_none(READ) | dict(B=0)) == 0


def test_cache_pointers(L):
    c = lambda **kw: _call(L, "mx_cache_write", WRITE, **kw)
    for p, off in (("x", 8), ("slots", 2), ("codes", 8)):
        assert c(**{p: None}) == NULL and c(**{p: at(20) + off}) == ALIGN, p
    assert c(scales=None) == NULL
    for kw in (dict(codes=at(0)), dict(codes=at(1)), dict(codes=at(3)), dict(scales=at(0)), dict(scales=at(1)),
               dict(scales=at(2) + 8 * 16 * 64 - 1)):
        assert c(**kw) == VALUE and "overlaps" in L.mx_last_error().decode(), kw
    c = lambda **kw: _call(L, "mx_cache_read", READ, **kw)
    for p, off in (("codes", 8), ("table", 2), ("off", 2), ("out", 8)):
        assert c(**{p: None}) == NULL and c(**{p: at(20) + off}) == ALIGN, p
    assert c(scales=None) == NULL
    for p in ("codes", "scales", "table", "off"):
        assert c(out=READ[p]) == VALUE and "overlaps" in L.mx_last_error().decode(), p


# ------------------------------------------------------------------ the binding

def beside(mx):
    """name -> a call of each operator that makes all it can itself."""
    z, ids, dw = t(8, 48, dtype=F32), t(8, 2, dtype=I32), t(8, 2, dtype=F32)
    off, x, w = t(3, dtype=I32), t(4, 128), t(96, 64, dtype=U8)
    codes, scales = t(5, 16, 128, dtype=U8), t(5, 16, 4, dtype=U8)
    return {
        "moe_gate": lambda **k: mx.moe_gate(z, 2, bias=t(48, dtype=F32), **k),
        "moe_balance": lambda **k: mx.moe_balance(z, ids, off, **k),
        "moe_gate_grad": lambda **k: mx.moe_gate_grad(z, ids, dw, t(2, 48, dtype=I32), t(2, dtype=F32), off, **k),
        "w4_linear": lambda **k: mx.w4_linear(x, w, t(96, 2), zeros=t(96, 2, dtype=U8), **k),
        "w4_linear, mxfp4": lambda **k: mx.w4_linear(x, w, t(96, 4, dtype=U8), **k),
        "cache_read": lambda **k: mx.cache_read("mxfp8", codes, scales, t(2, 3, dtype=I32), off, rows=9, **k),
        "cache_write": lambda **k: mx.cache_write("mxfp8", x, t(4, dtype=I32), codes, scales, **k),
    }


@pytest.fixture
def fake(monkeypatch):
    f = stand_in(monkeypatch)
    for name in ("moe_balance", "w4_linear"):       # sizes of this library only
        size = name + "_workspace_size"
        monkeypatch.setattr(f.binding, size, getattr(f.binding, size).__wrapped__)
    return f


@pytest.mark.parametrize("name", sorted(beside(None)))
def test_memory_of_a_call_is_the_given_streams(fake, name):
    s = Stream()
    out = beside(fake.binding)[name](stream=s)
    assert fake.lib.streams == [s.cuda_stream]
    assert (name == "cache_write" or fake.torch.made) and all(m.made_on is s for m in fake.torch.made)
    out = [o for o in (out if isinstance(out, tuple) else (out,)) if o in fake.torch.made]
    assert all(o.told for o in out)
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        beside(fake.binding)[name](stream=Stream(torch.device("cuda", 1)))
    assert len(fake.lib.streams) == 1


def _grad_calls(mx):
    """name -> (call, its float arguments by name), and what of them is written."""
    z, w, loss, x, y = t(8, 48, dtype=F32), t(8, 2, dtype=F32), t(1, dtype=F32), t(4, 128), t(4, 96)
    ids, counts = t(8, 2, dtype=I32), t(1, 48, dtype=I32)
    codes, scales, slots = t(5, 16, 128, dtype=U8), t(5, 16, 4, dtype=U8), t(4, dtype=I32)
    return {
        "gate": (lambda a: mx.moe_gate(a["z"], 2, bias=a["b"], topk_ids=ids, topk_w=a["w"]),
                 dict(z=z, b=t(48, dtype=F32), w=w), {"w"}),
        "balance": (lambda a: mx.moe_balance(a["z"], ids, loss=a["l"], counts=counts), dict(z=z, l=loss), {"l"}),
        "grad": (lambda a: mx.moe_gate_grad(a["z"], ids, a["dw"], counts, a["dl"], d_logits=a["dz"]),
                 dict(z=z, dw=w, dl=loss, dz=t(8, 48, dtype=F32)), {"dz"}),
        "w4": (lambda a: mx.w4_linear(a["x"], t(96, 64, dtype=U8), a["s"], out=a["y"]), dict(x=x, s=t(96, 2), y=y), {"y"}),
        "write": (lambda a: mx.cache_write("mxfp8", a["x"], slots, codes, scales), dict(x=x), set()),
        "read": (lambda a: mx.cache_read("mxfp8", codes, scales, t(2, 3, dtype=I32), t(3, dtype=I32), out=a["o"]),
                 dict(o=t(9, 128)), {"o"}),
    }


CASES = [(n, a) for n, (_, args, _) in _grad_calls(None).items() for a in args]


@pytest.mark.parametrize("name,arg", CASES)
def test_an_input_that_requires_a_gradient_is_refused(fake, name, arg):
    call, args, written = _grad_calls(fake.binding)[name]
    args[arg].requires_grad = True
    with pytest.raises(ValueError, match="requires a gradient"):
        call(args)
    assert not fake.lib.streams and not fake.torch.written
    with torch.no_grad():
        call(args)
    assert len(fake.lib.streams) == 1
    told = {id(v) for v in fake.torch.written}
    assert {id(args[k]) for k in written} <= told
    if name == "write":
        assert len(told) == 2


def test_the_binding_refuses(fake):
    mx = fake.binding
    z, ids = t(8, 48, dtype=F32), t(8, 2, dtype=I32)
    x, w = t(4, 128), t(96, 64, dtype=U8)
    codes, scales = t(5, 16, 128, dtype=U8), t(5, 16, 4, dtype=U8)
    table, off = t(2, 3, dtype=I32), t(3, dtype=I32)
    for call, what in (
            (lambda: mx.moe_gate(z, 0), "k 0"), (lambda: mx.moe_gate(z, 49), "k 49"), (lambda: mx.moe_gate(z, 2, score="x"), "score"),
            (lambda: mx.moe_gate(z, 2, bias=t(47, dtype=F32)), "bias"), (lambda: mx.moe_gate(z, 2, bias=t(48)), "bias"),
            (lambda: mx.moe_gate(t(8, 48, dtype=I32), 2), "logits"),
            (lambda: mx.moe_balance(z, t(7, 2, dtype=I32)), "topk_ids"), (lambda: mx.moe_balance(z, ids, t(1, dtype=I32)), "seq_off"),
            (lambda: mx.moe_gate_grad(z, ids), "nothing to do"),
            (lambda: mx.moe_gate_grad(z, ids, counts=t(1, 48, dtype=I32)), "nothing to do"),
            (lambda: mx.moe_gate_grad(z, ids, t(8, 2, dtype=F32), counts=t(1, 48, dtype=I32)), "go together"),
            (lambda: mx.w4_linear(x, w, t(96, 3)), "w_s"), (lambda: mx.w4_linear(x, w, t(96, 8)), "w_s"),
            (lambda: mx.w4_linear(x, w, t(96, 2, dtype=U8)), "w_s"), (lambda: mx.w4_linear(x, t(96, 63, dtype=U8), t(96, 2)), "w must"),
            (lambda: mx.w4_linear(x, w, t(96, 2, dtype=F32)), "w_s"), (lambda: mx.w4_linear(x, w, t(96, 0)), "w_s"),
            (lambda: mx.w4_linear(x, w, t(96, 4, dtype=U8), zeros=t(96, 4, dtype=U8)), "no zeros"),
            (lambda: mx.w4_linear(x, w, t(96, 2), out=t(4, 95)), "out"), (lambda: mx.w4_linear(x, w, t(96, 2), out=t(3, 96)), "out"),
            (lambda: mx.cache_write("nvfp4", x, t(4, dtype=I32), codes, scales), "format"),
            (lambda: mx.cache_write("mxfp4", x, t(4, dtype=I32), codes, scales), "codes"),
            (lambda: mx.cache_write("mxfp8", t(4, 96), t(4, dtype=I32), codes, scales), "columns"),
            (lambda: mx.cache_write("mxfp8", x, t(3, dtype=I32), codes, scales), "slots"),
            (lambda: mx.cache_read("mxfp8", codes, scales, table, off), "rows or out"),
            (lambda: mx.cache_read("mxfp8", codes, scales, table, t(2, dtype=I32), rows=3), "seq_off"),
            (lambda: mx.cache_read("mxfp8", codes, scales, table, off, rows=3, out=t(4, 128)), "out"),
            (lambda: mx.cache_read("mxfp8", codes, scales, table, off, rows=3, dtype=I32), "out"),
            (lambda: mx.cache_read("mxfp8", codes, scales, table, off, out=t(4, 96)), "out")):
        with pytest.raises(ValueError, match=what):
            call()
    assert not fake.lib.streams


def test_cpu_tensors_are_refused():
    import mxfp4_block_scaled_e2m1_amd as mx
    z, i, u = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=I32), torch.zeros((2, 4, 2), dtype=U8)
    for call in (lambda: mx.moe_gate(z, 2), lambda: mx.moe_balance(z, i), lambda: mx.moe_gate_grad(z, i, z[:, :2]),
                 lambda: mx.w4_linear(z.to(BF16), u[0], u[0]), lambda: mx.cache_write("mxfp8", z, i[:, 0], u, u),
                 lambda: mx.cache_read("mxfp8", u, u, i, i[:, 0], rows=4)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the same under the sanitizers

@pytest.mark.timeout(600)
def test_under_the_host_sanitizers():
    """These checks against a build whose host code runs under AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("MXFP4_LIB"):
        pytest.skip("already on a chosen build")
    from mxfp4_block_scaled_e2m1_amd import build
    try:
        runtime = build.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    if not os.path.exists(build.LIB_SAN) or os.path.getmtime(build.LIB_SAN) < A._newest(build.CSRC):
        build.build(jobs=8, sanitize=True)
    env = dict(os.environ)
    env.update(LD_PRELOAD=runtime, MXFP4_LIB=build.LIB_SAN,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-s", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=500)
    out = r.stdout + r.stderr
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]
