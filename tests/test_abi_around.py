"""The operators around the experts: host-side validation of the C ABI (nothing here reaches a kernel) and of
the binding's own checks, on the CPU; the same checks again under the host sanitizers."""

import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, VALUE = 1, 2, 3, 4, 5, 7
BF16, F16, F32 = 0, 1, 2


def at(i):
    """A distinct, 1 TiB apart, never dereferenced address."""
    return (i + 1) << 40


@pytest.fixture(scope="module")
def L():
    from mxfp4_block_scaled_e2m1_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def _err(L):
    return L.mx_last_error().decode()


def _call(L, name, good, order, **over):
    kw = {**good, **over}
    return getattr(L, name)(*[kw[k] for k in order])


# ------------------------------------------------------------------ sort

SORT = dict(ids=at(0), T=8, k=8, E=48, off=at(1), rs=at(2), sr=at(3), ws=at(4), n=1 << 40, s=None)


def _sort(L, **over):
    return _call(L, "mx_moe_sort", SORT, list(SORT), **over)


def test_sort_sizes(L):
    for kw in (dict(T=-1), dict(k=0), dict(k=-3), dict(E=0), dict(E=513), dict(T=1 << 30, k=2), dict(T=1 << 62, k=8)):
        assert _sort(L, **kw) == SHAPE, kw
    size = L.mx_moe_sort_workspace_size
    assert size(8, 8, 48) == 0 and size(4096, 1, 2) == 0
    assert size(4096, 8, 48) >= 32 * 48 * 4 and size(4097, 1, 1) > 0
    assert size(64, 64, 512) > 0                       # few pairs, but their counts do not fit one workgroup
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 513), (1 << 62, 8, 8)):
        assert size(*bad) == 0


def test_sort_pointers(L):
    for p in ("ids", "off", "rs", "sr"):
        assert _sort(L, **{p: None}) == NULL, p
        assert _sort(L, **{p: at(20) + 2}) == ALIGN, p
    assert _sort(L, T=4096, ws=None) == NULL
    assert _sort(L, T=4096, ws=at(4) + 128) == ALIGN
    need = L.mx_moe_sort_workspace_size(4096, 8, 48)
    assert _sort(L, T=4096, n=need - 1) == WORKSPACE and "workspace" in _err(L)
    for kw in (dict(rs=at(3)), dict(off=at(0) + 16), dict(sr=at(0)), dict(rs=at(2), off=at(2) + 64 * 4 - 4)):
        assert _sort(L, **kw) == VALUE and "overlaps" in _err(L), kw
    assert _sort(L, T=4096, ws=at(0) + 256) == VALUE


# ------------------------------------------------------------------ rows

PERM = dict(dt=BF16, x=at(0), T=4, H=64, sr=at(1), k=2, rows=8, xs=at(2), s=None)
UNPERM = dict(dt=BF16, ys=at(0), rows=8, H=64, sr=at(1), w=at(2), T=4, k=2, y=at(3), s=None)
GRAD = dict(dt=BF16, dy=at(0), ys=at(1), rows=8, H=64, sr=at(2), w=at(3), T=4, k=2, dys=at(4), dw=at(5), s=None)
ROWS = [("mx_moe_permute", PERM), ("mx_moe_unpermute", UNPERM), ("mx_moe_unpermute_grad", GRAD)]


@pytest.mark.parametrize("name,good", ROWS)
def test_rows_sizes(L, name, good):
    for kw in (dict(H=0), dict(H=-8), dict(H=(1 << 20) + 1), dict(T=-1), dict(k=0), dict(rows=-1),
               dict(rows=(1 << 30) + 1), dict(T=1 << 30, k=4)):
        assert _call(L, name, good, list(good), **kw) == SHAPE, kw
    for dt in (-1, 3, 99):
        assert _call(L, name, good, list(good), dt=dt) == FORMAT
    empty = {k: (None if isinstance(v, int) and v >= at(0) else v) for k, v in good.items()}
    assert _call(L, name, empty, list(good), T=0) == 0


@pytest.mark.parametrize("name,good", ROWS)
def test_rows_pointers(L, name, good):
    for p, v in good.items():
        if p in ("s", "dt", "T", "H", "k", "rows"):
            continue
        if not (name == "mx_moe_unpermute" and p == "w"):       # its weights are optional
            assert _call(L, name, good, list(good), **{p: None}) == NULL, p
        assert _call(L, name, good, list(good), **{p: v + 1}) == ALIGN, p
        if p in ("sr", "w", "dw"):
            assert _call(L, name, good, list(good), **{p: v + 2}) == ALIGN, p
    assert _call(L, name, good, list(good), dt=F32, **{"xs" if "xs" in good else "ys": at(9) + 2}) == ALIGN


def test_rows_overlap(L):
    over = lambda name, good, **kw: (_call(L, name, good, list(good), **kw), "overlaps" in _err(L))
    assert over("mx_moe_permute", PERM, xs=at(0)) == (VALUE, True)
    assert over("mx_moe_permute", PERM, xs=at(0) + 4 * 64 * 2 - 2) == (VALUE, True)
    assert over("mx_moe_unpermute", UNPERM, y=at(0) + 128) == (VALUE, True)
    assert over("mx_moe_unpermute", UNPERM, y=at(2)) == (VALUE, True)
    assert over("mx_moe_unpermute_grad", GRAD, dys=at(1)) == (VALUE, True)
    assert over("mx_moe_unpermute_grad", GRAD, dw=at(3)) == (VALUE, True)
    assert over("mx_moe_unpermute_grad", GRAD, dw=at(4) + 64) == (VALUE, True)


# ------------------------------------------------------------------ norms

NORM = dict(dt=BF16, rdt=F32, y=at(0), res=at(1), wpost=at(2), kind=1, gate=at(3), scale=1.0, wpre=at(4), eps=1e-6,
            T=4, H=64, ro=at(5), normed=at(6), s=None)
NGRAD = dict(dt=BF16, rdt=F32, y=at(0), ro=at(1), wpost=at(2), kind=1, gate=at(3), scale=1.0, wpre=at(4), eps=1e-6,
             T=4, H=64, dn=at(5), dro=at(6), dres=at(7), dy=at(8), dgate=at(9), dwpost=at(10), dwpre=at(11),
             ws=at(12), n=1 << 30, s=None)
NORMS = [("mx_block_norm", NORM), ("mx_block_norm_grad", NGRAD)]


@pytest.mark.parametrize("name,good", NORMS)
def test_norm_values(L, name, good):
    c = lambda **kw: _call(L, name, good, list(good), **kw)
    for kw in (dict(H=0), dict(H=16385), dict(T=-1), dict(T=(1 << 30) + 1)):
        assert c(**kw) == SHAPE, kw
    for kw in (dict(dt=3), dict(dt=-1), dict(rdt=F16), dict(dt=F32, rdt=BF16), dict(kind=4), dict(kind=-1)):
        assert c(**kw) == FORMAT, kw
    for kw in (dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("inf")),
               dict(scale=float("nan"))):
        assert c(**kw) == VALUE, kw
    assert c(kind=0) == VALUE and "gate" in _err(L)            # a gate that no kind names
    assert c(gate=None) == NULL


def test_norm_pointers(L):
    c = lambda **kw: _call(L, "mx_block_norm", NORM, list(NORM), **kw)
    for p in ("res", "ro", "normed"):
        assert c(**{p: None}) == NULL, p
    assert c(y=None) == VALUE                                   # w_post and gate without y
    assert c(y=None, wpost=None, kind=0, gate=None) == VALUE    # residual_out without y
    assert c(y=None, wpost=None, kind=0, gate=None, ro=None, wpre=None, normed=None) == NULL
    assert c(wpre=None) == VALUE                                # normed without w_pre
    for p in ("y", "wpost", "gate", "wpre", "normed"):
        assert c(**{p: at(20) + 1}) == ALIGN, p
    for p in ("res", "ro"):
        assert c(**{p: at(20) + 2}) == ALIGN, p
    for kw in (dict(ro=at(0)), dict(ro=at(1) + 256), dict(normed=at(1)), dict(normed=at(0) + 2), dict(normed=at(4)),
               dict(ro=at(6))):
        assert c(**kw) == VALUE and "overlaps" in _err(L), kw


def test_norm_grad_pointers(L):
    c = lambda **kw: _call(L, "mx_block_norm_grad", NGRAD, list(NGRAD), **kw)
    for p in ("ro", "dn", "dres", "dy", "dgate", "dwpost", "dwpre", "ws"):
        assert c(**{p: None}) == NULL, p
    assert c(wpre=None) == VALUE and c(wpre=None, dwpre=None) == VALUE          # dw_pre, then d_normed, left over
    assert c(wpre=None, dwpre=None, dn=None, dro=None) == NULL
    assert c(wpost=None) == VALUE and "dw_post" in _err(L)
    assert c(kind=0, gate=None) == VALUE and "d_gate" in _err(L)
    assert c(y=None, wpost=None, dwpost=None, kind=0, gate=None, dgate=None) == VALUE and "d_y" in _err(L)
    for p, a in dict(y=2, dn=2, dy=2, gate=2, dgate=4, ro=4, dro=4, dres=4, dwpre=4, dwpost=4).items():
        assert c(**{p: at(20) + a // 2}) == ALIGN, p
    assert c(ws=at(12) + 128) == ALIGN
    need = L.mx_block_norm_grad_workspace_size(4, 64)
    assert need >= 4 * 2 * 64 * 4 and c(n=need - 1) == WORKSPACE
    for kw in (dict(dres=at(1)), dict(dy=at(1)), dict(dy=at(5) + 2), dict(dres=at(6) + 4), dict(dwpre=at(10)),
               dict(dgate=at(0)), dict(ws=at(5)), dict(dres=at(8))):
        assert c(**kw) == VALUE and "overlaps" in _err(L), kw
    assert L.mx_block_norm_grad_workspace_size(0, 64) == 0
    for bad in ((-1, 8), (4, 0), (4, 16385)):
        assert L.mx_block_norm_grad_workspace_size(*bad) == 0


# ------------------------------------------------------------------ adapters

LORA = dict(dt=BF16, x=at(0), ldx=64, M=4, K=64, a=at(1), b=at(2), scale=at(3), n=2, R=16, off=at(4), tok=at(5),
            y=at(6), ldy=128, N=128, ws=at(7), wn=1 << 30, s=None)


def test_lora_values(L):
    c = lambda **kw: _call(L, "mx_lora_add", LORA, list(LORA), **kw)
    for kw in (dict(M=-1), dict(M=(1 << 24) + 1), dict(K=0), dict(K=60), dict(K=1 << 21), dict(N=4), dict(N=132),
               dict(R=0), dict(R=12), dict(R=136), dict(n=0), dict(n=513), dict(ldx=56), dict(ldx=68), dict(ldy=120),
               dict(ldy=132), dict(ldx=1 << 31)):
        assert c(**kw) == SHAPE, kw
    for dt in (F32, 3, -1):
        assert c(dt=dt) == FORMAT
    none = {k: None for k in ("x", "a", "b", "scale", "off", "tok", "y", "ws")}
    assert c(M=0, **none) == 0
    size = L.mx_lora_add_workspace_size
    assert size(4, 64, 16, 2) >= 4 * 16 * 4
    for bad in ((-1, 64, 16, 2), (4, 0, 16, 2), (4, 64, 0, 2), (4, 64, 136, 2), (4, 64, 16, 0), (4, 64, 16, 513)):
        assert size(*bad) == 0


def test_lora_pointers(L):
    c = lambda **kw: _call(L, "mx_lora_add", LORA, list(LORA), **kw)
    for p in ("x", "a", "b", "off", "tok", "y", "ws"):
        assert c(**{p: None}) == NULL, p
    for p in ("x", "a", "b", "y"):
        assert c(**{p: at(20) + 8}) == ALIGN, p
    for p in ("scale", "off", "tok"):
        assert c(**{p: at(20) + 2}) == ALIGN, p
    assert c(ws=at(7) + 128) == ALIGN
    assert c(wn=L.mx_lora_add_workspace_size(4, 64, 16, 2) - 1) == WORKSPACE
    for kw in (dict(y=at(1)), dict(y=at(2) + 16), dict(ws=at(6)), dict(ws=at(0)), dict(y=at(0)),
               dict(y=at(0) + 2 * 64, ldy=128), dict(x=at(6) + 32, ldx=256, ldy=256)):
        assert c(**kw) == VALUE and "overlaps" in _err(L), kw
    # column ranges of one matrix that overlap, in either order
    assert c(ldx=256, ldy=256, y=at(0) + 2 * 56) == VALUE
    assert c(ldx=256, ldy=256, y=at(0) + 2 * 136) == VALUE


def test_binding_refuses_before_the_library(L):
    """CPU tensors, wrong types and shapes raise without a call."""
    import torch
    import mxfp4_block_scaled_e2m1_amd as mx
    ids = torch.zeros((2, 2), dtype=torch.int32)
    x = torch.zeros((2, 8), dtype=torch.bfloat16)
    for call in (lambda: mx.moe_sort(ids, 4), lambda: mx.moe_permute(x, ids), lambda: mx.moe_unpermute(x, ids),
                 lambda: mx.moe_unpermute_grad(x, x, ids, ids.float()), lambda: mx.block_norm(x, x[0]),
                 lambda: mx.block_norm(x), lambda: mx.block_norm_grad(x, x[0], x),
                 lambda: mx.lora_add(x, x, x[None], x[None], ids[0], ids[0])):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the same under the sanitizers

def _newest(folder):
    return max(os.path.getmtime(os.path.join(folder, f)) for f in os.listdir(folder))


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
    if not os.path.exists(build.LIB_SAN) or os.path.getmtime(build.LIB_SAN) < _newest(build.CSRC):
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
