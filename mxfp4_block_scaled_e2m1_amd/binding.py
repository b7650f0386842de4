"""Thin ctypes binding of libmxfp4 (include/mxfp4.h): argument marshalling only.

Every step of the path runs in the HIP library; this module only turns torch
device tensors into pointers and the current torch stream into a hipStream_t,
and raises MxError when the library reports a failure. There is no fallback:
if the library is missing, calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# MXFP4_LIB selects another build of the same library (the host-sanitized copy
# the CPU tests load); by default the in-tree libmxfp4.so.
LIB_PATH = os.environ.get("MXFP4_LIB") or os.path.join(HERE, "libmxfp4.so")

MX_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MX_GATE = {"none": 0, "channel": 1, "token": 2, "full": 3}
MX_FMT = {"mxfp4": 0, "fp8_b128": 1, "nvfp4": 2, "mxfp8": 3}
STATUS = {0: "MX_OK", 1: "MX_ERR_NULL", 2: "MX_ERR_SHAPE", 3: "MX_ERR_ALIGN", 4: "MX_ERR_FORMAT",
          5: "MX_ERR_WORKSPACE", 6: "MX_ERR_HIP", 7: "MX_ERR_VALUE"}

#: name -> (restype, argtypes) for every symbol declared in include/mxfp4.h
_P, _I64, _I32, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


class PhaseStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("total_ms", ctypes.c_double), ("launches", ctypes.c_int64)]


SIGNATURES = {
    "mx_dequant": (_I32, [_I32, _P, _P, _P, _I64, _I64, _P, _P]),
    "mx_quantize_act": (_I32, [_I32, _P, _I64, _I64, _P, _P, _P, _P]),
    "mx_expert_mlp": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "mx_nvfp4_global_warmup": (_I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                      _P]),
    "mx_nvfp4_global_warmup_workspace_size": (_SZ, [_I64, _I64, _I64, _I32, _I32]),
    "mx_expert_mlp_workspace_size": (_SZ, [_I64, _I64, _I64, _I32]),
    "mx_expert_mlp_noalloc": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P]),
    "mx_expert_mlp_noalloc_max_bytes": (_SZ, []),
    "mx_grouped_expert_mlp": (_I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                     _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "mx_grouped_expert_mlp_workspace_size": (_SZ, [_I64, _I64, _I64, _I32, _I32, _I32]),
    "mx_pack_weight_scales": (_I32, [_P, _P, _P, _I64, _I64, _I32, _P, _SZ, _P]),
    "mx_packed_weight_scales_size": (_SZ, [_I64, _I64, _I32]),
    "mx_pack_weight_codes": (_I32, [_P, _P, _P, _I64, _I64, _I32, _P, _SZ, _P]),
    "mx_packed_weight_codes_size": (_SZ, [_I64, _I64, _I32]),
    "mx_debug_gemm_f32": (_I32, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P]),
    "mx_fp8_block_linear": (_I32, [_P, _I64, _I64, _P, _P, _I64, _P, _P, _SZ, _P]),
    "mx_fp8_block_linear_workspace_size": (_SZ, [_I64, _I64]),
    "mx_nvfp4_linear": (_I32, [_P, _I64, _I64, _P, _P, _F, _I64, _F, _P, _P, _SZ, _P]),
    "mx_nvfp4_linear_workspace_size": (_SZ, [_I64, _I64]),
    "mx_nvfp4_expert_mlp": (_I32, [_P, _I64, _I64, _I64, _P, _P, _F, _P, _P, _F, _P, _P, _F, _F, _F, _P, _P, _SZ,
                                   _P]),
    "mx_nvfp4_expert_mlp_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "mx_grouped_nvfp4_expert_mlp": (_I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _P, _F, _F, _P, _P, _SZ, _P]),
    "mx_grouped_nvfp4_expert_mlp_workspace_size": (_SZ, [_I64, _I64, _I64, _I32, _I32]),
    "mx_fp8_expert_mlp": (_I32, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "mx_fp8_expert_mlp_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "mx_moe_runner_create": (_I32, [_P, _I64, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _I32, _P, _P, ctypes.POINTER(_P)]),
    "mx_moe_runner_replay": (_I32, [_P, _P]),
    "mx_moe_runner_destroy": (_I32, [_P]),
    "mx_status_string": (ctypes.c_char_p, [_I32]),
    "mx_last_error": (ctypes.c_char_p, []),
    "mx_profile_start": (_I32, []),
    "mx_profile_stop": (_I32, [ctypes.POINTER(PhaseStat), _I32, ctypes.POINTER(_I32)]),
    "mx_moe_sort": (_I32, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "mx_moe_sort_workspace_size": (_SZ, [_I64, _I32, _I32]),
    "mx_moe_permute": (_I32, [_I32, _P, _I64, _I64, _P, _I32, _I64, _P, _P]),
    "mx_moe_unpermute": (_I32, [_I32, _P, _I64, _I64, _P, _P, _I64, _I32, _P, _P]),
    "mx_moe_unpermute_grad": (_I32, [_I32, _P, _P, _I64, _I64, _P, _P, _I64, _I32, _P, _P, _P]),
    "mx_block_norm": (_I32, [_I32, _I32, _P, _P, _P, _I32, _P, _F, _P, _F, _I64, _I64, _P, _P, _P]),
    "mx_block_norm_grad": (_I32, [_I32, _I32, _P, _P, _P, _I32, _P, _F, _P, _F, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                  _P, _P, _SZ, _P]),
    "mx_block_norm_grad_workspace_size": (_SZ, [_I64, _I64]),
    "mx_lora_add": (_I32, [_I32, _P, _I64, _I64, _I64, _P, _P, _P, _I32, _I64, _P, _P, _P, _I64, _I64, _P, _SZ, _P]),
    "mx_lora_add_workspace_size": (_SZ, [_I64, _I64, _I64, _I32]),
    "mx_probe_mfma_fp4": (_I32, [_P, _I64, _I32, _P, _P]),
    "mx_probe_read": (_I32, [_I32, _I32, _I32, _P, _I64, _P, _P]),
    "mx_probe_copy": (_I32, [_P, _P, _I64, _P]),
}

_lib = None


class MxError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


def lib():
    """Load libmxfp4.so (built in-tree). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mxfp4_block_scaled_e2m1_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise MxError(status, lib().mx_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmxfp4 takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libmxfp4 takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _made(stream, make, *args, **kwargs):
    """make(...): an output that a call on the given `stream` makes itself, from that stream's memory. A block of the
    current stream's may still be in use there by work that `stream` does not wait for. The current stream is
    made known to the tensor, since the caller will mostly go on with it there."""
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty(shape, dtype, device, stream):
    """torch.empty for an output of a call on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _made(stream, torch.empty, shape, dtype=dtype, device=device)


def _fmt(f) -> int:
    return MX_FMT[f] if isinstance(f, str) else int(f)


def _global(g, device, stream=None):
    """An NVFP4 global scale as the library takes it: a one-element fp32 device
    tensor (passed through), a Python float (copied into a new device tensor),
    or None. Returns the tensor, which the caller keeps alive until the call
    that reads it has been made (a temporary is memory of that call's stream)."""
    if g is None:
        return None
    if isinstance(g, torch.Tensor):
        if g.dtype != torch.float32 or g.numel() != 1:
            raise ValueError("a global scale tensor must hold one fp32 value")
        return g
    with torch.cuda.stream(stream):
        return torch.tensor([float(g)], dtype=torch.float32, device=device)


# ---------------------------------------------------------------------------

def dequant(fmt, codes, scales, rows: int, cols: int, global_scale=None, out=None, stream=None):
    """mx_dequant -> bf16 tensor [rows, cols]. global_scale (NVFP4): float or
    one-element fp32 device tensor."""
    if out is None:
        out = _empty((rows, cols), torch.bfloat16, codes.device, stream)
    g = _global(global_scale, codes.device, stream)
    _check(lib().mx_dequant(_fmt(fmt), _ptr(codes), _ptr(scales), _ptr(g), rows, cols,
                            _ptr(out), _stream(stream)))
    return out


def quantize_act(fmt, x, global_scale=None, codes=None, scales=None, stream=None):
    """mx_quantize_act: bf16 x [rows, cols] -> (codes [rows, cols/2], or [rows, cols]
    for MXFP8, scales). global_scale (NVFP4): float or one-element fp32 device tensor."""
    rows, cols = x.shape
    f = _fmt(fmt)
    per = 16 if f == MX_FMT["nvfp4"] else 32
    if codes is None:
        width = cols if f == MX_FMT["mxfp8"] else cols // 2
        codes = _empty((rows, width), torch.uint8, x.device, stream)
    if scales is None:
        scales = _empty((rows, cols // per), torch.uint8, x.device, stream)
    g = _global(global_scale, x.device, stream)
    _check(lib().mx_quantize_act(f, _ptr(x), rows, cols, _ptr(g), _ptr(codes), _ptr(scales),
                                 _stream(stream)))
    return codes, scales


def expert_mlp_workspace_size(M, hidden, inter, requant="mxfp4") -> int:
    return int(lib().mx_expert_mlp_workspace_size(M, hidden, inter, _fmt(requant)))


def grouped_expert_mlp_workspace_size(T, hidden, inter, k, E, requant="mxfp4") -> int:
    return int(lib().mx_grouped_expert_mlp_workspace_size(T, hidden, inter, k, E, _fmt(requant)))


def _workspace(nbytes, device, workspace, stream):
    """`workspace`, or memory of the call's stream: let go of afterwards, it comes back for later work of that
    stream only."""
    if workspace is not None:
        return workspace
    if stream is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def packed_weight_scales_size(hidden, inter, E=1) -> int:
    return int(lib().mx_packed_weight_scales_size(hidden, inter, E))


def pack_weight_scales(w1s, w3s, w2s, out=None, stream=None):
    """mx_pack_weight_scales: tile-major copy of the weight scales of one expert
    (w1s [inter, hidden/32]) or of E stacked experts (w1s [E, inter, hidden/32])."""
    E = w1s.shape[0] if w1s.dim() == 3 else 1
    inter, hidden = w1s.shape[-2], 32 * w1s.shape[-1]
    nbytes = packed_weight_scales_size(hidden, inter, E)
    if out is None:
        out = _empty(nbytes, torch.uint8, w1s.device, stream)
    _check(lib().mx_pack_weight_scales(_ptr(w1s), _ptr(w3s), _ptr(w2s), hidden, inter, E, _ptr(out),
                                       out.numel(), _stream(stream)))
    return out


def packed_weight_codes_size(hidden, inter, E=1) -> int:
    return int(lib().mx_packed_weight_codes_size(hidden, inter, E))


def pack_weight_codes(w1, w3, w2, out=None, stream=None):
    """mx_pack_weight_codes: tile-major copy of the weight codes of one expert
    (w1 [inter, hidden/2]) or of E stacked experts (w1 [E, inter, hidden/2])."""
    E = w1.shape[0] if w1.dim() == 3 else 1
    inter, hidden = w1.shape[-2], 2 * w1.shape[-1]
    nbytes = packed_weight_codes_size(hidden, inter, E)
    if out is None:
        out = _empty(nbytes, torch.uint8, w1.device, stream)
    _check(lib().mx_pack_weight_codes(_ptr(w1), _ptr(w3), _ptr(w2), hidden, inter, E, _ptr(out), out.numel(),
                                      _stream(stream)))
    return out


def expert_mlp(x, w1, w1s, w3, w3s, w2, w2s, requant="mxfp4", requant_global=None,
               out=None, workspace=None, stream=None, packed_scales=None, packed_codes=None):
    """mx_expert_mlp: the shared expert on bf16 x [M, hidden] -> bf16 y [M, hidden].
    requant_global (NVFP4): float or one-element fp32 device tensor."""
    M, hidden = x.shape
    inter = w1.shape[0]
    if out is None:
        out = _empty((M, hidden), torch.bfloat16, x.device, stream)
    nbytes = expert_mlp_workspace_size(M, hidden, inter, requant)
    ws = _workspace(nbytes, x.device, workspace, stream)
    g = _global(requant_global, x.device, stream)
    _check(lib().mx_expert_mlp(_ptr(x), M, hidden, inter, _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s),
                               _ptr(w2), _ptr(w2s), _ptr(packed_scales), _ptr(packed_codes), _fmt(requant),
                               _ptr(g), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def expert_mlp_noalloc(x, w1, w1s, w3, w3s, w2, w2s, requant="mxfp4", requant_global=None, out=None,
                       stream=None, packed_scales=None, packed_codes=None):
    """mx_expert_mlp_noalloc: mx_expert_mlp on the library's fixed device scratch
    (no workspace argument; calls on one GPU must not overlap)."""
    M, hidden = x.shape
    inter = w1.shape[0]
    if out is None:
        out = _empty((M, hidden), torch.bfloat16, x.device, stream)
    g = _global(requant_global, x.device, stream)
    _check(lib().mx_expert_mlp_noalloc(_ptr(x), M, hidden, inter, _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s),
                                       _ptr(w2), _ptr(w2s), _ptr(packed_scales), _ptr(packed_codes),
                                       _fmt(requant), _ptr(g), _ptr(out), _stream(stream)))
    return out


def grouped_expert_mlp(x, topk_ids, topk_w, w1, w1s, w3, w3s, w2, w2s, requant="mxfp4",
                       requant_global=None, out=None, workspace=None, stream=None, packed_scales=None,
                       packed_codes=None):
    """mx_grouped_expert_mlp: routed experts, stacked weights [E, ...]. requant_global
    (NVFP4): float or one-element fp32 device tensor."""
    T, hidden = x.shape
    k = topk_ids.shape[1]
    E, inter = w1.shape[0], w1.shape[1]
    if out is None:
        out = _empty((T, hidden), torch.bfloat16, x.device, stream)
    nbytes = grouped_expert_mlp_workspace_size(T, hidden, inter, k, E, requant)
    ws = _workspace(nbytes, x.device, workspace, stream)
    g = _global(requant_global, x.device, stream)
    _check(lib().mx_grouped_expert_mlp(_ptr(x), T, hidden, inter, _ptr(topk_ids), _ptr(topk_w), k, E,
                                       _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s), _ptr(w2), _ptr(w2s),
                                       _ptr(packed_scales), _ptr(packed_codes), _fmt(requant), _ptr(g),
                                       _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def nvfp4_global_warmup(x, w1, w1s, w3, w3s, topk_ids=None, topk_w=None, packed_scales=None, out=None,
                        workspace=None, stream=None):
    """mx_nvfp4_global_warmup: g = f32(max |h| / (6 * 448)) of a warm-up batch, as a
    one-element fp32 device tensor. One expert (w1 [inter, hidden/2]) when
    topk_ids is None, else routed over stacked weights [E, ...]."""
    T, hidden = x.shape
    routed = topk_ids is not None
    inter = w1.shape[-2]
    k = topk_ids.shape[1] if routed else 0
    E = w1.shape[0] if routed else 1
    if out is None:
        out = _empty((1,), torch.float32, x.device, stream)
    nbytes = int(lib().mx_nvfp4_global_warmup_workspace_size(T, hidden, inter, k, E))
    ws = _workspace(nbytes, x.device, workspace, stream)
    _check(lib().mx_nvfp4_global_warmup(_ptr(x), T, hidden, inter, _ptr(topk_ids), _ptr(topk_w), k, E,
                                        _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s), _ptr(packed_scales), _ptr(out),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def debug_gemm_f32(a, a_s, b, b_s, out=None, stream=None):
    """mx_debug_gemm_f32: C [M, N] = A . B^T for MXFP4 A [M, K/2] and B [N, K/2]."""
    M, N, K = a.shape[0], b.shape[0], 2 * a.shape[1]
    if out is None:
        out = _empty((M, N), torch.float32, a.device, stream)
    _check(lib().mx_debug_gemm_f32(_ptr(a), _ptr(a_s), _ptr(b), _ptr(b_s), M, N, K, _ptr(out),
                                   _stream(stream)))
    return out


def profile_start():
    _check(lib().mx_profile_start())


def profile_stop():
    """Returns {kernel name: (total_ms, launches)} for launches since profile_start()."""
    buf = (PhaseStat * 64)()
    n = _I32(0)
    _check(lib().mx_profile_stop(buf, 64, ctypes.byref(n)))
    return {buf[i].name.decode(): (buf[i].total_ms, int(buf[i].launches)) for i in range(min(n.value, 64))}


def probe_mfma_fp4(operands, iters: int, workgroups: int, out=None, stream=None):
    """mx_probe_mfma_fp4: operands uint32 [512, 16] (device); returns float32 [workgroups, 512]."""
    if out is None:
        out = _empty((workgroups, 512), torch.float32, operands.device, stream)
    _check(lib().mx_probe_mfma_fp4(_ptr(operands), iters, workgroups, _ptr(out), _stream(stream)))
    return out


def probe_read(src, mode: int, loads_per_wave: int, workgroups: int, out=None, stream=None):
    """mx_probe_read over all bytes of src; returns the per-wave XOR words (int32 [workgroups * 4])."""
    if out is None:
        out = _empty(workgroups * 4, torch.int32, src.device, stream)
    nbytes = src.numel() * src.element_size()
    _check(lib().mx_probe_read(mode, loads_per_wave, workgroups, _ptr(src), nbytes, _ptr(out), _stream(stream)))
    return out


def probe_copy(src, dst, stream=None):
    """mx_probe_copy: dst = src (same byte size)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst differ in size")
    _check(lib().mx_probe_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)))
    return dst


def fp8_block_linear_workspace_size(M, K) -> int:
    return int(lib().mx_fp8_block_linear_workspace_size(M, K))


def fp8_block_linear(x, w, w_s, out=None, workspace=None, stream=None):
    """mx_fp8_block_linear: bf16 x [M, K], E4M3 w [N, K], E8M0 w_s [N/128, K/128] -> bf16 y [M, N]."""
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.device, stream)
    ws = _workspace(fp8_block_linear_workspace_size(M, K), x.device, workspace, stream)
    _check(lib().mx_fp8_block_linear(_ptr(x), M, K, _ptr(w), _ptr(w_s), N, _ptr(out), _ptr(ws), ws.numel(),
                                     _stream(stream)))
    return out


def nvfp4_linear_workspace_size(M, K) -> int:
    return int(lib().mx_nvfp4_linear_workspace_size(M, K))


def nvfp4_linear(x, w, w_s, w_global: float, x_global: float, out=None, workspace=None, stream=None):
    """mx_nvfp4_linear: bf16 x [M, K], NVFP4 w [N, K/2] + E4M3 w_s [N, K/16] + w_global -> bf16 y [M, N]."""
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = _empty((M, N), torch.bfloat16, x.device, stream)
    ws = _workspace(nvfp4_linear_workspace_size(M, K), x.device, workspace, stream)
    _check(lib().mx_nvfp4_linear(_ptr(x), M, K, _ptr(w), _ptr(w_s), float(w_global), N, float(x_global), _ptr(out),
                                 _ptr(ws), ws.numel(), _stream(stream)))
    return out


def nvfp4_expert_mlp_workspace_size(M, hidden, inter) -> int:
    return int(lib().mx_nvfp4_expert_mlp_workspace_size(M, hidden, inter))


def nvfp4_expert_mlp(x, w1, w1s, w1g, w3, w3s, w3g, w2, w2s, w2g, x_global, h_global, out=None, workspace=None,
                     stream=None):
    """mx_nvfp4_expert_mlp: one expert with NVFP4 weights on bf16 x [M, hidden] -> bf16 y [M, hidden]."""
    M, hidden = x.shape
    inter = w1.shape[0]
    if out is None:
        out = _empty((M, hidden), torch.bfloat16, x.device, stream)
    ws = _workspace(nvfp4_expert_mlp_workspace_size(M, hidden, inter), x.device, workspace, stream)
    _check(lib().mx_nvfp4_expert_mlp(_ptr(x), M, hidden, inter, _ptr(w1), _ptr(w1s), float(w1g), _ptr(w3),
                                     _ptr(w3s), float(w3g), _ptr(w2), _ptr(w2s), float(w2g), float(x_global),
                                     float(h_global), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def grouped_nvfp4_expert_mlp_workspace_size(T, hidden, inter, k, E) -> int:
    return int(lib().mx_grouped_nvfp4_expert_mlp_workspace_size(T, hidden, inter, k, E))


def grouped_nvfp4_expert_mlp(x, topk_ids, topk_w, w1, w1s, w1g, w3, w3s, w3g, w2, w2s, w2g, x_global, h_global,
                             out=None, workspace=None, stream=None):
    """mx_grouped_nvfp4_expert_mlp: routed experts with NVFP4 weights; w*g are device fp32 [E] tensors."""
    T, hidden = x.shape
    k = topk_ids.shape[1]
    E, inter = w1.shape[0], w1.shape[1]
    if out is None:
        out = _empty((T, hidden), torch.bfloat16, x.device, stream)
    ws = _workspace(grouped_nvfp4_expert_mlp_workspace_size(T, hidden, inter, k, E), x.device, workspace, stream)
    _check(lib().mx_grouped_nvfp4_expert_mlp(_ptr(x), T, hidden, inter, _ptr(topk_ids), _ptr(topk_w), k, E,
                                             _ptr(w1), _ptr(w1s), _ptr(w1g), _ptr(w3), _ptr(w3s), _ptr(w3g),
                                             _ptr(w2), _ptr(w2s), _ptr(w2g), float(x_global), float(h_global),
                                             _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def fp8_expert_mlp_workspace_size(M, hidden, inter) -> int:
    return int(lib().mx_fp8_expert_mlp_workspace_size(M, hidden, inter))


def fp8_expert_mlp(x, w1, w1s, w3, w3s, w2, w2s, out=None, workspace=None, stream=None):
    """mx_fp8_expert_mlp: the FP8 shared expert on bf16 x [M, hidden] -> bf16 y [M, hidden]."""
    M, hidden = x.shape
    inter = w1.shape[0]
    if out is None:
        out = _empty((M, hidden), torch.bfloat16, x.device, stream)
    ws = _workspace(fp8_expert_mlp_workspace_size(M, hidden, inter), x.device, workspace, stream)
    _check(lib().mx_fp8_expert_mlp(_ptr(x), M, hidden, inter, _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s), _ptr(w2),
                                   _ptr(w2s), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# The operators around the experts. Their tensors are checked here against each
# other (type, shape, device), since the library sees pointers only; a call runs
# on the tensors' device, on its current stream unless one is given. Autograd
# records none of them: the gradients are calls of their own (for a
# torch.autograd.Function, whose passes run without recording), and a call that
# autograd would have to record raises.

def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _unrecorded(t, name):
    """Raises where a result would silently miss t's gradient, or t, if written, its history."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and autograd does not record this call: call it under "
                         "torch.no_grad() or in a torch.autograd.Function")


def _wrote(given):
    """Tells autograd that the caller's tensors among these were written, as an operation of torch's in place does: an
    operation that has saved one for its backward pass then raises there instead of reading the new values."""
    for t in given:
        if t is not None:
            torch._C._increment_version((t,))     # torch.autograd.graph.increment_version, twice as fast


def _tensor(t, name, dtype, shape, device):
    """t as a device pointer, once its type, shape, device and layout are as said."""
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != device.index or t.requires_grad
            or not t.is_contiguous()):
        _unrecorded(t, name)
        if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}: got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}"
                             f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _dtype(t, name):
    if not t.is_cuda:
        raise ValueError("libmxfp4 takes device tensors")
    dt = MX_DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} is {t.dtype}: bf16, fp16 or fp32 is taken")
    return dt


def _run(fn, device, stream, *args):
    """fn(*args, stream) on `device`."""
    if stream is None:
        # torch.cuda.current_stream(device).cuda_stream and current_device() without what they
        # build and check on the way, which costs as much as the library call
        s = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != 0:
        _check(status)


def _out(out, name, like, stream):
    """(`out` or a new tensor, its pointer): of the type, shape and device of the contiguous `like`."""
    if out is not None:
        return out, _tensor(out, name, like.dtype, like.shape, like.device)
    out = torch.empty_like(like) if stream is None else _made(stream, torch.empty_like, like)
    return out, out.data_ptr()


def _new(out, name, shape, dtype, device, stream):
    """_out for a tensor that is like no other, of one or two dimensions."""
    if out is not None:
        return out, _tensor(out, name, dtype, shape, device)
    # torch.empty, which takes a third longer
    strides = (1,) if len(shape) == 1 else (shape[1], 1)
    if stream is None:
        out = torch.empty_strided(shape, strides, dtype=dtype, device=device)
    else:
        out = _made(stream, torch.empty_strided, shape, strides, dtype=dtype, device=device)
    return out, out.data_ptr()


def _scratch(workspace, nbytes, device, stream):
    """(tensor to keep until the call has been made, pointer, bytes). Memory of the call's own is the call's stream's:
    let go of afterwards, it comes back for later work of that stream only."""
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, None, 0
    if stream is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        with torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), nbytes


# The size calls depend on their arguments alone, and a call through ctypes takes half a microsecond.
@functools.lru_cache(4096)
def moe_sort_workspace_size(T, k, E) -> int:
    return int(lib().mx_moe_sort_workspace_size(T, k, E))


def moe_sort(topk_ids, E: int, expert_off=None, row_slot=None, slot_row=None, workspace=None, stream=None):
    """mx_moe_sort: int32 topk_ids [T, k] -> (expert_off [E+1], row_slot [T*k], slot_row [T, k]), all int32."""
    given = (expert_off, row_slot, slot_row)
    T, k = topk_ids.shape
    dev, i32 = topk_ids.device, torch.int32
    _need(topk_ids.is_cuda, "libmxfp4 takes device tensors")
    if not 1 <= E <= 512:
        raise ValueError(f"E {E} not in [1, 512]")
    ids = _tensor(topk_ids, "topk_ids", i32, (T, k), dev)
    expert_off, op = _new(expert_off, "expert_off", (E + 1,), i32, dev, stream)
    row_slot, rp = _new(row_slot, "row_slot", (T * k,), i32, dev, stream)
    slot_row, sp = _out(slot_row, "slot_row", topk_ids, stream)
    ws, wp, wn = _scratch(workspace, moe_sort_workspace_size(T, k, E), dev, stream)
    _run(lib().mx_moe_sort, dev, stream, ids, T, k, E, op, rp, sp, wp, wn)
    _wrote(given)
    return expert_off, row_slot, slot_row


def moe_permute(x, slot_row, out=None, stream=None):
    """mx_moe_permute: x [T, H] to its rows of out [rows, H] (default: a new [T*k, H], whose other rows are
    whatever they are)."""
    given = (out,)
    T, H = x.shape
    k = slot_row.shape[1]
    dev = x.device
    dt = _dtype(x, "x")
    out, op = _new(out, "out", (T * k if out is None else out.shape[0], H), x.dtype, dev, stream)
    _run(lib().mx_moe_permute, dev, stream, dt, _tensor(x, "x", x.dtype, (T, H), dev), T, H,
         _tensor(slot_row, "slot_row", torch.int32, (T, k), dev), k, out.shape[0], op)
    _wrote(given)
    return out


def moe_unpermute(ys, slot_row, topk_w=None, out=None, stream=None):
    """mx_moe_unpermute: ys [rows, H] -> y [T, H], weighted by fp32 topk_w [T, k] (None: 1)."""
    given = (out,)
    rows, H = ys.shape
    T, k = slot_row.shape
    dev = ys.device
    dt = _dtype(ys, "ys")
    out, op = _new(out, "out", (T, H), ys.dtype, dev, stream)
    _run(lib().mx_moe_unpermute, dev, stream, dt, _tensor(ys, "ys", ys.dtype, (rows, H), dev), rows, H,
         _tensor(slot_row, "slot_row", torch.int32, (T, k), dev),
         None if topk_w is None else _tensor(topk_w, "topk_w", torch.float32, (T, k), dev), T, k, op)
    _wrote(given)
    return out


def moe_unpermute_grad(d_y, ys, slot_row, topk_w, d_ys=None, d_w=None, stream=None):
    """mx_moe_unpermute_grad -> (d_ys [rows, H], d_w [T, k] fp32). Without d_ys, rows that no slot names come
    back as zeros; a given d_ys keeps them."""
    given = (d_ys, d_w)
    rows, H = ys.shape
    T, k = slot_row.shape
    dev = ys.device
    dt = _dtype(ys, "ys")
    yp = _tensor(ys, "ys", ys.dtype, (rows, H), dev)
    if d_ys is None:
        d_ys = torch.zeros_like(ys) if stream is None else _made(stream, torch.zeros_like, ys)
    wp = _tensor(topk_w, "topk_w", torch.float32, (T, k), dev)
    d_w, dwp = _out(d_w, "d_w", topk_w, stream)
    _run(lib().mx_moe_unpermute_grad, dev, stream, dt, _tensor(d_y, "d_y", ys.dtype, (T, H), dev), yp, rows, H,
         _tensor(slot_row, "slot_row", torch.int32, (T, k), dev), wp, T, k,
         _tensor(d_ys, "d_ys", ys.dtype, (rows, H), dev), dwp)
    _wrote(given)
    return d_ys, d_w


def _gate(gate, T, H):
    """(mx_gate, shape of the gate) from the gate's shape: None, [H], [T, 1] or [T, H]."""
    if gate is None:
        return MX_GATE["none"], None
    if gate.shape == (H,):
        return MX_GATE["channel"], (H,)
    if gate.shape == (T, H) and H > 1:
        return MX_GATE["full"], (T, H)
    if gate.shape == (T, 1):
        return MX_GATE["token"], (T, 1)
    raise ValueError(f"gate of shape {tuple(gate.shape)}: [H], [T, 1] or [T, H] is taken, T {T}, H {H}")


def block_norm(residual, w_pre=None, y=None, w_post=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6,
               residual_out=None, normed=None, stream=None):
    """mx_block_norm -> (normed [T, H] or None without w_pre, residual_out [T, H] or, without y, the residual).
    gate: None, [H] (per channel), [T, 1] (per token) or [T, H]."""
    given = (residual_out, normed)
    T, H = residual.shape
    dev = residual.device
    rdt = _dtype(residual, "residual")
    _need(y is not None or w_pre is not None, "y and w_pre are both None: nothing to do")
    like = y if y is not None else w_pre
    dt, adt = _dtype(like, "y or w_pre"), like.dtype
    kind, gshape = _gate(gate, T, H)
    res = _tensor(residual, "residual", residual.dtype, (T, H), dev)
    yp = ro = no = None
    if y is not None:
        yp = _tensor(y, "y", adt, (T, H), dev)
        residual_out, ro = _out(residual_out, "residual_out", residual, stream)
    else:
        _need(w_post is None and gate is None and residual_out is None, "w_post, gate and residual_out need y")
    if w_pre is not None:
        normed, no = _out(normed, "normed", y, stream) if y is not None else \
            _new(normed, "normed", (T, H), adt, dev, stream)
    else:
        _need(normed is None, "normed needs w_pre")
    _run(lib().mx_block_norm, dev, stream, dt, rdt, yp, res,
         None if w_post is None else _tensor(w_post, "w_post", adt, (H,), dev), kind,
         None if gate is None else _tensor(gate, "gate", adt, gshape, dev), res_scale,
         None if w_pre is None else _tensor(w_pre, "w_pre", adt, (H,), dev), eps, T, H, ro, no)
    _wrote(given)
    return normed, (residual if y is None else residual_out)


@functools.lru_cache(4096)
def block_norm_grad_workspace_size(T, H) -> int:
    return int(lib().mx_block_norm_grad_workspace_size(T, H))


def block_norm_grad(residual_out, w_pre=None, d_normed=None, d_residual_out=None, y=None, w_post=None, gate=None,
                    res_scale: float = 1.0, eps: float = 1e-6, d_residual=None, d_y=None, workspace=None, stream=None):
    """mx_block_norm_grad at the stored residual_out (without y: the residual) -> (d_residual, dw_pre, d_y, dw_post,
    d_gate); None for what there is none of. dw_pre, dw_post and the d_gate of a [H] or [T, 1] gate are fp32."""
    given = (d_residual, d_y)
    T, H = residual_out.shape
    dev, f32 = residual_out.device, torch.float32
    rdt = _dtype(residual_out, "residual_out")
    _need(y is not None or w_pre is not None, "y and w_pre are both None: nothing to do")
    _need((w_pre is None) == (d_normed is None), "w_pre and d_normed go together")
    _need(w_pre is not None or d_residual_out is not None, "d_residual_out is needed without w_pre")
    _need(y is not None or (w_post is None and gate is None and d_y is None), "w_post, gate and d_y need y")
    like = y if y is not None else w_pre
    dt, adt = _dtype(like, "y or w_pre"), like.dtype
    kind, gshape = _gate(gate, T, H)

    def act(t, name, shape):
        return None if t is None else _tensor(t, name, adt, shape, dev)
    yp, rp = act(y, "y", (T, H)), _tensor(residual_out, "residual_out", residual_out.dtype, (T, H), dev)
    none = (None, None)
    dw_pre, wpre_p = none if w_pre is None else _new(None, "dw_pre", (H,), f32, dev, stream)
    dw_post, wpost_p = none if w_post is None else _new(None, "dw_post", (H,), f32, dev, stream)
    d_gate, gate_p = none if gate is None else _new(None, "d_gate", gshape, adt if kind == MX_GATE["full"] else f32, dev, stream)
    d_residual, dr_p = _out(d_residual, "d_residual", residual_out, stream)
    d_y, dy_p = none if y is None else _out(d_y, "d_y", y, stream)
    ws, wp, wn = _scratch(workspace, block_norm_grad_workspace_size(T, H), dev, stream)
    _run(lib().mx_block_norm_grad, dev, stream, dt, rdt, yp, rp, act(w_post, "w_post", (H,)), kind,
         act(gate, "gate", gshape), res_scale, act(w_pre, "w_pre", (H,)), eps, T, H, act(d_normed, "d_normed", (T, H)),
         None if d_residual_out is None else _tensor(d_residual_out, "d_residual_out", residual_out.dtype, (T, H), dev),
         dr_p, dy_p, gate_p, wpost_p, wpre_p, wp, wn)
    _wrote(given)
    return d_residual, dw_pre, d_y, dw_post, d_gate


@functools.lru_cache(4096)
def lora_add_workspace_size(M, K, R, n) -> int:
    return int(lib().mx_lora_add_workspace_size(M, K, R, n))


def _rows(t, name, dtype, rows, device):
    """(pointer, width, row stride) of a matrix whose rows are contiguous."""
    if t.requires_grad:
        _unrecorded(t, name)
    if t.dtype != dtype or t.dim() != 2 or t.shape[0] != rows or t.device != device or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a {dtype} matrix of {rows} rows with contiguous columns on {device}: got "
                         f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")
    return t.data_ptr(), t.shape[1], t.stride(0) if rows > 1 else (t.shape[1] + 7) // 8 * 8


def lora_add(y, x, a, b, adapter_off, row_token, scale=None, workspace=None, stream=None):
    """mx_lora_add: y [M, N] += scale[a] * (x [M, K] . a[a]^T) . b[a]^T in place, a [n, R, K], b [n, N, R], for the
    tokens sorted by adapter (expert_off and row_slot of moe_sort over adapter ids [M, 1]). x and y may be column
    ranges of wider matrices. Returns y."""
    M = x.shape[0]
    dev = x.device
    dt = _dtype(x, "x")
    n, R, K = a.shape
    xp, kx, ldx = _rows(x, "x", x.dtype, M, dev)
    yp, N, ldy = _rows(y, "y", x.dtype, M, dev)
    if kx != K:
        raise ValueError(f"x has {kx} columns, a takes {K}")
    ws, wp, wn = _scratch(workspace, lora_add_workspace_size(M, K, R, n), dev, stream)
    _run(lib().mx_lora_add, dev, stream, dt, xp, ldx, M, K, _tensor(a, "a", x.dtype, (n, R, K), dev),
         _tensor(b, "b", x.dtype, (n, N, R), dev),
         None if scale is None else _tensor(scale, "scale", torch.float32, (n,), dev), n, R,
         _tensor(adapter_off, "adapter_off", torch.int32, (n + 1,), dev),
         _tensor(row_token, "row_token", torch.int32, (M,), dev), yp, ldy, N, wp, wn)
    _wrote((y,))
    return y


class MoeRunner:
    """mx_moe_runner: the routed experts over fixed device buffers, captured once
    into a hipGraph. Refresh x, topk_ids, topk_w (and the NVFP4 global tensor) in
    place, then replay()."""

    def __init__(self, x, topk_ids, topk_w, w1, w1s, w3, w3s, w2, w2s, requant="mxfp4",
                 requant_global=None, out=None, packed_scales=None, packed_codes=None):
        T, hidden = x.shape
        k = topk_ids.shape[1]
        E, inter = w1.shape[0], w1.shape[1]
        self.out = out if out is not None else torch.empty((T, hidden), dtype=torch.bfloat16, device=x.device)
        g = _global(requant_global, x.device)
        # keep the bound tensors alive as long as the runner
        self._bound = (x, topk_ids, topk_w, w1, w1s, w3, w3s, w2, w2s, packed_scales, packed_codes, self.out, g)
        h = _P()
        _check(lib().mx_moe_runner_create(_ptr(x), T, hidden, inter, _ptr(topk_ids), _ptr(topk_w), k, E,
                                          _ptr(w1), _ptr(w1s), _ptr(w3), _ptr(w3s), _ptr(w2), _ptr(w2s),
                                          _ptr(packed_scales), _ptr(packed_codes), _fmt(requant), _ptr(g),
                                          _ptr(self.out), ctypes.byref(h)))
        self._h = h

    def replay(self, stream=None):
        _check(lib().mx_moe_runner_replay(self._h, _stream(stream)))
        return self.out

    def close(self):
        if self._h is not None and self._h.value is not None:
            _check(lib().mx_moe_runner_destroy(self._h))
        self._h = None

