"""Stand-ins for the binding's CPU tests: device tensors without a device, memory that notes the stream it was made
on, and a library whose calls all succeed."""

import contextlib
import ctypes
import types

import numpy as np
import torch

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
DEVICE = torch.device("cuda", 0)


class Tensor:
    """A contiguous device tensor as the binding sees it."""
    is_cuda, requires_grad, device = True, False, DEVICE

    def __init__(self, shape, dtype=BF16, made_on=None):
        self.shape, self.dtype, self.made_on = torch.Size(shape), dtype, made_on
        self.told = []

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = [int(np.prod(self.shape[j + 1:], dtype=np.int64)) for j in range(len(self.shape))]
        return tuple(s) if i is None else s[i]

    def numel(self):
        return int(np.prod(self.shape, dtype=np.int64))

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return id(self)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def record_stream(self, s):
        self.told.append(s)


class Stream:
    cuda_stream = 77

    def __init__(self, device=DEVICE):
        self.device = device


CURRENT = Stream()


class Torch:
    """torch, but memory comes from a note of the current stream."""
    Tensor = Tensor

    def __init__(self):
        self.now, self.made = CURRENT, []
        self.cuda = types.SimpleNamespace(stream=self._stream, current_stream=lambda device=None: self.now,
                                          device=contextlib.nullcontext)
        self.written = []
        self._C = types.SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda i: 0,
                                        _increment_version=self.written.extend)

    def __getattr__(self, name):
        return getattr(torch, name)

    @contextlib.contextmanager
    def _stream(self, s):
        before, self.now = self.now, s or self.now
        yield
        self.now = before

    def _make(self, shape, dtype):
        self.made.append(Tensor((shape,) if isinstance(shape, int) else shape, dtype, self.now))
        return self.made[-1]

    def empty(self, shape, dtype, device):
        return self._make(shape, dtype)

    def empty_strided(self, shape, strides, dtype, device):
        return self._make(shape, dtype)

    def empty_like(self, t):
        return self._make(t.shape, t.dtype)

    zeros_like = empty_like

    def tensor(self, values, dtype, device):
        return self._make((len(values),), dtype)


class Library:
    """Every call succeeds and asks for a workspace."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 512

        def call(*a):
            self.streams.append(a[-1].value if isinstance(a[-1], ctypes.c_void_p) else a[-1])
            return 0
        return call


def t(*shape, dtype=BF16):
    return Tensor(shape, dtype)


def around(mx):
    """name -> a call of each operator around the experts that makes all it can itself."""
    x, w, ids, gw, off, tok = t(4, 64), t(64), t(4, 2, dtype=I32), t(4, 2, dtype=F32), t(3, dtype=I32), t(4, dtype=I32)
    ys, a, b = t(8, 64), t(2, 8, 64), t(2, 32, 8)
    return {
        "moe_sort": lambda **k: mx.moe_sort(ids, 4, **k),
        "moe_permute": lambda **k: mx.moe_permute(x, ids, **k),
        "moe_unpermute": lambda **k: mx.moe_unpermute(ys, ids, gw, **k),
        "moe_unpermute_grad": lambda **k: mx.moe_unpermute_grad(x, ys, ids, gw, **k),
        "block_norm": lambda **k: mx.block_norm(x, w, y=x, w_post=w, gate=w, **k),
        "block_norm, no block": lambda **k: mx.block_norm(x, w, **k),
        "block_norm_grad": lambda **k: mx.block_norm_grad(x, w, x, d_residual_out=x, y=x, w_post=w, gate=w, **k),
        "lora_add": lambda **k: mx.lora_add(t(4, 32), x, a, b, off, tok, **k),
    }


def stand_in(monkeypatch):
    """The binding over the stand-ins."""
    from mxfp4_block_scaled_e2m1_amd import binding
    f = types.SimpleNamespace(torch=Torch(), lib=Library(), binding=binding)
    monkeypatch.setattr(binding, "torch", f.torch)
    monkeypatch.setattr(binding, "lib", lambda: f.lib)
    for name in ("moe_sort", "block_norm_grad", "lora_add"):       # sizes of this library only
        size = name + "_workspace_size"
        monkeypatch.setattr(binding, size, getattr(binding, size).__wrapped__)
    return f
