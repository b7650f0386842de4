"""Inputs and tolerances of the tests of the operators around the experts.

A device tensor and its float64 values on the host go together. Tolerances are
worst-case bounds of the arithmetic the operators document: fp32 sums in any
order of the stated depth, then one rounding to the output's type, which is off
by at most half a step (eps / 2 of the value, or half the smallest subnormal).
"""

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24                                   # half a step of fp32
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half the smallest subnormal


def half_step(name):
    return torch.finfo(DTYPES[name]).eps / 2


def pair(values, name, device="cuda"):
    """(device tensor of the type, its exact values as float64 numpy)."""
    t = torch.as_tensor(np.ascontiguousarray(values)).to(DTYPES[name])
    return t.to(device), t.to(torch.float64).numpy()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def depth(H):
    """Longest chain of additions an element of a row sum goes through: at worst one wave's 64 lanes
    share the row, then six steps over the lanes and sixteen over the waves."""
    return H / 64 + 32


def within(got, ref, tol, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - ref).max():.3g}, {over.max():.3g} over the bound"


def rounded(ref, name):
    """Bound of one rounding of ref to the type."""
    return half_step(name) * np.abs(ref) + TINY[name]


def routing(rng, T, k, E, total=None, repeat=False):
    """ids [T, k] int32: distinct experts of 0 .. total - 1 (repeat: any), of which E are local."""
    total = total or E
    if repeat:
        return rng.integers(0, total, size=(T, k)).astype(np.int32)
    return np.stack([rng.permutation(total)[:k] for _ in range(T)]).astype(np.int32).reshape(T, k)
