"""The operators around the experts and torch's autograd, which records none of them: a call that it would have to
record is refused, a tensor written in place is known to have changed, and in a torch.autograd.Function the operators
and their gradient calls give a model's gradients."""

import numpy as np
import pytest
import torch

from around_util import U, depth, pair, routing, within
from binding_util import BF16, F32, I32, Tensor, around, stand_in, t


@pytest.fixture
def fake(monkeypatch):
    return stand_in(monkeypatch)


def _calls(mx):
    """name -> (call, its float arguments by name): one may need a gradient."""
    T, H = 4, 64
    n = lambda *names, **over: {k: over.get(k) or t(T, H) for k in names}
    ids, off, tok = t(T, 2, dtype=I32), t(3, dtype=I32), t(T, dtype=I32)
    return {
        "permute": (lambda a: mx.moe_permute(a["x"], ids, out=a["out"]), n("x", "out", out=t(8, H))),
        "unpermute": (lambda a: mx.moe_unpermute(a["ys"], ids, a["w"], out=a["out"]),
                      n("ys", "w", "out", ys=t(8, H), w=t(T, 2, dtype=F32))),
        "unpermute_grad": (lambda a: mx.moe_unpermute_grad(a["dy"], a["ys"], ids, a["w"], d_ys=a["dys"], d_w=a["dw"]),
                           n("dy", "ys", "w", "dys", "dw", ys=t(8, H), w=t(T, 2, dtype=F32), dys=t(8, H),
                             dw=t(T, 2, dtype=F32))),
        "norm": (lambda a: mx.block_norm(a["r"], a["w"], y=a["y"], w_post=a["p"], gate=a["g"], residual_out=a["ro"],
                                         normed=a["o"]), n("r", "w", "y", "p", "g", "ro", "o", w=t(H), p=t(H))),
        "norm_grad": (lambda a: mx.block_norm_grad(a["r"], a["w"], a["dn"], d_residual_out=a["dro"], y=a["y"], w_post=a["p"],
                                                   gate=a["g"], d_residual=a["dr"], d_y=a["dy"]),
                      n("r", "w", "dn", "dro", "y", "p", "g", "dr", "dy", w=t(H), p=t(H))),
        "lora": (lambda a: mx.lora_add(a["y"], a["x"], a["a"], a["b"], off, tok, a["s"]),
                 n("y", "x", "a", "b", "s", y=t(T, 32), a=t(2, 8, H), b=t(2, 32, 8), s=t(2, dtype=F32))),
    }


CASES = [(name, arg) for name, (_, args) in _calls(None).items() for arg in args]


@pytest.mark.parametrize("name,arg", CASES)
def test_an_input_that_requires_a_gradient_is_refused(fake, name, arg):
    call, args = _calls(fake.binding)[name]
    args[arg].requires_grad = True
    with pytest.raises(ValueError, match="requires a gradient"):
        call(args)
    assert not fake.lib.streams and not fake.torch.written
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            call(args)
    assert len(fake.lib.streams) == 2


WRITTEN = {"permute": {"out"}, "unpermute": {"out"}, "unpermute_grad": {"dys", "dw"}, "norm": {"ro", "o"},
           "norm_grad": {"dr", "dy"}, "lora": {"y"}}


@pytest.mark.parametrize("name", sorted(WRITTEN))
def test_what_a_call_writes_is_made_known(fake, name):
    call, args = _calls(fake.binding)[name]
    call(args)
    assert {id(v) for v in fake.torch.written} == {id(args[k]) for k in WRITTEN[name]}
    maps = [Tensor((5,), I32), Tensor((8,), I32), Tensor((4, 2), I32)]
    fake.torch.written.clear()
    fake.binding.moe_sort(t(4, 2, dtype=I32), 4, *maps)
    assert fake.torch.written == maps


def test_memory_of_a_call_needs_no_mark(fake):
    for name, call in around(fake.binding).items():
        call()
        assert len(fake.torch.written) == (name == "lora_add")
        fake.torch.written.clear()


# ------------------------------------------------------------------ on the GPU

@pytest.mark.gpu
def test_a_saved_tensor_that_was_written_is_noticed():
    """exp saves its output for the backward pass: adapters on top of it, or any output buffer over it, would change it."""
    import mxfp4_block_scaled_e2m1_amd as mx
    off, tok, _ = mx.moe_sort(torch.zeros((8, 1), dtype=I32, device="cuda"), 1)
    a, b = torch.ones((1, 8, 64), dtype=BF16, device="cuda"), torch.ones((1, 64, 8), dtype=BF16, device="cuda")
    other, w = torch.ones((8, 64), dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    for write in (lambda y: mx.lora_add(y, other, a, b, off, tok), lambda y: mx.moe_permute(other, tok.view(8, 1), out=y),
                  lambda y: mx.block_norm(other, w, normed=y)):
        leaf = torch.zeros((8, 64), dtype=BF16, device="cuda", requires_grad=True)
        y = leaf.exp()
        with pytest.raises(ValueError, match="requires a gradient"):
            write(y)
        assert (y == 1).all()
        with torch.no_grad():
            write(y)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():                       # serving: such tensors have no version
        y = torch.zeros((8, 64), dtype=BF16, device="cuda")
        assert (mx.lora_add(y, other, a, b, off, tok) == 512).all()


@pytest.mark.gpu
def test_gradients_of_a_block_through_autograd():
    """Norm, rows to a weight per expert and back, in autograd Functions over the operators, in fp32, against torch's
    own differentiation in float64."""
    import mxfp4_block_scaled_e2m1_amd as mx
    eps = 1e-5

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, r, w):
            ctx.save_for_backward(r, w)
            return mx.block_norm(r, w, eps=eps)[0]

        @staticmethod
        def backward(ctx, d):
            return mx.block_norm_grad(*ctx.saved_tensors, d, eps=eps)[:2]

    class Back(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ys, w, slot_row):
            ctx.save_for_backward(ys, w, slot_row)
            return mx.moe_unpermute(ys, slot_row, w)

        @staticmethod
        def backward(ctx, d):
            ys, w, slot_row = ctx.saved_tensors
            return *mx.moe_unpermute_grad(d, ys, slot_row, w), None

    class There(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, slot_row):
            ctx.save_for_backward(slot_row)
            return mx.moe_permute(x, slot_row)

        @staticmethod
        def backward(ctx, d):
            return mx.moe_unpermute(d, *ctx.saved_tensors), None

    rng = np.random.default_rng(0)
    T, k, E, H = 40, 3, 6, 96
    ids = routing(rng, T, k, E)
    res, w, gw, m, g = (pair(rng.standard_normal(s), "fp32") for s in ((T, H), (H,), (T, k), (E, H), (T, H)))
    off, _, slot_row = mx.moe_sort(torch.from_numpy(ids).cuda(), E)
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), (off[1:] - off[:-1]).long())
    leaves = [v[0].requires_grad_() for v in (res, w, gw, m)]
    r, wt, gt, mt = leaves
    y = Back.apply(There.apply(Norm.apply(r, wt), slot_row) * mt[expert], gt, slot_row)
    y.backward(g[0])
    ref = [torch.tensor(v[1], requires_grad=True) for v in (res, w, gw, m)]
    r, wt, gt, mt = ref
    n = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * wt
    yr = (n[:, None, :] * mt[torch.from_numpy(ids).long()] * gt[:, :, None]).sum(1)
    yr.backward(torch.tensor(g[1]))
    # products of at most five fp32 numbers of size below 5, sums over a row, k slots and, for w and m, the tokens:
    # every term off by at most depth(H) steps of itself and the sums by T k of theirs, of terms below 5^5 that
    # average out to a tenth of that
    tol = 5 ** 5 / 10 * (depth(H) + T * k) * U
    for a, b in zip([y.detach()] + [v.grad for v in leaves], [yr.detach()] + [v.grad for v in ref]):
        within(a, b.numpy(), tol * np.maximum(1.0, np.abs(b.numpy())))
