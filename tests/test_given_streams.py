"""Calls on a stream that is not the current one: where the memory comes from that a call makes itself.

torch's allocator gives a freed block out again at once on the stream it was made on, although that stream's earlier
work may still be using it. So what a call on stream s makes (outputs, workspaces) has to be s's memory: a block of the
current stream's could still be read or written there. On the CPU the binding runs over stand-ins that note which
stream was current when memory was made; on the GPU calls meet a just-freed block with work pending in it."""

import numpy as np
import pytest
import torch

from binding_util import BF16, CURRENT, F32, I32, U8, Stream, Tensor, around, stand_in, t

AROUND = sorted(around(None))


@pytest.fixture
def fake(monkeypatch):
    return stand_in(monkeypatch)


def _check(f, call):
    s = Stream()
    out = call(stream=s)
    assert f.lib.streams == [s.cuda_stream]
    assert f.torch.made and all(m.made_on is s for m in f.torch.made)
    # what goes to the caller is known to the stream that the caller is on
    out = [o for o in (out if isinstance(out, tuple) else (out,)) if isinstance(o, Tensor) and o in f.torch.made]
    assert all(CURRENT in o.told for o in out)
    f.torch.made.clear()
    call()
    assert all(m.made_on is CURRENT for m in f.torch.made)


@pytest.mark.parametrize("name", AROUND)
def test_memory_of_a_call_is_the_given_streams(fake, name):
    _check(fake, around(fake.binding)[name])


@pytest.mark.parametrize("name", AROUND)
def test_a_stream_of_another_device_is_refused(fake, name):
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        around(fake.binding)[name](stream=Stream(torch.device("cuda", 1)))
    assert not fake.lib.streams


def quantised(mx):
    """The same of the calls on quantised operands."""
    x, c, w, ws = t(4, 64), t(4, 32, dtype=U8), t(64, 32, dtype=U8), t(64, 2, dtype=U8)
    ids, gw, e, es, eg = t(4, 2, dtype=I32), t(4, 2, dtype=F32), t(3, 64, 32, dtype=U8), t(3, 64, 2, dtype=U8), t(3, dtype=F32)
    one, all_ = (w, ws, w, ws, w, ws), (e, es, e, es, e, es)
    return {
        "dequant": lambda **k: mx.dequant("nvfp4", c, ws, 4, 64, 0.5, **k),
        "quantize_act": lambda **k: mx.quantize_act("nvfp4", x, 0.5, **k),
        "pack_weight_scales": lambda **k: mx.pack_weight_scales(ws, ws, ws, **k),
        "pack_weight_codes": lambda **k: mx.pack_weight_codes(w, w, w, **k),
        "expert_mlp": lambda **k: mx.expert_mlp(x, *one, requant="nvfp4", requant_global=0.5, **k),
        "expert_mlp_noalloc": lambda **k: mx.expert_mlp_noalloc(x, *one, requant="nvfp4", requant_global=0.5, **k),
        "grouped_expert_mlp": lambda **k: mx.grouped_expert_mlp(x, ids, gw, *all_, requant="nvfp4", requant_global=0.5, **k),
        "nvfp4_global_warmup": lambda **k: mx.nvfp4_global_warmup(x, w, ws, w, ws, **k),
        "debug_gemm_f32": lambda **k: mx.debug_gemm_f32(c, ws, c, ws, **k),
        "probe_mfma_fp4": lambda **k: mx.probe_mfma_fp4(t(512, 16, dtype=I32), 1, 1, **k),
        "probe_read": lambda **k: mx.probe_read(x, 0, 8, 1, **k),
        "fp8_block_linear": lambda **k: mx.fp8_block_linear(x, w, ws, **k),
        "nvfp4_linear": lambda **k: mx.nvfp4_linear(x, w, ws, 0.5, 0.5, **k),
        "nvfp4_expert_mlp": lambda **k: mx.nvfp4_expert_mlp(x, w, ws, 0.5, w, ws, 0.5, w, ws, 0.5, 0.5, 0.5, **k),
        "grouped_nvfp4_expert_mlp": lambda **k: mx.grouped_nvfp4_expert_mlp(x, ids, gw, e, es, eg, e, es, eg, e, es, eg,
                                                                            0.5, 0.5, **k),
        "fp8_expert_mlp": lambda **k: mx.fp8_expert_mlp(x, *one, **k),
    }


@pytest.mark.parametrize("name", sorted(quantised(None)))
def test_memory_of_a_quantised_call_is_the_given_streams(fake, name):
    _check(fake, quantised(fake.binding)[name])


# ------------------------------------------------------------------ on the GPU

def _pending(block):
    """Work on the current stream that ends by overwriting `block`: some tens of milliseconds of matrix products."""
    a = torch.ones((4096, 4096), device="cuda")
    for _ in range(24):
        a = a @ a * 2.0 ** -12
    block.fill_(0xFF)


@pytest.mark.gpu
def test_freed_blocks_of_the_current_stream_are_left_alone():
    """On the current stream a block of every size that the calls ask for is written late and let go of early; the same
    calls on another stream, with all outputs and workspaces their own, give what they give on an idle device."""
    import mxfp4_block_scaled_e2m1_amd as mx
    rng = np.random.default_rng(0)
    T, H, k, E, R, n = 2048, 1024, 4, 16, 16, 3
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(BF16).cuda()
    x, res, dn, w1, w2, gate = mk(T, H), mk(T, H), mk(T, H), mk(H), mk(H), mk(H)
    a, b = mk(n, R, H), mk(n, H, R)
    ids = torch.from_numpy(rng.integers(0, E, size=(T, k)).astype(np.int32)).cuda()
    aid = torch.from_numpy(rng.integers(0, n, size=(T, 1)).astype(np.int32)).cuda()
    gw = torch.rand((T, k), device="cuda")
    off, tok, _ = mx.moe_sort(aid, n)
    slot_row = mx.moe_sort(ids, E)[2]
    ys = mk(T * k, H)
    calls = {
        "sort": (lambda **s: mx.moe_sort(ids, E, **s), [4 * (E + 1), 4 * T * k, mx.moe_sort_workspace_size(T, k, E)]),
        "permute": (lambda **s: mx.moe_permute(x, slot_row, **s), [2 * T * k * H]),
        "unpermute": (lambda **s: mx.moe_unpermute(ys, slot_row, gw, **s), [2 * T * H]),
        "unpermute_grad": (lambda **s: mx.moe_unpermute_grad(dn, ys, slot_row, gw, **s), [2 * T * k * H, 4 * T * k]),
        "norm": (lambda **s: mx.block_norm(res, w1, y=x, w_post=w2, gate=gate, **s), [2 * T * H] * 2),
        "norm_grad": (lambda **s: mx.block_norm_grad(res, w1, dn, d_residual_out=res, y=x, w_post=w2, gate=gate, **s),
                      [2 * T * H, 2 * T * H, 4 * H, 4 * H, 4 * H, mx.block_norm_grad_workspace_size(T, H)]),
        "lora": (lambda **s: mx.lora_add(y, x, a, b, off, tok, **s), [mx.lora_add_workspace_size(T, H, R, n)]),
    }
    side = torch.cuda.Stream()
    for name, (call, sizes) in calls.items():
        print(name, flush=True)
        y = x.clone()
        want = call()
        want = [v.clone() for v in (want if isinstance(want, tuple) else (want,))]
        y = x.clone()
        torch.cuda.synchronize()
        blocks = [torch.empty(s, dtype=U8, device="cuda") for s in sizes]
        held = {v.data_ptr() for v in blocks}
        for v in blocks:
            _pending(v)
        del blocks, v
        got = call(stream=side)
        got = got if isinstance(got, tuple) else (got,)
        assert not held & {v.data_ptr() for v in got}, name
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name


@pytest.mark.gpu
def test_freed_blocks_are_left_alone_by_quantised_calls():
    """The same of quantisation, one expert and routed experts."""
    import mxfp4_block_scaled_e2m1_amd as mx
    import workloads as W
    T, H, I, E, k = 512, 512, 256, 4, 2
    d = W.grouped(tokens=T, n_experts=E, k=k, seed=1, hidden=H, inter=I)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    w = [dev(d[n]) for n in ("w1", "w1s", "w3", "w3s", "w2", "w2s")]
    x = dev(d["x"].view(np.int16)).view(BF16)
    ids, gw = dev(d["ids"]), dev(d["w"])
    calls = {
        "quantize": (lambda **s: mx.quantize_act("mxfp4", x, **s), [T * H // 2, T * H // 32]),
        "expert": (lambda **s: mx.expert_mlp(x, *(v[0] for v in w), **s), [2 * T * H, mx.expert_mlp_workspace_size(T, H, I)]),
        "routed": (lambda **s: mx.grouped_expert_mlp(x, ids, gw, *w, **s),
                   [2 * T * H, mx.grouped_expert_mlp_workspace_size(T, H, I, k, E)]),
    }
    side = torch.cuda.Stream()
    for name, (call, sizes) in calls.items():
        print(name, flush=True)
        want = call()
        want = [v.clone() for v in (want if isinstance(want, tuple) else (want,))]
        torch.cuda.synchronize()
        blocks = [torch.empty(s, dtype=U8, device="cuda") for s in sizes]
        held = {v.data_ptr() for v in blocks}
        for v in blocks:
            _pending(v)
        del blocks, v
        got = call(stream=side)
        got = got if isinstance(got, tuple) else (got,)
        assert not held & {v.data_ptr() for v in got}, name
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name


@pytest.mark.gpu
def test_given_streams_under_capture():
    """Captured on the capturing stream, given by name, and on one that forks from it and joins it again, with outputs
    and workspaces of the calls' own: replays give what eager calls give, also after other work on both streams."""
    import mxfp4_block_scaled_e2m1_amd as mx
    rng = np.random.default_rng(1)
    T, H, k, E, R, n = 1500, 512, 3, 8, 24, 4
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(BF16).cuda()
    x, w, y0, a, b = mk(T, H), mk(H), mk(T, H), mk(n, R, H), mk(n, H, R)
    ids = torch.from_numpy(rng.integers(-1, E, size=(T, k)).astype(np.int32)).cuda()
    aid = torch.from_numpy(rng.integers(-1, n, size=(T, 1)).astype(np.int32)).cuda()
    gw = torch.rand((T, k), device="cuda")

    def step(s):
        norm, r = mx.block_norm(x, w, y=y0, w_post=w, stream=s)
        slot_row = mx.moe_sort(ids, E, stream=s)[2]
        xs = mx.moe_permute(norm, slot_row, stream=s)
        back = mx.moe_unpermute(xs, slot_row, gw, stream=s)
        off, tok, _ = mx.moe_sort(aid, n, stream=s)
        mx.lora_add(back, x, a, b, off, tok, stream=s)
        grads = mx.block_norm_grad(r, w, back, y=y0, w_post=w, stream=s)
        return (back, r) + grads[:4]

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    want = [v.clone() for v in step(None)]
    torch.cuda.synchronize()
    for fork in (False, True):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            if fork:
                side.wait_stream(main)
                got = step(side)
                main.wait_stream(side)
            else:
                got = step(main)
        for _ in range(3):
            for v in got:
                v.zero_()
            junk = step(main), step(side), step(None)
            torch.cuda.synchronize()
            del junk
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), fork
        del got, g
