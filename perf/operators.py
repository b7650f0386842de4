"""The operators that stand around the quantised experts, as cases that can be timed and compared:

- sorting routed tokens by expert and moving their rows there (`moe_sort`, `moe_permute`),
- bringing the experts' rows back, weighted and summed, and the gradient of that (`moe_unpermute`,
  `moe_unpermute_grad`; without weights it is also the gradient of `moe_permute`),
- the norms before and after a block with its gate and residual scale, forward and backward
  (`block_norm`, `block_norm_grad`),
- the low-rank adapters of many requests on top of a shared projection (`lora_add`).

`run` computes them in plain torch operations, or, with `own`, through this repository's package.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's tail: 8 tokens, top-8 over the rank's 48 experts
        {"name": "sort_decode", "op": "sort", "tokens": 8, "k": 8, "experts": 48, "ranks": 1, "skew": 0.0,
         "hidden": 7168, "dtype": "bf16"},
        # the routed batch: 4096 tokens, every pair local
        {"name": "sort_batch", "op": "sort", "tokens": 4096, "k": 8, "experts": 48, "ranks": 1, "skew": 0.0,
         "hidden": 7168, "dtype": "bf16"},
        # one of 8 expert-parallel ranks: 48 of 384 experts, popular and unpopular ones, most pairs on other ranks
        {"name": "sort_share", "op": "sort", "tokens": 5003, "k": 8, "experts": 48, "ranks": 8, "skew": 1.2,
         "hidden": 7168, "dtype": "fp16"},
        # the weighted combine of the routed batch
        {"name": "back_batch", "op": "back", "tokens": 4096, "k": 8, "experts": 48, "ranks": 1, "skew": 0.0,
         "hidden": 7168, "dtype": "bf16", "weighted": True},
        # its backward pass when experts or the router are fine-tuned
        {"name": "back_grad_batch", "op": "back_grad", "tokens": 4096, "k": 8, "experts": 48, "ranks": 1,
         "skew": 1.2, "hidden": 7168, "dtype": "bf16"},
        # between two blocks of a decode step
        {"name": "norm_decode", "op": "norm", "tokens": 8, "hidden": 7168, "dtype": "bf16", "res_dtype": "bf16",
         "post": True, "gate": "none"},
        # between two blocks of a prompt, the residual stream kept in 32 bits, a gate per channel
        {"name": "norm_batch", "op": "norm", "tokens": 4096, "hidden": 7168, "dtype": "bf16", "res_dtype": "fp32",
         "post": True, "gate": "channel"},
        # the backward pass of a training batch, a gate per token (a gated shared expert)
        {"name": "norm_grad_batch", "op": "norm_grad", "tokens": 4096, "hidden": 7168, "dtype": "bf16",
         "res_dtype": "bf16", "post": True, "gate": "token"},
        # a small model trained in 32 bits: odd token count, a width that is no power of two, a full gate
        {"name": "norm_grad_odd", "op": "norm_grad", "tokens": 1537, "hidden": 1000, "dtype": "fp32",
         "res_dtype": "fp32", "post": True, "gate": "full"},
        # one request's next token through its adapter
        {"name": "lora_one", "op": "lora", "tokens": 1, "requests": 1, "adapters": 4, "rank": 64, "k": 7168,
         "n": 1536, "dtype": "bf16", "bare": 0.0},
        # a decode step of 64 requests over 32 small adapters, some requests without one
        {"name": "lora_decode", "op": "lora", "tokens": 64, "requests": 64, "adapters": 32, "rank": 16, "k": 7168,
         "n": 7168, "dtype": "bf16", "bare": 0.1},
        # the prompts of a few requests packed into one batch
        {"name": "lora_prompts", "op": "lora", "tokens": 4096, "requests": 7, "adapters": 8, "rank": 64, "k": 7168,
         "n": 7168, "dtype": "bf16", "bare": 0.1},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A row width: mostly a multiple of 8, sometimes any number."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.2 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["sort", "back", "back_grad", "norm", "norm_grad", "lora"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("sort", "back", "back_grad"):
        experts = _log(rng, 4, 256)
        c = {"op": op, "tokens": _log(rng, 1, 2048 if dtype == "fp32" else 4096),
             "k": rng.randint(1, min(8, experts)), "experts": experts, "ranks": rng.choice([1, 1, 2, 8]),
             "skew": rng.choice([0.0, 0.8, 1.2]), "hidden": _width(rng, 64, 7168), "dtype": dtype}
        if op == "back":
            c["weighted"] = rng.random() < 0.7
        return c
    if op in ("norm", "norm_grad"):
        return {"op": op, "tokens": _log(rng, 1, 4096), "hidden": _width(rng, 64, 7168), "dtype": dtype,
                "res_dtype": rng.choice([dtype, "fp32"]), "post": rng.random() < 0.8,
                "gate": rng.choice(["none", "channel", "token", "full"])}
    tokens = _log(rng, 1, 4096)
    rank = 8 * rng.randint(1, 16)
    return {"op": op, "tokens": tokens, "requests": rng.randint(1, min(tokens, 128)),
            "adapters": rng.randint(1, min(64, 2048 // rank)), "rank": rank, "k": 8 * _log(rng, 16, 896),
            "n": 8 * _log(rng, 16, 896), "dtype": rng.choice(["bf16", "fp16"]), "bare": rng.choice([0.0, 0.1, 0.5])}


# ---------------------------------------------------------------- inputs

class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, shape, dtype, scale=1.0):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    def uniform(self, shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(hi - lo).add_(lo)


def _routing(m, case):
    """Each token's k distinct experts of all ranks, as this rank numbers them (its own are 0 .. experts - 1), and
    the gate weights, which sum to 1 over a token's slots."""
    total = case["experts"] * case["ranks"]
    popular = -case["skew"] * torch.log(torch.arange(1, total + 1, device="cuda", dtype=torch.float32))
    popular = popular[torch.randperm(total, generator=m.g, device="cuda")]
    gumbel = -torch.log(-torch.log(m.uniform((case["tokens"], total), 1e-6, 1.0 - 1e-6)))
    ids = torch.topk(popular + gumbel, case["k"], dim=1).indices
    ids = (ids - (case["ranks"] // 2) * case["experts"]).to(torch.int32).contiguous()
    w = torch.softmax(m.normal((case["tokens"], case["k"]), torch.float32), dim=1)
    return ids, w


def _sorted_rows(ids, experts):
    """(first row of each expert, the slot of each row, the row of each slot); -1 where there is none."""
    flat = ids.reshape(-1).to(torch.int64)
    local = (flat >= 0) & (flat < experts)
    key = torch.where(local, flat, experts)
    order = torch.argsort(key, stable=True)
    off = torch.searchsorted(key[order], torch.arange(experts + 1, device=ids.device))
    place = torch.arange(flat.numel(), device=ids.device)
    row_slot = torch.where(place < off[experts], order, -1)
    slot_row = torch.empty_like(order)
    slot_row[order] = place
    slot_row = torch.where(local, slot_row, -1)
    return off.to(torch.int32), row_slot.to(torch.int32), slot_row.to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    m = _Maker(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("sort", "back", "back_grad"):
        dt, hidden, rows = DTYPES[case["dtype"]], case["hidden"], case["tokens"] * case["k"]
        s["ids"], s["w"] = _routing(m, case)
        s["experts"] = case["experts"]
        if op == "sort":
            s["x"] = m.normal((case["tokens"], hidden), dt)
            # the experts' input buffer, which a program keeps: rows that no pair takes stay as they are
            s["xs"] = torch.zeros((rows, hidden), device="cuda", dtype=dt)
            return s
        s["slot_row"] = _sorted_rows(s["ids"], case["experts"])[2]
        s["ys"] = m.normal((rows, hidden), dt)
        if op == "back":
            s["weighted"] = case["weighted"]
        else:
            s["dy"] = m.normal((case["tokens"], hidden), dt)
            s["dys"] = torch.zeros((rows, hidden), device="cuda", dtype=dt)
    elif op in ("norm", "norm_grad"):
        t, h = case["tokens"], case["hidden"]
        dt, rdt = DTYPES[case["dtype"]], DTYPES[case["res_dtype"]]
        s["y"] = m.normal((t, h), dt)
        s["residual"] = m.normal((t, h), rdt, 3.0)   # on the way back: the stored sum
        s["w_pre"] = (1.0 + 0.2 * m.normal((h,), torch.float32)).to(dt)
        s["w_post"] = (1.0 + 0.2 * m.normal((h,), torch.float32)).to(dt) if case["post"] else None
        shape = {"none": None, "channel": (h,), "token": (t, 1), "full": (t, h)}[case["gate"]]
        s["gate"] = None if shape is None else m.uniform(shape, 0.1, 1.0).to(dt)
        s["res_scale"] = 0.5
        if op == "norm_grad":
            s["d_normed"] = m.normal((t, h), dt)
            s["d_residual_out"] = m.normal((t, h), rdt)
    else:
        dt, n, r = DTYPES[case["dtype"]], case["adapters"], case["rank"]
        s["x"] = m.normal((case["tokens"], case["k"]), dt)
        s["y"] = m.normal((case["tokens"], case["n"]), dt)     # the shared projection's output
        s["a"] = m.normal((n, r, case["k"]), dt, case["k"] ** -0.5)
        s["b"] = m.normal((n, case["n"], r), dt, r ** -0.5)
        s["scale"] = m.uniform((n,), 0.5, 2.0)
        # requests are runs of tokens; each has an adapter, or none
        cuts = torch.randperm(case["tokens"] - 1, generator=m.g, device="cuda")[:case["requests"] - 1] + 1
        mark = torch.zeros(case["tokens"], device="cuda", dtype=torch.int64)
        mark[cuts] = 1
        of_request = torch.randint(0, n, (case["requests"],), generator=m.g, device="cuda")
        of_request = torch.where(m.uniform((case["requests"],)) < case["bare"], -1, of_request)
        s["adapter"] = of_request[torch.cumsum(mark, 0)].to(torch.int32).reshape(-1, 1)
        # the plan, made once for a step and used by all of its projections
        s["adapter_off"], s["row_slot"], _ = _sorted_rows(s["adapter"], n)
    return s


# ---------------------------------------------------------------- the operators

def _sort(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        off, row_slot, slot_row = mx.moe_sort(s["ids"], s["experts"])
        xs = mx.moe_permute(s["x"], slot_row, out=s["xs"])
    else:
        off, row_slot, slot_row = _sorted_rows(s["ids"], s["experts"])
        token = (row_slot.clamp(min=0) // s["ids"].shape[1]).to(torch.int64)
        xs = torch.where((row_slot >= 0)[:, None], s["x"][token], s["xs"])
    return {"expert_off": off, "row_slot": row_slot, "slot_row": slot_row, "xs": xs}


def _back(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        return {"y": mx.moe_unpermute(s["ys"], s["slot_row"], topk_w=s["w"] if s["weighted"] else None)}
    row = s["slot_row"].to(torch.int64)
    w = (s["w"] if s["weighted"] else torch.ones_like(s["w"])) * (row >= 0)
    picked = s["ys"][row.clamp(min=0)].float()
    return {"y": (picked * w[:, :, None]).sum(1).to(s["ys"].dtype)}


def _back_grad(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        dys, dw = mx.moe_unpermute_grad(s["dy"], s["ys"], s["slot_row"], s["w"], d_ys=s["dys"])
        return {"dys": dys, "dw": dw}
    row = s["slot_row"].to(torch.int64)
    kept = row >= 0
    dy = s["dy"].float()
    dw = (s["ys"][row.clamp(min=0)].float() * dy[:, None, :]).sum(2) * kept
    # an extra row takes what the slots without a row would write
    dys = torch.cat([s["dys"], s["dys"][:1]])
    to = torch.where(kept, row, s["dys"].shape[0]).reshape(-1)
    dys[to] = (dy[:, None, :] * s["w"][:, :, None]).to(dys.dtype).reshape(to.numel(), -1)
    return {"dys": dys[:-1], "dw": dw}


def _norm(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        normed, residual = mx.block_norm(s["residual"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                                         res_scale=s["res_scale"], eps=EPS)
        return {"normed": normed, "residual": residual}
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + s["res_scale"] * u
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"normed": n.to(s["y"].dtype), "residual": r.to(s["residual"].dtype)}


def _norm_back(x, w, dn):
    """(the gradient of x * rsqrt(mean(x^2) + eps) * w for x, and x * rsqrt(...))."""
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    xh = x * rstd
    d = dn * w
    return rstd * (d - xh * (d * xh).mean(1, keepdim=True)), xh


def _norm_grad(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        g = mx.block_norm_grad(s["residual"], s["w_pre"], s["d_normed"], d_residual_out=s["d_residual_out"],
                               y=s["y"], w_post=s["w_post"], gate=s["gate"], res_scale=s["res_scale"], eps=EPS)
        return {"d_residual": g[0], "dw_pre": g[1], "dy": g[2], "dw_post": g[3], "dgate": g[4]}
    dn, y, r = s["d_normed"].float(), s["y"].float(), s["residual"].float()
    dr, rh = _norm_back(r, s["w_pre"].float(), dn)
    dr = dr + s["d_residual_out"].float()
    out = {"d_residual": dr.to(s["residual"].dtype), "dw_pre": (dn * rh).sum(0), "dw_post": None, "dgate": None}
    gate = torch.ones((), device=y.device) if s["gate"] is None else s["gate"].float()
    du = s["res_scale"] * dr * gate
    u = y
    if s["w_post"] is not None:
        w_post = s["w_post"].float()
        dy, yh = _norm_back(y, w_post, du)
        u = yh * w_post
        out["dw_post"] = (du * yh).sum(0)
    else:
        dy = du
    out["dy"] = dy.to(s["y"].dtype)
    if s["gate"] is not None:
        dg = s["res_scale"] * dr * u
        if s["gate"].dim() == 1:
            out["dgate"] = dg.sum(0)
        elif s["gate"].shape[1] == 1:
            out["dgate"] = dg.sum(1, keepdim=True)
        else:
            out["dgate"] = dg.to(s["gate"].dtype)
    return out


def _lora(s):
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        return {"y": mx.lora_add(s["y"], s["x"], s["a"], s["b"], s["adapter_off"], s["row_slot"],
                                 scale=s["scale"])}
    n, r, k = s["a"].shape
    # every token through every adapter's narrow side, then only its own kept
    v = (s["x"].float() @ s["a"].float().reshape(n * r, k).t()).reshape(-1, n, r)
    mine = (s["adapter"].to(torch.int64) == torch.arange(n, device=v.device)) * s["scale"]
    v = v * mine[:, :, None]
    delta = v.reshape(-1, n * r) @ s["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    s["y"].copy_(s["y"].float() + delta)
    return {"y": s["y"]}


OPS = {"sort": _sort, "back": _back, "back_grad": _back_grad, "norm": _norm, "norm_grad": _norm_grad, "lora": _lora}


def run(state):
    return OPS[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("sort", "back", "back_grad"):
        t, pairs, h, z = case["tokens"], case["tokens"] * case["k"], case["hidden"], SIZE[case["dtype"]]
        local = pairs / case["ranks"]            # on average
        if op == "sort":
            return {"bytes": 12 * pairs + 4 * case["experts"] + z * h * (min(t, local) + local), "flops": 0}
        if op == "back":
            return {"bytes": 8 * pairs + z * h * (local + t), "flops": 2 * local * h}
        return {"bytes": 12 * pairs + z * h * (min(t, local) + 2 * local), "flops": 3 * local * h}
    if op in ("norm", "norm_grad"):
        t, h, z, rz = case["tokens"], case["hidden"], SIZE[case["dtype"]], SIZE[case["res_dtype"]]
        gate = {"none": 0, "channel": h, "token": t, "full": t * h}[case["gate"]]
        vec = z * h * (1 + case["post"])
        if op == "norm":
            return {"bytes": t * h * (2 * z + 2 * rz) + vec + z * gate, "flops": 10 * t * h}
        back = gate * (z if case["gate"] == "full" else 4)
        return {"bytes": t * h * (3 * z + 3 * rz) + vec + 4 * h * (1 + case["post"]) + z * gate + back,
                "flops": 25 * t * h}
    z, r, k, n = SIZE[case["dtype"]], case["rank"], case["k"], case["n"]
    tokens = case["tokens"] * (1 - case["bare"])
    # adapters that some request has, on average
    busy = case["adapters"] * (1 - (1 - (1 - case["bare"]) / case["adapters"]) ** case["requests"])
    return {"bytes": z * (tokens * (k + 2 * n) + busy * r * (k + n)), "flops": 2 * tokens * r * (k + n)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """What `run` gives, from the definitions, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        # rows in the order of (expert, slot), counted instead of sorted
        ids = s["ids"].reshape(-1)
        xs = s["xs"].double()
        at = 0
        for e in range(case["experts"]):
            slots = torch.nonzero(ids == e).reshape(-1)
            xs[at:at + slots.numel()] = s["x"][torch.div(slots, case["k"], rounding_mode="floor")].double()
            at += slots.numel()
        return {"expert_off": None, "row_slot": None, "slot_row": None, "xs": xs}
    if op in ("back", "back_grad"):
        rows = s["slot_row"].to(torch.int64)
        w = s["w"].double()
        if op == "back":
            y = torch.zeros((case["tokens"], case["hidden"]), device="cuda", dtype=torch.float64)
            for j in range(case["k"]):
                has = torch.nonzero(rows[:, j] >= 0).reshape(-1)
                part = s["ys"][rows[has, j]].double()
                y[has] += part * w[has, j, None] if case["weighted"] else part
            return {"y": y}
        dys = s["dys"].double()
        dw = torch.zeros_like(w)
        for j in range(case["k"]):
            has = torch.nonzero(rows[:, j] >= 0).reshape(-1)
            dy = s["dy"][has].double()
            dys[rows[has, j]] = w[has, j, None] * dy
            dw[has, j] = torch.linalg.vecdot(dy, s["ys"][rows[has, j]].double())
        return {"dys": dys, "dw": dw}
    if op in ("norm", "norm_grad"):
        y = s["y"].double()
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        if op == "norm":
            u = y
            if s["w_post"] is not None:
                u = u / torch.sqrt(y.square().sum(1, keepdim=True) / case["hidden"] + EPS) * s["w_post"].double()
            r = s["residual"].double() + s["res_scale"] * gate * u
            n = r / torch.sqrt(r.square().sum(1, keepdim=True) / case["hidden"] + EPS) * s["w_pre"].double()
            return {"normed": n, "residual": r}
        # through torch's own differentiation of the formula, with the stored sum as a variable
        r = s["residual"].double().requires_grad_()
        w_pre = s["w_pre"].double().requires_grad_()
        n = r / torch.sqrt(r.square().sum(1, keepdim=True) / case["hidden"] + EPS) * w_pre
        dr, dw_pre = torch.autograd.grad(n, (r, w_pre), s["d_normed"].double())
        dr = dr + s["d_residual_out"].double()
        y.requires_grad_()
        w_post = None if s["w_post"] is None else s["w_post"].double().requires_grad_()
        g = None if s["gate"] is None else gate.requires_grad_()
        u = y
        if w_post is not None:
            u = u / torch.sqrt(y.square().sum(1, keepdim=True) / case["hidden"] + EPS) * w_post
        u = s["res_scale"] * (u if g is None else g * u)
        wanted = [v for v in (y, w_post, g) if v is not None]
        got = dict(zip([id(v) for v in wanted], torch.autograd.grad(u, wanted, dr)))
        return {"d_residual": dr, "dw_pre": dw_pre, "dy": got[id(y)],
                "dw_post": None if w_post is None else got[id(w_post)], "dgate": None if g is None else got[id(g)]}
    y = s["y"].double()
    for a in range(case["adapters"]):
        mine = torch.nonzero(s["adapter"].reshape(-1) == a).reshape(-1)
        if mine.numel():
            v = s["x"][mine].double() @ s["a"][a].double().t()
            y[mine] += s["scale"][a].double() * (v @ s["b"][a].double().t())
    return {"y": y}
