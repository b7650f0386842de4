"""More of what a MoE layer runs next to its quantised experts, as cases that can be timed and compared:

- the router: scores, top-k and weights (`moe_gate`), the balance loss with the experts' counts (`moe_balance`), and the
  gradient of both (`moe_gate_grad`),
- projections of unquantised activations with 4-bit weights and group scales (`w4_linear`),
- a paged cache held in MXFP8 or MXFP4, written and read back (`cache_write`, `cache_read`).

`run` computes them in plain torch operations, or, with `own`, through this repository's package.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's router: 8 tokens over the 48 experts of a rank, serving
        {"name": "route_decode", "op": "route", "tokens": 8, "experts": 48, "k": 8, "score": "softmax", "bias": False,
         "renorm": True, "balance": False, "sequences": 1, "masked": 0.0, "dtype": "fp32"},
        # the router of a training batch: 4096 tokens over 384 experts, sigmoid scores with a selection bias, the
        # balance loss of each of 8 sequences
        {"name": "route_batch", "op": "route", "tokens": 4096, "experts": 384, "k": 8, "score": "sigmoid", "bias": True,
         "renorm": True, "balance": True, "sequences": 8, "masked": 0.0, "dtype": "fp32"},
        # logits in 16 bits, an odd number of experts of which some are switched off, one loss over the whole batch
        {"name": "route_odd", "op": "route", "tokens": 5003, "experts": 257, "k": 3, "score": "softmax", "bias": False,
         "renorm": False, "balance": True, "sequences": 1, "masked": 0.1, "dtype": "bf16"},
        # the backward pass of that training batch
        {"name": "route_grad_batch", "op": "route_grad", "tokens": 4096, "experts": 384, "k": 8, "score": "sigmoid",
         "bias": True, "renorm": True, "balance": True, "sequences": 8, "masked": 0.0, "dtype": "fp32"},
        # of a small model's, in 16 bits
        {"name": "route_grad_odd", "op": "route_grad", "tokens": 1537, "experts": 60, "k": 6, "score": "softmax",
         "bias": False, "renorm": False, "balance": True, "sequences": 11, "masked": 0.0, "dtype": "bf16"},
        # one request's next token through a narrow projection
        {"name": "w4_one", "op": "w4", "tokens": 1, "k": 7168, "n": 1536, "format": "mxfp4", "group": 32, "zeros": False,
         "dtype": "bf16"},
        # a decode step of 64 requests through a wide one
        {"name": "w4_decode", "op": "w4", "tokens": 64, "k": 7168, "n": 7168, "format": "int4", "group": 128,
         "zeros": True, "dtype": "fp16"},
        # a few tokens, sizes that are no powers of two, small groups
        {"name": "w4_odd", "op": "w4", "tokens": 11, "k": 4128, "n": 5003, "format": "int4", "group": 32,
         "zeros": False, "dtype": "bf16"},
        # the prompts of a batch
        {"name": "w4_prompts", "op": "w4", "tokens": 4096, "k": 7168, "n": 7168, "format": "mxfp4", "group": 32,
         "zeros": False, "dtype": "bf16"},
        # one short conversation's next token: its row written, the conversation read
        {"name": "cache_one", "op": "cache", "sequences": 1, "mean": 100, "new": 1, "width": 576, "page": 16,
         "format": "mxfp8", "dtype": "bf16"},
        # a decode step of 64 conversations of some thousand tokens each
        {"name": "cache_decode", "op": "cache", "sequences": 64, "mean": 2000, "new": 1, "width": 576, "page": 64,
         "format": "mxfp8", "dtype": "bf16"},
        # the prompts of a few requests written whole, wide rows in 4 bits, read for their attention
        {"name": "cache_prompts", "op": "cache", "sequences": 7, "mean": 1200, "new": 0, "width": 2048, "page": 128,
         "format": "mxfp4", "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "w4", "w4", "cache", "cache"])
    if op in ("route", "route_grad"):
        tokens, experts = _log(rng, 1, 4096), _log(rng, 4, 384)
        return {"op": op, "tokens": tokens, "experts": experts, "k": rng.randint(1, min(8, experts)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7,
                "balance": rng.random() < (0.6 if op == "route" else 0.8),
                "sequences": _log(rng, 1, min(tokens, 64)), "masked": rng.choice([0.0, 0.0, 0.1]),
                "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"])}
    if op == "w4":
        fmt = rng.choice(["mxfp4", "int4"])
        group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
        return {"op": op, "tokens": _log(rng, 1, 4096), "k": group * _log(rng, 4, 7168 // group),
                "n": _log(rng, 64, 7168), "format": fmt, "group": group, "zeros": fmt == "int4" and rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "fp16"])}
    sequences, width = _log(rng, 1, 64), 32 * _log(rng, 2, 64)
    return {"op": op, "sequences": sequences, "mean": _log(rng, 1, min(8000, 70_000_000 // (sequences * width))),
            "new": rng.choice([0, 1, 1, 3]), "width": width, "page": rng.choice([16, 32, 64, 128]),
            "format": rng.choice(["mxfp8", "mxfp4"]), "dtype": rng.choice(["bf16", "fp16", "fp32"])}


# ---------------------------------------------------------------- inputs

class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, shape, dtype, scale=1.0):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    def uniform(self, shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(hi - lo).add_(lo)

    def integers(self, shape, lo, hi, dtype):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda").to(dtype)

    def cuts(self, total, parts):
        """Offsets [parts + 1] of `parts` ragged pieces of 0 .. total, none empty where total allows it."""
        cut = torch.randperm(total - 1, generator=self.g, device="cuda")[:parts - 1] + 1
        ends = torch.tensor([0, total], device="cuda")
        return torch.cat([ends[:1], torch.sort(cut).values, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    m = _Maker(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("route", "route_grad"):
        t, e = case["tokens"], case["experts"]
        # some experts are more popular than others
        logits = m.normal((t, e), torch.float32, 1.5) + m.normal((e,), torch.float32, 0.5)
        # those that are switched off; k stay on in any case
        off = m.uniform((e,)) < case["masked"]
        off[torch.randperm(e, generator=m.g, device="cuda")[:case["k"]]] = False
        s["logits"] = logits.masked_fill(off, -math.inf).to(DTYPES[case["dtype"]])
        s["bias"] = m.uniform((e,), -0.05, 0.05) if case["bias"] else None
        s["seq_off"] = m.cuts(t, case["sequences"]) if case["balance"] and case["sequences"] > 1 else None
        s["scale"], s["coef"] = (2.5 if case["renorm"] else 1.0), 0.01
        if op == "route_grad":
            s["ids"] = _top_k(s)
            s["d_w"] = m.normal((t, case["k"]), torch.float32)
            s["counts"] = _counts(s, s["ids"]) if case["balance"] else None
            s["d_loss"] = m.uniform((case["sequences"],), 0.5, 1.5) if case["balance"] else None
    elif op == "w4":
        dt, k, n, g = DTYPES[case["dtype"]], case["k"], case["n"], case["group"]
        s["x"] = m.normal((case["tokens"], k), dt)
        s["w"] = m.integers((n, k // 2), 0, 256, torch.uint8)
        s["zeros"] = m.integers((n, k // g), 0, 16, torch.uint8) if case["zeros"] else None
        if case["format"] == "mxfp4":
            s["w_s"] = m.integers((n, k // g), 114, 125, torch.uint8)
        else:
            s["w_s"] = m.uniform((n, k // g), 0.2 * k ** -0.5, 0.6 * k ** -0.5).to(dt)
    else:
        width, page, seqs = case["width"], case["page"], case["sequences"]
        total = max(seqs * max(1, case["new"]), seqs * case["mean"])
        off = m.cuts(total, seqs)
        length = off[1:] - off[:-1]
        # pages in no order, a table of them for each sequence, as wide as the longest needs
        need = (length + page - 1) // page
        wide, pages = int(need.max()), int(need.sum()) + 3
        order = torch.randperm(pages, generator=m.g, device="cuda").to(torch.int32)
        first = torch.cumsum(need, 0) - need
        col = torch.arange(wide, device="cuda")
        s["table"] = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=pages - 1)], -1)
        s["table"] = s["table"].to(torch.int32).contiguous()
        s["seq_off"], s["rows"] = off, total
        seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), length)
        pos = torch.arange(total, device="cuda") - off[seq]
        s["seq"], s["pos"] = seq, pos
        slot = s["table"][seq, pos // page].to(torch.int64) * page + pos % page
        # what is new: the last rows of each sequence, or all
        late = pos >= (length - case["new"])[seq] if case["new"] else torch.ones_like(pos, dtype=torch.bool)
        s["slots"] = slot[late].to(torch.int32)
        dt = DTYPES[case["dtype"]]
        # channels differ in size, some rows are small
        channel = torch.exp(m.normal((width,), torch.float32))
        rows = s["slots"].numel()
        s["x"] = (m.normal((rows, width), torch.float32) * channel * m.uniform((rows, 1), 0.01, 1.0)).to(dt)
        wide8 = width if case["format"] == "mxfp8" else width // 2
        s["codes"] = torch.zeros((pages, page, wide8), device="cuda", dtype=torch.uint8)
        s["scales"] = torch.zeros((pages, page, width // 32), device="cuda", dtype=torch.uint8)
        old = slot[~late]
        if old.numel():
            # what stands there: finite codes under scales of ordinary size
            codes = m.integers((old.numel(), wide8), 0, 256, torch.uint8)
            if case["format"] == "mxfp8":
                codes = torch.where((codes & 0x7F) == 0x7F, 0x30, codes)
            s["codes"].view(-1, wide8)[old] = codes
            s["scales"].view(-1, width // 32)[old] = m.integers((old.numel(), width // 32), 114, 122, torch.uint8)
    return s


# ---------------------------------------------------------------- the router

def _scores(s):
    """The scores in 64 bits: which experts are chosen hangs on values that lie side by side."""
    z = s["logits"].double()
    if s["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def _top_k(s):
    """The k experts of each token by score (and bias), the lower index first; -1 where none that is on is left."""
    z, k = s["logits"].double(), s["case"]["k"]
    key = z if s["bias"] is None else _scores(s) + s["bias"].double()
    key = torch.where(z == -math.inf, -math.inf, key)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(top[:, :k] == -math.inf, -1, ids[:, :k]).to(torch.int32)


def _sequence(s):
    """(the sequence of each token, the tokens of each sequence)."""
    t = s["logits"].shape[0]
    if s["seq_off"] is None:
        return torch.zeros(t, device="cuda", dtype=torch.int64), torch.tensor([t], device="cuda")
    length = (s["seq_off"][1:] - s["seq_off"][:-1]).to(torch.int64)
    return torch.repeat_interleave(torch.arange(length.numel(), device="cuda"), length, output_size=t), length


def _counts(s, ids):
    """The slots of each expert in each sequence."""
    seq, length = _sequence(s)
    e = s["case"]["experts"]
    place = torch.where(ids >= 0, seq[:, None] * e + ids, length.numel() * e)
    counts = torch.zeros(length.numel() * e + 1, device="cuda", dtype=torch.int32)
    counts.index_add_(0, place.reshape(-1).to(torch.int64), torch.ones(ids.numel(), device="cuda", dtype=torch.int32))
    return counts[:-1].reshape(-1, e)


def _probabilities(s):
    """The scores in 32 bits, and the same as shares of one."""
    z = s["logits"].float()
    if s["case"]["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
        total = score.sum(1, keepdim=True)
        return score, torch.where(total > 0, score / total, 0.0)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    return p, p


def _route(s):
    c = s["case"]
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        ids, w = mx.moe_gate(s["logits"], c["k"], score=c["score"], bias=s["bias"], renorm=c["renorm"],
                             scale=s["scale"])
        if not c["balance"]:
            return {"ids": ids, "w": w, "counts": None, "loss": None}
        loss, counts = mx.moe_balance(s["logits"], ids, seq_off=s["seq_off"], score=c["score"], coef=s["coef"])
        return {"ids": ids, "w": w, "counts": counts, "loss": loss}
    ids = _top_k(s)
    score, p = _probabilities(s)
    w = torch.gather(score, 1, ids.clamp(min=0).to(torch.int64)) * (ids >= 0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * s["scale"]
    if not c["balance"]:
        return {"ids": ids, "w": w, "counts": None, "loss": None}
    counts = _counts(s, ids)
    seq, length = _sequence(s)
    share = torch.zeros(counts.shape, device="cuda", dtype=torch.float32).index_add_(0, seq, p) / length[:, None]
    load = counts.float() * (c["experts"] / c["k"]) / length[:, None]
    return {"ids": ids, "w": w, "counts": counts, "loss": s["coef"] * (load * share).sum(1)}


def _route_grad(s):
    c = s["case"]
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        return {"d_logits": mx.moe_gate_grad(s["logits"], s["ids"], d_w=s["d_w"], counts=s["counts"],
                                             d_loss=s["d_loss"], seq_off=s["seq_off"], score=c["score"],
                                             renorm=c["renorm"], scale=s["scale"], coef=s["coef"])}
    score, p = _probabilities(s)
    at, has = s["ids"].clamp(min=0).to(torch.int64), s["ids"] >= 0
    d = s["d_w"] * s["scale"] * has
    if c["renorm"]:
        mine = torch.gather(score, 1, at) * has
        total = mine.sum(1, keepdim=True)
        mean = (d * mine).sum(1, keepdim=True) / total
        d = torch.where(total > 0, (d - mean) / total, 0.0) * has
    g = torch.zeros_like(score).scatter_add_(1, at, d)             # for the scores
    b = torch.zeros_like(score)                                    # for the shares of one
    if c["balance"]:
        seq, length = _sequence(s)
        n = length.float()
        b = ((s["coef"] * c["experts"] / c["k"]) * s["d_loss"] / (n * n))[:, None] * s["counts"].float()
        b = b[seq]
    b = p * (b - (p * b).sum(1, keepdim=True))                     # times the score
    if c["score"] == "sigmoid":
        d = (g * score + b) * (1.0 / (1.0 + torch.exp(s["logits"].float())))
    else:
        d = score * (g - (score * g).sum(1, keepdim=True)) + b
    return {"d_logits": torch.where(s["logits"] == -math.inf, 0.0, d).to(s["logits"].dtype)}


# ---------------------------------------------------------------- 4-bit weights

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _codes(w):
    """The 4-bit codes of packed bytes, the low one first."""
    return torch.stack([w & 15, w >> 4], dim=-1).reshape(*w.shape[:-1], -1).to(torch.int32)


def _e8m0(b):
    """2^(b - 127), NaN for 255."""
    return torch.where(b == 255, math.nan, torch.ldexp(torch.ones((), device=b.device), b.to(torch.int32) - 127))


def _w4(s):
    c = s["case"]
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        return {"y": mx.w4_linear(s["x"], s["w"], s["w_s"], zeros=s["zeros"])}
    codes = _codes(s["w"])
    if c["format"] == "mxfp4":
        lut = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
        w, scale = lut[codes], _e8m0(s["w_s"])
    else:
        zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(c["group"], 1)
        w, scale = codes.float() - zero, s["w_s"].float()
    w = (w.reshape(c["n"], -1, c["group"]) * scale[:, :, None]).reshape(c["n"], -1)
    return {"y": (s["x"].float() @ w.t()).to(s["x"].dtype)}


# ---------------------------------------------------------------- the cache

# bits of the mantissa, the smallest normal exponent, the largest exponent, the largest value
ELEMENT = {"mxfp8": (3, -6, 8, 448.0), "mxfp4": (1, 0, 2, 6.0)}


def _encode(x, fmt):
    """(codes, scales) of rows of 32-bit values."""
    mantissa, low, high, largest = ELEMENT[fmt]
    rows = x.shape[0]
    x = x.reshape(rows, -1, 32)
    amax = x.abs().amax(2)
    byte = (torch.frexp(amax).exponent - 1 - high + 127).clamp(0, 254)
    byte = torch.where(amax == 0, 0, byte)
    v = torch.ldexp(x, (127 - byte)[:, :, None])
    size = v.abs()
    exponent = (torch.frexp(size).exponent - 1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(size), exponent - mantissa)
    size = (torch.round(size / step) * step).clamp(max=largest)      # halves to even
    # the code of a size: its exponent's field and what is above the field's first value
    exponent = (torch.frexp(size).exponent - 1).clamp(min=low)
    place = torch.ldexp(size, mantissa - exponent).to(torch.int32)     # with the leading one where there is one
    code = ((exponent - low) << mantissa) + place
    sign = torch.signbit(v).to(torch.int32)
    code = (code + (sign << (7 if fmt == "mxfp8" else 3))).reshape(rows, -1)
    if fmt == "mxfp4":
        code = code[:, 0::2] + (code[:, 1::2] << 4)
    return code.to(torch.uint8), byte.to(torch.uint8)


def _decode(codes, scales, fmt):
    if fmt == "mxfp8":
        c = torch.arange(256, device="cuda")
        e, f = (c >> 3) & 15, (c & 7).float()
        lut = torch.where(e > 0, torch.ldexp(8 + f, e - 10), torch.ldexp(f, e - 9))
        lut = torch.where((c & 127) == 127, math.nan, torch.where(c >= 128, -lut, lut))
        v = lut[codes.to(torch.int32)]
    else:
        v = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")[_codes(codes)]
    return (v.reshape(v.shape[0], -1, 32) * _e8m0(scales)[:, :, None]).reshape(v.shape[0], -1)


def _cache(s):
    c = s["case"]
    fmt, page = c["format"], c["page"]
    if own:
        import mxfp4_block_scaled_e2m1_amd as mx
        mx.cache_write(fmt, s["x"], s["slots"], s["codes"], s["scales"])
        return {"rows": mx.cache_read(fmt, s["codes"], s["scales"], s["table"], s["seq_off"], rows=s["rows"],
                                      dtype=s["x"].dtype)}
    codes, scales = s["codes"].view(-1, s["codes"].shape[2]), s["scales"].view(-1, s["scales"].shape[2])
    at = s["slots"].to(torch.int64)
    codes[at], scales[at] = _encode(s["x"].float(), fmt)
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["seq_off"], row, right=True) - 1
    pos = row - s["seq_off"][seq]
    at = s["table"][seq, pos // page].to(torch.int64) * page + pos % page
    return {"rows": _decode(codes[at], scales[at], fmt).to(s["x"].dtype)}


OPS = {"route": _route, "route_grad": _route_grad, "w4": _w4, "cache": _cache}


def run(state):
    return OPS[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        t, e, k, z = case["tokens"], case["experts"], case["k"], SIZE[case["dtype"]]
        stats = case["balance"] * case["sequences"] * (4 * e + 8)
        if op == "route":
            return {"bytes": z * t * e + 8 * t * k + stats + 4 * e * case["bias"], "flops": 10 * t * e}
        return {"bytes": 2 * z * t * e + 8 * t * k + stats, "flops": 12 * t * e}
    if op == "w4":
        t, k, n, z = case["tokens"], case["k"], case["n"], SIZE[case["dtype"]]
        group = k // case["group"] * (1 if case["format"] == "mxfp4" else z + case["zeros"])
        return {"bytes": z * t * (k + n) + n * (k // 2 + group), "flops": 2 * t * k * n}
    rows = max(case["sequences"] * max(1, case["new"]), case["sequences"] * case["mean"])
    # a sequence shorter than what is new has fewer new rows; none is in the listed cases
    new = case["sequences"] * case["new"] if case["new"] else rows
    held = case["width"] // (1 if case["format"] == "mxfp8" else 2) + case["width"] // 32
    z = SIZE[case["dtype"]]
    return {"bytes": new * (z * case["width"] + held + 4) + rows * (held + z * case["width"]),
            "flops": 2 * rows * case["width"]}


# ---------------------------------------------------------------- 64 bits

def _exact_route(s, case):
    """Token by token in order of preference, one expert after the other taken away."""
    z = s["logits"].double()
    if case["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(z, 1))
        score = share = p
    else:
        score = torch.sigmoid(z)
        share = score / score.sum(1, keepdim=True)
    left = z.clone() if s["bias"] is None else torch.where(z == -math.inf, z, score + s["bias"].double())
    w = torch.zeros((case["tokens"], case["k"]), device="cuda", dtype=torch.float64)
    taken = torch.zeros_like(z)
    for j in range(case["k"]):
        best = left.amax(1, keepdim=True)
        here = (left == best) & (best > -math.inf)
        here = here & (torch.cumsum(here, 1) == 1)
        w[:, j] = (score * here).sum(1)
        taken += here
        left = left.masked_fill(here, -math.inf)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    loss = None
    if case["balance"]:
        bounds = [0, case["tokens"]] if s["seq_off"] is None else s["seq_off"].tolist()
        loss = torch.stack([(taken[a:b].mean(0) * share[a:b].mean(0)).sum() for a, b in zip(bounds, bounds[1:])])
        loss = loss * (s["coef"] * case["experts"] / case["k"])
    return {"ids": None, "w": w * s["scale"], "counts": None, "loss": loss}


def _exact_route_grad(s, case):
    """Through torch's own differentiation of the formula. Experts that are off are left out of it."""
    z = s["logits"].double()
    on = z > -math.inf
    z = torch.where(on, z, 0.0).requires_grad_()
    if case["score"] == "softmax":
        score = share = torch.softmax(torch.where(on, z, -math.inf), 1)
    else:
        score = torch.sigmoid(z) * on
        share = score / score.sum(1, keepdim=True)
    has = s["ids"] >= 0
    w = torch.gather(score, 1, s["ids"].clamp(min=0).to(torch.int64)) * has
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    total = (w * s["scale"] * s["d_w"].double()).sum()
    if case["balance"]:
        bounds = [0, case["tokens"]] if s["seq_off"] is None else s["seq_off"].tolist()
        for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
            load = s["counts"][i].double() / (b - a)
            total = total + s["d_loss"][i].double() * (s["coef"] * case["experts"] / case["k"]) * \
                (load * share[a:b].mean(0)).sum()
    return {"d_logits": torch.autograd.grad(total, z)[0]}


def _exact_w4(s, case):
    w = s["w"].to(torch.int64)
    code = torch.empty((case["n"], case["k"]), device="cuda", dtype=torch.int64)
    code[:, 0::2], code[:, 1::2] = w % 16, w // 16
    group = torch.arange(case["k"], device="cuda") // case["group"]
    if case["format"] == "mxfp4":
        size, sign = code % 8, 1.0 - 2.0 * (code // 8)
        # 0, 1/2, 1, 3/2, then two values a power of two
        value = torch.where(size < 4, size * 0.5, (2.0 + size % 2) * torch.where(size < 6, 1.0, 2.0)).double() * sign
        scale = torch.exp2(s["w_s"].double() - 127.0)
    else:
        value = code.double() - (8.0 if s["zeros"] is None else s["zeros"].double()[:, group])
        scale = s["w_s"].double()
    return {"y": s["x"].double() @ (value * scale[:, group]).t()}


def _grid(fmt):
    """The sizes that an element can have, in order; the place of a size has the parity of its code."""
    if fmt == "mxfp4":
        return torch.tensor(E2M1, device="cuda", dtype=torch.float64)
    sizes = [f * 2.0 ** -9 for f in range(8)] + [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)]
    return torch.tensor(sizes[:127], device="cuda", dtype=torch.float64)


def _exact_cache(s, case):
    fmt, page, width = case["format"], case["page"], case["width"]
    grid = _grid(fmt)
    # what stands in the cache
    slot = s["table"][s["seq"], s["pos"] // page].to(torch.int64) * page + s["pos"] % page
    codes = s["codes"].reshape(-1, s["codes"].shape[2])[slot].to(torch.int64)
    if fmt == "mxfp4":
        codes = torch.stack([codes % 16, codes // 16], 2).reshape(-1, width)
    half = 8 if fmt == "mxfp4" else 128
    out = grid[(codes % half).clamp(max=grid.numel() - 1)] * (1.0 - 2.0 * (codes // half))
    scale = torch.exp2(s["scales"].reshape(-1, width // 32)[slot].double() - 127.0)
    out = out * scale.repeat_interleave(32, 1)
    # the new rows: each value to the nearest of the grid, the even one of two
    x = s["x"].double().reshape(-1, 32)
    amax = x.abs().amax(1, keepdim=True)
    power = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    power = power - (torch.exp2(power) > amax).double() + (torch.exp2(power + 1) <= amax).double()
    scale = torch.where(amax > 0, torch.exp2((power - (2 if fmt == "mxfp4" else 8)).clamp(min=-127)), 2.0 ** -127)
    v = (x / scale).abs()
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - v, v - grid[lo]
    near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (v >= grid[-1]), hi, lo)
    new = (grid[near] * torch.sign(x) * scale).reshape(-1, width)
    where = torch.full((s["codes"].shape[0] * page,), -1, device="cuda", dtype=torch.int64)
    where[s["slots"].to(torch.int64)] = torch.arange(new.shape[0], device="cuda")
    at = where[slot]
    return {"rows": torch.where((at >= 0)[:, None], new[at.clamp(min=0)], out)}


def exact(case, seed):
    """What `run` gives, from the definitions, in 64 bits."""
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "w4": _exact_w4,
            "cache": _exact_cache}[case["op"]](s, case)
