"""More of the experts' operators, as cases to measure: routing (scores, groups,
top-k, gate weights) and its backward pass, quantisation to MX-FP4, and the
gated feed-forward block and the linear layer whose weights are MX-FP4.

``own = False`` computes a case in plain torch operations, in 32 bits, rounded
once at the end (what decides between experts in 64 bits, so that the order does
not hang on a rounding); ``own = True`` calls libmoe.  Rows that hold no token
(pad rows and rows past the last one in use) are not part of any result: both
sides leave them as prepare() made them.

MX-FP4: 32 neighbouring values share a scale 2^X, X = floor(log2 amax) - 2, held
as the byte X + 127; a value is E2M1(v 2^-X), two of them in a byte, the first in
the low half.
"""
import math

import numpy as np
import torch

own = False

ACT = ("none", "silu", "gelu_tanh", "relu")
GELU_C = math.sqrt(2.0 / math.pi)


def _route(name, op, tokens, experts, top_k, **more):
    c = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score="softmax", logits="fp32", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, dense=False, masked=0.0, padded=0.0)
    c.update(more)
    return dict(c, name=name) if name else c


def _expert(name, op, tokens, hidden, ffn, experts, top_k, **more):
    c = dict(op=op, tokens=tokens, hidden=hidden, ffn=ffn, experts=experts, top_k=top_k, pad=1, x="mxfp4",
             act="silu" if op == "glu" else "none", bias=False, residual=False, out="bf16", skew=0.0, masked=0.0)
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a chat: sigmoid scores, a balancing bias, four of eight groups
        _route("route_one_token", "route", 1, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4,
               group_top=2, scale=2.5),
        # a long prompt's routing from a bf16 router
        _route("route_prefill", "route", 16384, 128, 8, logits="bf16"),
        # the same with groups, bias and a padded batch's empty rows
        _route("route_groups", "route", 8192, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4,
               group_top=2, scale=2.5, padded=0.05),
        # a small fine-tuning batch, some experts switched off, with the gradient of a balance loss
        _route("route_backward_odd", "route_backward", 333, 60, 3, renormalize=False, dense=True, masked=0.05,
               padded=0.1),
        # a training step's routing gradients
        _route("route_backward", "route_backward", 16384, 128, 8, logits="bf16", dense=True),
        # a few activations' rows
        dict(name="quantize_rows", op="quantize", rows=333, cols=544, dtype="bf16"),
        # the gate and up projections of 64 experts, laid out once after loading
        dict(name="quantize_weights", op="quantize", rows=131072, cols=4096, dtype="bf16"),
        # one token of a chat: six experts' weights are read, nothing else counts
        _expert("glu_one_token", "glu", 1, 4096, 1024, 64, 6),
        # a decode batch: FP8 rows, and the result quantised for the next product
        _expert("glu_decode", "glu", 128, 7168, 2048, 256, 8, x="fp8", out="mxfp4"),
        # a long prefill from MX-FP4 rows: the largest case
        _expert("glu_prefill", "glu", 8192, 7168, 2048, 256, 8),
        # a prompt's down projection from FP8 rows, with bias and residual rows in the epilogue
        _expert("linear_prefill", "linear", 4096, 4096, 2048, 64, 6, pad=128, x="fp8", bias=True, residual=True),
        # a skewed, ragged prompt; rows whose scales are not a whole number of 32-bit words
        _expert("linear_ragged", "linear", 1501, 7168, 1056, 32, 4, skew=1.0, masked=0.05),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


MOST_FLOPS, MOST_WEIGHTS = 3.0e12, 3.0e9  # of a drawn case: below the largest listed one


def _draw_route(rng, op):
    groups = rng.choice((1, 1, 2, 4, 8))
    each = _log(rng, 2, 512 // groups)
    experts = groups * each
    top_groups = rng.randint(1, groups)
    top_k = rng.randint(1, min(16, top_groups * each))
    return _route(None, op, _log(rng, 1, 32768), experts, top_k, score=rng.choice(("softmax", "sigmoid")),
                  logits=rng.choice(("fp32", "bf16")), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                  group_top=rng.choice((1, 2)), renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                  dense=rng.random() < 0.5, masked=rng.choice((0.0, 0.0, 0.05, 0.5)),
                  padded=rng.choice((0.0, 0.0, 0.1, 0.5)))


def draw(rng):
    while True:
        op = rng.choice(("route", "route", "route_backward", "quantize", "glu", "glu", "linear", "linear"))
        if op.startswith("route"):
            return _draw_route(rng, op)
        if op == "quantize":
            c = dict(op=op, rows=_log(rng, 1, 1 << 18), cols=32 * _log(rng, 1, 512), dtype="bf16")
            if c["rows"] * c["cols"] < 5e8:
                return c
            continue
        fmt = rng.choice(("mxfp4", "mxfp4", "fp8"))
        # the contraction covers whole scale blocks of the rows; the other size is in 32s
        wide = 128 if fmt == "fp8" else 32
        by_hidden, by_ffn = (wide, 32) if op == "glu" else (32, wide)
        hidden = by_hidden * _log(rng, max(1, 64 // by_hidden), 7168 // by_hidden)
        ffn = by_ffn * _log(rng, max(1, 64 // by_ffn), 2048 // by_ffn)
        experts = _log(rng, 1, 256)
        c = _expert(None, op, _log(rng, 1, 16384), hidden, ffn, experts, rng.randint(1, min(8, experts)),
                    pad=rng.choice((1, 1, 16, 128)), x=fmt, bias=rng.random() < 0.5,
                    skew=rng.choice((0.0, 0.0, 0.5, 1.0)), masked=rng.choice((0.0, 0.0, 0.1, 0.5)))
        if op == "glu":
            c["act"] = rng.choice(ACT[1:])
            # small enough that decoding the result does not hide the product's time
            small = c["tokens"] * c["top_k"] * ffn < 1 << 23
            c["out"] = rng.choice(("bf16", "mxfp4")) if small else "bf16"
        else:
            c["act"], c["residual"] = rng.choice(ACT), rng.random() < 0.5
        # padded to the longest expert, the plain form does more than the operator
        longest = min(c["tokens"], 1 + int(c["tokens"] * c["top_k"] / experts * (1 + 3 * c["skew"])))
        sizes = experts * ffn * hidden * (2 if op == "glu" else 1)
        if 2 * longest * sizes < MOST_FLOPS and sizes < MOST_WEIGHTS:
            return c


def _dims(case):
    """(columns of the weights, rows of the weights, columns of the result) of one expert."""
    if case["op"] == "glu":
        return case["hidden"], 2 * case["ffn"], case["ffn"]
    return case["ffn"], case["hidden"], case["hidden"]


def work(case):
    op = case["op"]
    if op.startswith("route"):
        pairs, cells = case["tokens"] * case["top_k"], case["tokens"] * case["experts"]
        size = 4 if case["logits"] == "fp32" else 2
        if op == "route":
            return {"bytes": cells * (size + 4 * case["dense"]) + 8 * pairs, "flops": 6 * cells}
        return {"bytes": cells * (2 * size + 4 * case["dense"]) + 8 * pairs, "flops": 10 * cells}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 + 0.5 + 1 / 32), "flops": 4 * n}
    pairs = case["tokens"] * case["top_k"] * (1 - case["masked"])
    active = case["experts"] * (1 - (1 - 1 / case["experts"]) ** pairs)
    k, n, out = _dims(case)
    x = 1 + 4 / 128 if case["x"] == "fp8" else 17 / 32
    y = 17 / 32 if case["out"] == "mxfp4" else 4 if case["residual"] else 2
    return {"bytes": pairs * (x * k + y * out) + active * k * n * 17 / 32, "flops": 2 * pairs * k * n}


# ---- number formats ---------------------------------------------------------------


def _mx(v):
    """MX-FP4 codes [.., C / 2] and scale bytes [.., C / 32] of fp32 values [.., C]."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    x = ((bits >> 23) - 129).clamp(min=-127)
    a = b.abs() * ((127 - x) << 23).view(torch.float32)[..., None]
    # round to nearest, ties to the even code: steps of 1/2 up to 2, of 1 up to 4, then of 2
    code = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    code = code.clamp(max=7).to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.reshape(*v.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (x + 127).to(torch.uint8)


def _mx_value(codes, scales):
    """The values, in 32 bits: an E2M1 code's bits are those of an fp16 number, times 2^14."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).to(torch.int16)
    v = (((c & 7) << 9) | ((c & 8) << 12)).view(torch.float16).float() * 2.0 ** 14
    v = v.reshape(*codes.shape[:-1], -1, 32) * (scales.int() << 23).view(torch.float32)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _fp8(x):
    """E4M3 codes and scales of 1x128 blocks: scale = amax / 448."""
    blocks = x.reshape(x.shape[0], -1, 128)
    scale = blocks.abs().amax(-1) / 448.0
    codes = (blocks / scale.clamp(min=1e-30)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape).view(torch.uint8), scale


def _fp8_value(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, dim=-1)


# ---- inputs -----------------------------------------------------------------------


def _route_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n, e, k = case["tokens"], case["experts"], case["top_k"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def chance(share, *shape):
        return torch.rand(*shape, generator=g, device="cuda") < share

    logits = randn(n, e) + 0.5 * randn(e)
    logits = logits.masked_fill(chance(case["masked"], e), -math.inf)  # experts switched off
    logits = logits.masked_fill(chance(case["padded"], n, 1), -math.inf)  # rows without a token
    s = {"case": case, "logits": logits.bfloat16() if case["logits"] == "bf16" else logits}
    s["bias"] = 0.1 * randn(e) if case["bias"] else None
    if case["op"] == "route_backward":
        s["dweights"] = randn(n, k)
        s["dscores"] = 0.01 * randn(n, e) if case["dense"] else None
        s["ids"] = _choose(case, s["logits"].float(), s["bias"])
        s["dlogits"] = torch.zeros_like(s["logits"])
    else:
        s["ids"] = torch.zeros(n, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(n, k, device="cuda")
        s["scores"] = torch.zeros(n, e, device="cuda") if case["dense"] else None
    return s


def _quantize_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.empty(case["rows"], case["cols"], dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    # a few columns of larger values, as activations and some projections have
    x *= 1 + 7 * (torch.rand(case["cols"], generator=g, device="cuda") < 0.02)
    s = {"case": case, "x": x}
    s["codes"] = torch.zeros(case["rows"], case["cols"] // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.zeros(case["rows"], case["cols"] // 32, dtype=torch.uint8, device="cuda")
    return s


def _expert_inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    tokens, experts, top_k, pad = case["tokens"], case["experts"], case["top_k"], case["pad"]
    logits = randn(tokens, experts) + case["skew"] * randn(experts)
    ids = logits.topk(top_k, dim=1).indices.int()
    if case["masked"]:
        ids[torch.rand(tokens, top_k, generator=g, device=dev) < case["masked"]] = -1
    flat = ids.cpu().numpy().reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // pad) * pad)])
    total = tokens * top_k + experts * (pad - 1)
    # the packed rows that hold a token, expert by expert
    rows = np.concatenate([np.arange(offsets[e], offsets[e] + counts[e]) for e in range(experts)])
    s = {"case": case, "ids": ids, "counts": counts, "offsets": offsets, "total": total,
         "rows": torch.from_numpy(rows.astype(np.int64)).to(dev)}

    def packed(cols):
        """Rows of a packed buffer: values where a token is, zeros elsewhere."""
        out = torch.zeros(total, cols, device=dev)
        out[s["rows"]] = randn(rows.size, cols)
        return out

    k, n, out = _dims(case)
    s["x"], s["x_scales"] = (_fp8 if case["x"] == "fp8" else _mx)(packed(k))
    s["w"] = torch.empty(experts, n, k // 2, dtype=torch.uint8, device=dev)
    s["w_scales"] = torch.empty(experts, n, k // 32, dtype=torch.uint8, device=dev)
    for e in range(experts):  # one expert at a time: little memory
        s["w"][e], s["w_scales"][e] = _mx(randn(n, k) / math.sqrt(k))
    s["bias"] = 0.3 * randn(experts, n) if case["bias"] else None
    s["residual"] = packed(out).bfloat16() if case["residual"] else None
    if case["out"] == "mxfp4":
        s["y"] = torch.zeros(total, out // 2, dtype=torch.uint8, device=dev)
        s["y_scales"] = torch.zeros(total, out // 32, dtype=torch.uint8, device=dev)
    else:
        s["y"], s["y_scales"] = torch.zeros(total, out, dtype=torch.bfloat16, device=dev), None
    return s


def _inputs(case, seed):
    if case["op"].startswith("route"):
        return _route_inputs(case, seed)
    return (_quantize_inputs if case["op"] == "quantize" else _expert_inputs)(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    expert = case["op"] in ("glu", "linear")
    if expert:
        counts, offsets = s["counts"], s["offsets"]
        # the layout a plain program keeps beside its routing: the experts that
        # have rows, and their rows padded to the longest of them
        active = np.flatnonzero(counts)
        longest = int(counts.max()) if counts.size else 0
        place = np.arange(longest)[None, :]
        live = place < counts[active][:, None]
        s["active"] = torch.from_numpy(active).cuda()
        s["gather"] = torch.from_numpy(np.where(live, offsets[active][:, None] + place, 0)).cuda()
        s["live"] = torch.from_numpy(live[..., None].astype(np.float32)).cuda()
        s["where"] = torch.from_numpy(np.flatnonzero(live)).cuda()
    if own and case["op"] != "quantize":
        from combine_topk_ids_amd import moe
        c = case
        if expert:
            p = moe.problem(c["tokens"], c["hidden"], c["top_k"], c["experts"], 1, pad_multiple=c["pad"])
            plan = moe.alloc_plan(p)
            moe.moe_dispatch_plan(p, s["ids"], plan)
            k, n, out = _dims(c)
            s["plan"], s["layer"] = plan, moe.expert_op(k, out, act=c["act"], fmt=c["x"])
        else:
            p = moe.problem(c["tokens"], 8, c["top_k"], c["experts"], 1)
            s["router"] = moe.router(c["score"], logits=c["logits"], n_groups=c["groups"],
                                     top_groups=c["top_groups"], group_top=c["group_top"],
                                     renormalize=c["renormalize"], scale=c["scale"])
        s["p"] = p
    return s


# ---- one pass ---------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from combine_topk_ids_amd import moe
    op = s["case"]["op"]
    if op == "route":
        moe.moe_route(s["p"], s["router"], s["logits"], s["ids"], s["weights"], bias=s["bias"], scores=s["scores"])
    elif op == "route_backward":
        moe.moe_route_backward(s["p"], s["router"], s["logits"], s["ids"], s["dlogits"], dweights=s["dweights"],
                               dscores=s["dscores"])
    elif op == "quantize":
        moe.moe_quantize_mxfp4(s["x"], s["codes"], s["scales"])
    elif op == "glu":
        moe.moe_expert_glu_mx(s["p"], s["plan"], s["layer"], s["x"], s["x_scales"], s["w"], s["w_scales"], s["y"],
                              h_scales=s["y_scales"], bias=s["bias"])
    else:
        moe.moe_expert_linear_mx(s["p"], s["plan"], s["layer"], s["x"], s["x_scales"], s["w"], s["w_scales"], s["y"],
                                 bias=s["bias"], residual=s["residual"])
    return _results(s)


def _results(s):
    op = s["case"]["op"]
    if op == "quantize":
        # codes and scale bytes: whole numbers, which both sides have to give bit for bit
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "route":
        return {"ids": s["ids"], "weights": s["weights"]} | ({"scores": s["scores"]} if s["case"]["dense"] else {})
    if op == "route_backward":
        return {"dlogits": s["dlogits"]}
    if s["y_scales"] is not None:
        # the values that the 4-bit results stand for; E5M2 holds them exactly
        return {"h": _mx_value(s["y"], s["y_scales"]).to(torch.float8_e5m2)}
    return {"y": s["y"]}


def _scores(case, l):
    """Scores in l's type; a row without a finite logit has none."""
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _best(keys, count):
    """The `count` largest of each row, in order; ties go to the lowest index."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :count]


def _choose(case, logits, bias):
    """Top-k experts, in falling order of score + bias in 64 bits (without a bias: of
    the logits, which have the scores' order); -1 where none is left."""
    n, e = logits.shape
    l, groups = logits.double(), case["groups"]
    off = torch.full_like(l, -math.inf)
    off = torch.where(l == -math.inf, off, torch.zeros_like(l))
    biased = _scores(case, l) + (0 if bias is None else bias.double()) + off
    keys = l if bias is None else biased
    if groups > 1:
        of = (biased if case["group_top"] == 2 else keys).view(n, groups, -1)
        best = torch.sort(of, dim=2, descending=True).values[..., : case["group_top"]]
        total = best[..., 0]
        if best.shape[-1] == 2:  # a group's only expert counts alone
            total = total + torch.where(best[..., 1] == -math.inf, torch.zeros_like(total), best[..., 1])
        in_group = torch.zeros(n, groups, dtype=torch.bool, device=l.device)
        in_group.scatter_(1, _best(total, case["top_groups"]), True)
        keys = keys.masked_fill(~in_group.repeat_interleave(e // groups, dim=1), -math.inf)
    ids = _best(keys, case["top_k"])
    return torch.where(keys.gather(1, ids) == -math.inf, -1, ids).int()


def _gates(case, l, s, ids):
    """Gate weights before the factor `scale`."""
    live, at = ids >= 0, ids.clamp(min=0).long()
    if not case["renormalize"]:
        return torch.where(live, s.gather(1, at), 0.0)
    if case["score"] == "softmax":  # of the chosen ones alone
        v = l.gather(1, at).masked_fill(~live, -math.inf)
        top = v.amax(1, keepdim=True)
        v = torch.exp(v - torch.where(top == -math.inf, torch.zeros_like(top), top))
    else:
        v = torch.where(live, s.gather(1, at), 0.0)
    return v / v.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(s):
    case, l = s["case"], s["logits"].float()
    scores = _scores(case, l)
    ids = _choose(case, l, s["bias"])
    s["ids"].copy_(ids)
    s["weights"].copy_(_gates(case, l, scores, ids) * case["scale"])
    if case["dense"]:
        s["scores"].copy_(scores)


def _plain_route_backward(s):
    case, l, ids = s["case"], s["logits"].float(), s["ids"]
    scores = _scores(case, l)
    live, at = ids >= 0, ids.clamp(min=0).long()
    d = torch.where(live, s["dweights"], 0.0) * case["scale"]
    ds = torch.zeros_like(l) if s["dscores"] is None else s["dscores"].clone()
    dl = torch.zeros_like(l)
    if case["renormalize"]:
        w = _gates(case, l, scores, ids)
        d = w * (d - (d * w).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * (1 - scores.gather(1, at))
        dl.scatter_add_(1, at, torch.where(live, d, 0.0))
    else:
        ds.scatter_add_(1, at, d)
    if case["score"] == "sigmoid":
        dl += ds * scores * (1 - scores)
    else:
        dl += scores * (ds - (ds * scores).sum(1, keepdim=True))
    s["dlogits"].copy_(dl)


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    return z.clamp(min=0) if act == "relu" else z


def _plain_expert(s):
    c = s["case"]
    value = _fp8_value if c["x"] == "fp8" else _mx_value
    x = value(s["x"][s["gather"]], s["x_scales"][s["gather"]]) * s["live"]
    z = torch.bmm(x, _mx_value(s["w"][s["active"]], s["w_scales"][s["active"]]).transpose(1, 2))
    if s["bias"] is not None:
        z += s["bias"][s["active"]][:, None, :]
    if c["op"] == "glu":
        y = _act(z[..., : c["ffn"]], c["act"]) * z[..., c["ffn"]:]
    else:
        y = _act(z, c["act"])
    rows = y.reshape(-1, y.shape[-1]).index_select(0, s["where"])
    if s["residual"] is not None:
        rows = rows + s["residual"][s["rows"]].float()
    if c["out"] == "mxfp4":
        codes, scales = _mx(rows)
        s["y_scales"].index_copy_(0, s["rows"], scales)
        s["y"].index_copy_(0, s["rows"], codes)
    else:
        s["y"].index_copy_(0, s["rows"], rows.bfloat16())


def _plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        codes, scales = _mx(s["x"].float())
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
    else:
        {"route": _plain_route, "route_backward": _plain_route_backward}.get(op, _plain_expert)(s)
    return _results(s)


# ---- the definition, in 64 bits -----------------------------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        return None  # whole numbers
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "route_backward":
        return _exact_route_backward(case, s)
    return _exact_expert(case, s)


def _f64_scores(case, l):
    """numpy, a row of -inf gives zeros."""
    if case["score"] == "sigmoid":
        return 1 / (1 + np.exp(-l))
    top = np.max(l, axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total > 0, total, 1)


def _f64_gates(case, l, s, ids):
    rows = np.arange(len(ids))[:, None]
    v = np.where(ids >= 0, s[rows, ids], 0)
    if case["renormalize"]:
        total = v.sum(axis=1, keepdims=True)
        v = v / np.where(total > 0, total, 1)
    return v


def _exact_route(case, s):
    l = s["logits"].double().cpu().numpy()
    bias = 0.0 if s["bias"] is None else s["bias"].double().cpu().numpy()
    n, e = l.shape
    scores = _f64_scores(case, l)
    key = l if s["bias"] is None else np.where(l == -np.inf, -np.inf, scores + bias)
    each = e // case["groups"]
    if case["groups"] > 1:
        total = np.full((n, case["groups"]), -np.inf)
        for q in range(case["groups"]):
            span = slice(q * each, (q + 1) * each)
            if case["group_top"] == 1:
                total[:, q] = key[:, span].max(axis=1)
            else:
                of = np.sort(np.where(l == -np.inf, -np.inf, scores + bias)[:, span], axis=1)[:, ::-1]
                second = of[:, 1] if each > 1 else np.full(n, -np.inf)
                total[:, q] = of[:, 0] + np.where(second == -np.inf, 0, second)
        kept = np.zeros((n, case["groups"]), dtype=bool)
        np.put_along_axis(kept, np.argsort(-total, axis=1, kind="stable")[:, : case["top_groups"]], True, axis=1)
        key = np.where(np.repeat(kept, each, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, : case["top_k"]]
    ids = np.where(np.take_along_axis(key, ids, axis=1) == -np.inf, -1, ids)
    out = {"ids": ids.astype(np.int32), "weights": _f64_gates(case, l, scores, ids) * case["scale"]}
    return out | ({"scores": scores} if case["dense"] else {})


def _exact_route_backward(case, s):
    l, ids = s["logits"].double().cpu().numpy(), s["ids"].cpu().numpy()
    n, e = l.shape
    scores = _f64_scores(case, l)
    dw = np.where(ids >= 0, s["dweights"].double().cpu().numpy(), 0) * case["scale"]
    da = dw
    if case["renormalize"]:
        total = np.where(ids >= 0, scores[np.arange(n)[:, None], ids], 0).sum(axis=1, keepdims=True)
        w = _f64_gates(case, l, scores, ids)
        da = (dw - (dw * w).sum(axis=1, keepdims=True)) / np.where(total > 0, total, 1)
    ds = np.zeros((n, e)) if s["dscores"] is None else s["dscores"].double().cpu().numpy().copy()
    for j in range(case["top_k"]):
        t = np.flatnonzero(ids[:, j] >= 0)
        ds[t, ids[t, j]] += da[t, j]
    if case["score"] == "sigmoid":
        return {"dlogits": ds * scores * (1 - scores)}
    return {"dlogits": scores * (ds - (ds * scores).sum(axis=1, keepdims=True))}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _f64_mx(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    v[:, 0::2], v[:, 1::2] = table[(codes % 16).int()], table[(codes // 16).int()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def _f64_quantised(v):
    """Values rounded to MX-FP4: to the nearest of the sixteen, ties to an even code."""
    if not v.numel():
        return v
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2, 0.0))
    a = (b / unit).abs()
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=v.device)
    high = torch.searchsorted(grid, a.clamp(max=6)).clamp(1, 7)
    low, middle = high - 1, (grid[high] + grid[high - 1]) / 2
    pick = torch.where((a > middle) | ((a == middle) & (high % 2 == 0)), high, low)
    return (torch.where(b < 0, -grid[pick], grid[pick]) * unit).reshape(v.shape)


def _f64_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        # (1 + tanh a) / 2 = 1 / (1 + exp(-2a))
        return z / (1 + torch.exp(-2 * GELU_C * (z + 0.044715 * z ** 3)))
    return torch.relu(z) if act == "relu" else z


def _exact_expert(case, s):
    out = torch.zeros(s["total"], _dims(case)[2], dtype=torch.float64, device="cuda")
    for e in np.flatnonzero(s["counts"]):
        r = slice(int(s["offsets"][e]), int(s["offsets"][e] + s["counts"][e]))
        if case["x"] == "fp8":
            x = s["x"][r].view(torch.float8_e4m3fn).to(torch.float32).double()
            x = x * torch.kron(s["x_scales"][r].double(), torch.ones(1, 128, dtype=torch.float64, device="cuda"))
        else:
            x = _f64_mx(s["x"][r], s["x_scales"][r])
        z = x @ _f64_mx(s["w"][e], s["w_scales"][e]).T
        if case["bias"]:
            z += s["bias"][e].double()
        if case["op"] == "glu":
            y = _f64_act(z[:, : case["ffn"]], case["act"]) * z[:, case["ffn"]:]
        else:
            y = _f64_act(z, case["act"])
            if case["residual"]:
                y = y + s["residual"][r].double()
        out[r] = _f64_quantised(y) if case["out"] == "mxfp4" else y
    return {"h" if case["out"] == "mxfp4" else "y": out}
