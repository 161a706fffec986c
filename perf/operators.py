"""The experts' operators, as cases to measure: the gated feed-forward block and
the linear layer over the packed expert-major rows, their backward passes, and
the backward pass of the combine.

``own = False`` computes a case in plain torch operations (one batched product
over the experts that have rows, padded to the longest expert, in 32 bits,
rounded once at the end); ``own = True`` calls libmoe.  Rows that hold no token
(pad rows and rows past the last one in use) are not part of any result: both
sides leave them as prepare() made them.
"""
import math

import numpy as np
import torch

own = False

ACT = ("none", "silu", "gelu_tanh", "relu")
GELU_C = math.sqrt(2.0 / math.pi)


def _case(name, op, tokens, hidden, ffn, experts, top_k, **more):
    c = dict(op=op, tokens=tokens, hidden=hidden, ffn=ffn, experts=experts, top_k=top_k, pad=1,
             fmt="bf16", act="silu" if op.startswith("glu") else "none", bias=False,
             residual=False, save=False, skew=0.0, masked=0.0)
    c.update(more)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token of a chat: six experts' weights are read, nothing else counts
        _case("glu_one_token", "glu", 1, 4096, 1024, 64, 6),
        # a decode batch over FP8 weights: every expert is active with a few rows
        _case("glu_decode_fp8", "glu", 128, 7168, 2048, 256, 8, fmt="fp8"),
        # a prompt's first products, 128-row expert alignment
        _case("glu_prefill", "glu", 4096, 4096, 2048, 64, 6, pad=128),
        # a long prefill from FP8 rows and weights: the largest case
        _case("glu_prefill_fp8", "glu", 8192, 7168, 2048, 256, 8, fmt="fp8"),
        # a training step's gradients of the gated block
        _case("glu_backward", "glu_backward", 4096, 4096, 1024, 64, 6),
        # a small fine-tuning batch with odd sizes, biases and masked pairs
        _case("glu_backward_odd", "glu_backward", 333, 520, 712, 12, 3, act="gelu_tanh", bias=True,
              skew=1.0, masked=0.1),
        # a decode batch's down projection
        _case("linear_decode", "linear", 128, 4096, 2048, 64, 6),
        # a prompt's down projection with bias and residual rows in the epilogue
        _case("linear_prefill", "linear", 4096, 4096, 2048, 64, 6, pad=128, bias=True, residual=True),
        # a skewed, ragged prompt through FP8 rows
        _case("linear_ragged_fp8", "linear", 1501, 7168, 2048, 32, 4, fmt="fp8", skew=1.0, masked=0.05),
        # a training step's gradients of the down projection
        _case("linear_backward", "linear_backward", 4096, 4096, 1024, 64, 6, skew=0.5),
        # the combine's gradients: a small batch, and a long one with wide rows
        _case("combine_backward_small", "combine_backward", 128, 4096, 8, 64, 6),
        _case("combine_backward_large", "combine_backward", 8192, 7168, 8, 256, 8, masked=0.02),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


MOST_FLOPS, MOST_WEIGHTS = 3.0e12, 3.0e9  # of a drawn case: below the largest listed one


def draw(rng):
    while True:
        op = rng.choice(("glu", "glu", "glu_backward", "linear", "linear", "linear_backward", "combine_backward"))
        backward = op.endswith("backward")
        fmt = rng.choice(("bf16", "fp8")) if not backward else "bf16"
        step = 128 if fmt == "fp8" else 8
        hidden, ffn = step * _log(rng, max(1, 64 // step), 7168 // step), step * _log(rng, max(1, 64 // step), 2048 // step)
        experts = _log(rng, 1, 256)
        c = _case(None, op, _log(rng, 1, 16384), hidden, ffn, experts, rng.randint(1, min(8, experts)),
                  pad=rng.choice((1, 1, 16, 128)), fmt=fmt, skew=rng.choice((0.0, 0.0, 0.5, 1.0)),
                  masked=rng.choice((0.0, 0.0, 0.1, 0.5)))
        if op.startswith("glu"):
            c["act"] = rng.choice(ACT[1:])
        elif op.startswith("linear"):
            c["act"] = rng.choice(ACT)
            c["residual"] = not backward and rng.random() < 0.5
        if op != "combine_backward":
            c["bias"] = rng.random() < 0.5
            c["save"] = not backward and rng.random() < 0.3 and (op == "glu" or c["act"] != "none")
        # padded to the longest expert, the plain form does more than the operator
        longest = min(c["tokens"], 1 + int(c["tokens"] * c["top_k"] / experts * (1 + 3 * c["skew"])))
        sizes = experts * ffn * hidden * (2 if op.startswith("glu") else 1)
        if 2 * longest * sizes * (2 if backward else 1) < MOST_FLOPS and sizes < MOST_WEIGHTS:
            return c


def _dims(case):
    """(columns of the weights, rows of the weights) of one expert."""
    if case["op"].startswith("glu"):
        return case["hidden"], 2 * case["ffn"]
    return case["ffn"], case["hidden"]


def work(case):
    pairs = case["tokens"] * case["top_k"] * (1 - case["masked"])
    active = case["experts"] * (1 - (1 - 1 / case["experts"]) ** pairs)
    k, n = _dims(case)
    op = case["op"]
    if op == "combine_backward":
        return {"bytes": 2 * case["hidden"] * (2 * pairs + case["tokens"]) + 12 * pairs, "flops": 3 * pairs * case["hidden"]}
    out = case["ffn"] if op.startswith("glu") else case["hidden"]
    size = 1 if case["fmt"] == "fp8" else 2
    if not op.endswith("backward"):
        rows = pairs * (size * k + 2 * out * (2 if case["residual"] else 1) + (2 * n if case["save"] else 0))
        return {"bytes": rows + size * active * k * n, "flops": 2 * pairs * k * n}
    # read: the rows, their gradients, what the forward pass kept, the weights;
    # written: the rows' gradients and the weights'
    kept = 2 * n if op == "glu_backward" else n if case["act"] != "none" else 0
    rows = pairs * 2 * (2 * k + out + kept + (n if kept else 0))
    return {"bytes": rows + 2 * active * k * n + 2 * case["experts"] * k * n, "flops": 4 * pairs * k * n}


# ---- inputs ---------------------------------------------------------------------


def _fp8_rows(x):
    """Codes and scales of 1x128 blocks: scale = amax / 448."""
    blocks = x.view(x.shape[0], -1, 128)
    scale = blocks.abs().amax(-1) / 448.0
    codes = (blocks / scale.clamp(min=1e-30)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(x.shape).view(torch.uint8), scale


def _inputs(case, seed):
    """Everything the case's operator takes, in plain tensors."""
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    tokens, experts, top_k, pad = case["tokens"], case["experts"], case["top_k"], case["pad"]
    logits = randn(tokens, experts) + case["skew"] * randn(experts)
    ids = logits.topk(top_k, dim=1).indices.int()
    if case["masked"]:
        ids[torch.rand(tokens, top_k, generator=g, device=dev) < case["masked"]] = -1
    flat = ids.cpu().numpy().reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // pad) * pad)])
    total = tokens * top_k + experts * (pad - 1)
    slot = np.full(flat.size, -1, dtype=np.int64)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable")[: int(counts.sum())]
    rank = np.arange(order.size) - np.repeat(np.cumsum(counts) - counts, counts)
    slot[order] = offsets[flat[order]] + rank
    rows = np.sort(slot[slot >= 0])  # the packed rows that hold a token
    s = {"case": case, "ids": ids, "counts": counts, "offsets": offsets, "total": total,
         "slot": torch.from_numpy(slot.reshape(tokens, top_k)).to(dev), "rows": torch.from_numpy(rows).to(dev)}

    def packed(cols, dtype=torch.bfloat16):
        """Rows of a packed buffer: values where a token is, zeros elsewhere."""
        out = torch.zeros(total, cols, dtype=dtype, device=dev)
        out[s["rows"]] = randn(rows.size, cols).to(dtype)
        return out

    op, hidden = case["op"], case["hidden"]
    if op == "combine_backward":
        s["weights"] = torch.softmax(randn(tokens, top_k), dim=1)
        s["expert_out"] = packed(hidden)
        s["dout"] = randn(tokens, hidden).bfloat16()
        s["dy"] = torch.zeros(total, hidden, dtype=torch.bfloat16, device=dev)
        s["dweights"] = torch.zeros(tokens, top_k, device=dev)
        return s
    k, n = _dims(case)
    out = case["ffn"] if op.startswith("glu") else hidden
    if case["fmt"] == "fp8":
        s["x"], s["x_scales"] = _fp8_rows(packed(k, torch.float32))
        s["w"] = torch.empty(experts, n, k, dtype=torch.uint8, device=dev)
        for e in range(experts):  # one expert at a time: little memory
            s["w"][e] = (100 * randn(n, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["w_scales"] = (0.5 + torch.rand(experts, n // 128, k // 128, generator=g, device=dev)) / (100 * math.sqrt(k))
    else:
        s["x"], s["x_scales"], s["w_scales"] = packed(k), None, None
        s["w"] = torch.empty(experts, n, k, dtype=torch.bfloat16, device=dev)
        for e in range(experts):
            s["w"][e] = randn(n, k) / math.sqrt(k)
    s["bias"] = 0.3 * randn(experts, n) if case["bias"] else None
    if not op.endswith("backward"):
        s["residual"] = packed(out) if case["residual"] else None
        s["y"] = torch.zeros(total, out, dtype=torch.bfloat16, device=dev)
        s["preact"] = torch.zeros(total, n, dtype=torch.bfloat16, device=dev) if case["save"] else None
        return s
    s["dy"] = packed(out)
    kept = op == "glu_backward" or case["act"] != "none"
    s["preact"] = packed(n) if kept else None  # what the forward pass kept
    s["dz"] = torch.zeros(total, n, dtype=torch.bfloat16, device=dev) if kept else None
    s["dx"] = torch.zeros(total, k, dtype=torch.bfloat16, device=dev)
    s["dw"] = torch.zeros(experts, n, k, dtype=torch.bfloat16, device=dev)
    s["dbias"] = torch.zeros(experts, n, device=dev) if case["bias"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    counts, offsets, dev = s["counts"], s["offsets"], "cuda"
    # the layout a plain program keeps beside its routing: the experts that
    # have rows, and their rows padded to the longest of them
    active = np.flatnonzero(counts)
    longest = int(counts.max()) if counts.size else 0
    place = np.arange(longest)[None, :]
    live = place < counts[active][:, None]
    s["active"] = torch.from_numpy(active).to(dev)
    s["gather"] = torch.from_numpy(np.where(live, offsets[active][:, None] + place, 0)).to(dev)
    s["live"] = torch.from_numpy(live[..., None].astype(np.float32)).to(dev)
    s["where"] = torch.from_numpy(np.flatnonzero(live)).to(dev)
    if own:
        from combine_topk_ids_amd import moe
        c = s["case"]
        p = moe.problem(c["tokens"], c["hidden"], c["top_k"], c["experts"], 1, pad_multiple=c["pad"], fmt=c["fmt"])
        plan = moe.alloc_plan(p)
        moe.moe_dispatch_plan(p, s["ids"], plan)
        s["p"], s["plan"] = p, plan
        if c["op"] != "combine_backward":
            k, n = _dims(c)
            glu = c["op"].startswith("glu")
            s["layer"] = moe.expert_op(k, c["ffn"] if glu else n, act=c["act"], fmt=c["fmt"])
            if c["op"].endswith("backward"):
                s["workspace"] = moe.alloc_expert_workspace(p, s["layer"])
    return s


# ---- one pass -------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from combine_topk_ids_amd import moe
    c, p, plan = s["case"], s["p"], s["plan"]
    op = c["op"]
    if op == "combine_backward":
        moe.moe_combine_backward(p, plan, s["expert_out"], s["weights"], s["dout"], s["dy"], s["dweights"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    layer = s["layer"]
    if op == "glu":
        moe.moe_expert_glu(p, plan, layer, s["x"], s["w"], s["y"], x_scales=s["x_scales"],
                           w_scales=s["w_scales"], bias=s["bias"], preact=s["preact"])
    elif op == "linear":
        moe.moe_expert_linear(p, plan, layer, s["x"], s["w"], s["y"], x_scales=s["x_scales"],
                              w_scales=s["w_scales"], bias=s["bias"], residual=s["residual"],
                              preact=s["preact"])
    elif op == "glu_backward":
        moe.moe_expert_glu_backward(p, plan, layer, s["dy"], s["preact"], s["x"], s["w"], s["dz"],
                                    s["dx"], s["dw"], dbias=s["dbias"], workspace=s["workspace"])
    else:
        moe.moe_expert_linear_backward(p, plan, layer, s["dy"], s["x"], s["w"], s["dx"], s["dw"],
                                       preact=s["preact"], dz=s["dz"], dbias=s["dbias"],
                                       workspace=s["workspace"])
    return _results(s)


def _results(s):
    if s["case"]["op"].endswith("backward"):
        names = ("dx", "dw", "dz", "dbias")
    else:
        names = ("y", "preact")
    return {name: s[name] for name in names if s[name] is not None}


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    return z.clamp(min=0) if act == "relu" else z


def _act_slope(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z)
    return (z > 0).to(z.dtype) if act == "relu" else torch.ones_like(z)


def _dense(s, name):
    """Rows [total, C] -> [active experts, longest, C] in 32 bits."""
    return s[name][s["gather"]].float() * s["live"]


def _packed(s, v, name):
    """[active experts, longest, C] -> the packed rows, rounded to the result's type."""
    rows = v.reshape(-1, v.shape[-1]).index_select(0, s["where"])
    s[name].index_copy_(0, s["rows"], rows.to(s[name].dtype))


def _wide(v, like):
    """A 1x128 (or 128x128) block's scale for each of its values."""
    v = v.repeat_interleave(128, dim=-1)
    return v if v.shape[-2] == like.shape[-2] else v.repeat_interleave(128, dim=-2)


def _plain(s):
    c = s["case"]
    op, act = c["op"], c["act"]
    if op == "combine_backward":
        held = s["slot"].clamp(min=0)
        live = (s["slot"] >= 0).float()
        dout = s["dout"].float()
        s["dweights"].copy_((s["expert_out"][held].float() * dout[:, None, :]).sum(-1) * live)
        rows = (s["weights"][..., None] * dout[:, None, :]).bfloat16()
        # masked pairs go to a row behind the last, which is cut off
        to = torch.where(s["slot"] >= 0, s["slot"], s["total"]).reshape(-1)
        dy = torch.zeros(s["total"] + 1, c["hidden"], dtype=torch.bfloat16, device="cuda")
        dy.index_copy_(0, to, rows.view(-1, c["hidden"]))
        return {"dy": dy[:-1], "dweights": s["dweights"]}
    if c["fmt"] == "fp8":
        x = s["x"][s["gather"]].view(torch.float8_e4m3fn).float() * s["live"]
        x *= s["x_scales"][s["gather"]].repeat_interleave(128, dim=-1)
        w = s["w"][s["active"]].view(torch.float8_e4m3fn).float()
        w *= _wide(s["w_scales"][s["active"]], w)
    else:
        x, w = _dense(s, "x"), s["w"][s["active"]].float()
    if not op.endswith("backward"):
        z = torch.bmm(x, w.transpose(1, 2))
        if s["bias"] is not None:
            z += s["bias"][s["active"]][:, None, :]
        if s["preact"] is not None:
            _packed(s, z, "preact")
        if op == "glu":
            y = _act(z[..., : c["ffn"]], act) * z[..., c["ffn"]:]
        else:
            y = _act(z, act)
            if s["residual"] is not None:
                y = y + _dense(s, "residual")
        _packed(s, y, "y")
        return _results(s)
    dz = _dense(s, "dy")
    if op == "glu_backward":
        z = _dense(s, "preact")
        gate, up = z[..., : c["ffn"]], z[..., c["ffn"]:]
        dz = torch.cat([dz * up * _act_slope(gate, act), dz * _act(gate, act)], dim=-1)
    elif act != "none":
        dz = dz * _act_slope(_dense(s, "preact"), act)
    if s["dz"] is not None:
        _packed(s, dz, "dz")
    _packed(s, torch.bmm(dz, w), "dx")
    dw = torch.bmm(dz.transpose(1, 2), x)
    s["dw"].zero_()
    s["dw"].index_copy_(0, s["active"], dw.to(s["dw"].dtype))
    if s["dbias"] is not None:
        s["dbias"].zero_()
        s["dbias"].index_copy_(0, s["active"], dz.sum(1))
    return _results(s)


# ---- the definition, in 64 bits, expert by expert ---------------------------------


def exact(case, seed):
    s = _inputs(case, seed)
    op, act, f64 = case["op"], case["act"], torch.float64
    total, dev = s["total"], "cuda"
    if op == "combine_backward":
        dy = torch.zeros(total, case["hidden"], dtype=f64, device=dev)
        dweights = torch.zeros(case["tokens"], case["top_k"], dtype=f64, device=dev)
        for j in range(case["top_k"]):
            t = torch.nonzero(s["slot"][:, j] >= 0).flatten()
            r, d = s["slot"][t, j], s["dout"][t].double()
            dy[r] = s["weights"][t, j].double()[:, None] * d
            dweights[t, j] = (s["expert_out"][r].double() * d).sum(1)
        return {"dy": dy, "dweights": dweights}
    out = {name: torch.zeros(v.shape, dtype=f64, device=dev) for name, v in _results(s).items()}
    for e in np.flatnonzero(s["counts"]):
        r = slice(int(s["offsets"][e]), int(s["offsets"][e] + s["counts"][e]))
        if case["fmt"] == "fp8":
            x = s["x"][r].view(torch.float8_e4m3fn).to(torch.float32).double()
            w = s["w"][e].view(torch.float8_e4m3fn).to(torch.float32).double()
            x = x * torch.kron(s["x_scales"][r].double(), torch.ones(1, 128, dtype=f64, device=dev))
            w = w * torch.kron(s["w_scales"][e].double(), torch.ones(128, 128, dtype=f64, device=dev))
        else:
            x, w = s["x"][r].double(), s["w"][e].double()
        if not op.endswith("backward"):
            z = x @ w.T
            if case["bias"]:
                z += s["bias"][e].double()
            if case["save"]:
                out["preact"][r] = z
            if op == "glu":
                y = _f64_act(z[:, : case["ffn"]], act)[0] * z[:, case["ffn"]:]
            else:
                y = _f64_act(z, act)[0]
                if case["residual"]:
                    y = y + s["residual"][r].double()
            out["y"][r] = y
            continue
        d = s["dy"][r].double()
        if op == "glu_backward":
            gate, up = s["preact"][r].double().split(case["ffn"], dim=1)
            value, slope = _f64_act(gate, act)
            d = torch.cat([d * up * slope, d * value], dim=1)
        elif act != "none":
            d = d * _f64_act(s["preact"][r].double(), act)[1]
        if s["dz"] is not None:
            out["dz"][r] = d
        out["dx"][r] = d @ w
        out["dw"][e] = d.T @ x
        if case["bias"]:
            out["dbias"][e] = d.sum(0)
    return out


def _f64_act(z, act):
    """(value, slope) of an activation."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s + z * s * (1 - s)
    if act == "gelu_tanh":
        # (1 + tanh a) / 2 = 1 / (1 + exp(-2a))
        a = GELU_C * (z + 0.044715 * z ** 3)
        s = 1 / (1 + torch.exp(-2 * a))
        return z * s, s + z * 2 * s * (1 - s) * GELU_C * (1 + 0.134145 * z * z)
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    return z, torch.ones_like(z)
