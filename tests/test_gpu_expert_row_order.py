"""GPU: within one problem and one layer, a row's results are its own: the same
bits wherever the routing places the row and whatever the other rows are (the
kernels choose their tiles by the problem and the layer alone).  Forward, and the
gradients of the rows."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_expert import Routed, weights

pytestmark = pytest.mark.gpu

# 16 x 64, 64 x 128, 128 x 128 and 256 x 256 tiles, and K in four
SIZES = [dict(tokens=7, experts=3, top_k=2, k=72, f=136), dict(tokens=150, experts=3, top_k=2, k=200, f=264),
         dict(tokens=1100, experts=64, top_k=6, k=136, f=264), dict(tokens=2000, experts=8, top_k=2, k=136, f=1552),
         dict(tokens=60, experts=5, top_k=2, k=2120, f=136)]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_rows_do_not_depend_on_each_other(moe, i, fmt):
    c = SIZES[i]
    say(f"[expert row order] {fmt} {c}")
    if fmt == "fp8":
        c = dict(c, k=-(-c["k"] // 128) * 128, f=-(-c["f"] // 128) * 128)
    r = Routed(moe, 1000 + i, c["tokens"], c["experts"], c["top_k"], masked=0.1)
    n, k, f, e = c["tokens"], c["k"], c["f"], c["experts"]
    p, tokens, grads = r.p, r.randn(n, k), r.randn(n, f).bfloat16()
    w1, w2 = weights(r, 2 * f, k), weights(r, f, k)
    b1, b2 = r.randn(e, 2 * f), r.randn(e, f)
    if fmt == "fp8":
        def quant(t):
            return (16 * t).to(torch.float8_e4m3fn).view(torch.uint8)
        tokens = quant(tokens)
        tok_scales = torch.rand(n, k // 128, generator=r.g, device="cuda") / 16
        w1, w2 = quant(k ** 0.5 * w1), quant(k ** 0.5 * w2)
        s1, s2 = (torch.rand(e, m // 128, k // 128, generator=r.g, device="cuda") / (16 * k ** 0.5) for m in (2 * f, f))
    else:
        tokens = tokens.bfloat16()
    glu, lin = moe.expert_op(k, f, "silu", fmt), moe.expert_op(k, f, "gelu_tanh", fmt)

    def run(ids, order):
        """Results of each (token, choice) of `order`, in that order's places."""
        plan = moe.alloc_plan(p)
        moe.moe_dispatch_plan(p, ids[order].contiguous(), plan)
        slot = plan.slot.long()
        live = slot >= 0
        src = torch.full((r.rows,), -1, dtype=torch.long, device="cuda")
        src[slot[live]] = order[:, None].expand_as(slot)[live]

        def rows(t):
            v = t[src.clamp(min=0)].clone()
            v[src < 0] = 0
            return v

        x, d = rows(tokens), rows(grads)
        more1 = dict(x_scales=rows(tok_scales), w_scales=s1) if fmt == "fp8" else {}
        more2 = dict(more1, w_scales=s2) if fmt == "fp8" else {}
        h, pre, y = r.sentinel(f), r.sentinel(2 * f), r.sentinel(f)
        moe.moe_expert_glu(p, plan, glu, x, w1, h, bias=b1, preact=pre, **more1)
        moe.moe_expert_linear(p, plan, lin, x, w2, y, bias=b2, residual=d, **more2)
        out = {"h": h, "z": pre, "y": y}
        if fmt == "bf16":
            dz, dx = r.sentinel(2 * f), r.sentinel(k)
            moe.moe_expert_glu_backward(p, plan, glu, d, pre, None, w1, dz, dx, None)
            out.update(dz=dz, dx=dx)
        torch.cuda.synchronize()
        back = {}
        for name, v in out.items():
            t = v.new_zeros(n, c["top_k"], v.shape[1])
            t[order] = torch.where(live[..., None], v[slot.clamp(min=0)], 0.0)
            back[name] = t
        return back

    straight = torch.arange(n, device="cuda")
    first = run(r.ids, straight)
    shuffled = run(r.ids, torch.randperm(n, generator=r.g, device="cuda"))
    for name, v in first.items():
        assert torch.equal(bits(shuffled[name]), bits(v)), f"{name}: other places"
    # half of the tokens go elsewhere: all to one expert, which then has far more rows
    other = r.ids.clone()
    other[n // 2:] = -1
    other[n // 2:, 0] = 1
    moved = run(other, straight)
    for name, v in first.items():
        assert torch.equal(bits(moved[name][:n // 2]), bits(v[:n // 2])), f"{name}: other rows"
