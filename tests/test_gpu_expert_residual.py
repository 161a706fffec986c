"""GPU: the linear layer's residual, in every tile that its launch rule picks
(the case's comment names it), bf16 and FP8: beside the activation and the bias, with
and without the kept pre-activation, and in place.  Against 64 bits, with the
bounds of expert_reference.py."""
import pytest
import torch

import expert_reference as ref
from expert_reference import assert_within
from gpu_helpers import say
from test_gpu_expert import Routed, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


BF16 = [
    dict(tokens=9, experts=4, top_k=2, k=72, f=136, act="silu"),                                 # 16 x 64
    dict(tokens=100, experts=3, top_k=2, k=200, f=264, act="relu", bias=True, masked=0.1),       # 64 x 128
    dict(tokens=1100, experts=64, top_k=6, k=136, f=328, act="none", bias=True, pad=16),         # 128 x 128
    dict(tokens=2000, experts=8, top_k=2, k=136, f=1552, act="gelu_tanh", bias=True, skew=0.3),  # 256 x 256
    dict(tokens=1031, experts=4, top_k=2, k=264, f=2568, act="none", masked=0.05, pad=7),        # 256 x 256
    dict(tokens=21, experts=3, top_k=2, k=2120, f=200, act="silu", bias=True),                   # K in four
]
FP8 = [
    dict(tokens=9, experts=4, top_k=2, k=256, f=256, act="silu"),                                # 16 x 64
    dict(tokens=100, experts=3, top_k=2, k=384, f=384, act="none", bias=True, masked=0.1),       # 64 x 128
    dict(tokens=300, experts=64, top_k=6, k=384, f=256, act="relu", pad=16, bias=True),          # 128 x 128, tile after tile
    dict(tokens=3000, experts=4, top_k=1, k=256, f=768, act="gelu_tanh", bias=True, skew=0.5),   # 128 x 128, one each
    dict(tokens=3, experts=2, top_k=2, k=2048, f=256, act="silu", bias=True),                    # K in four
    dict(tokens=200, experts=40, top_k=2, k=2176, f=384, act="none", masked=0.1),                # K in four, many tiles
]


@pytest.mark.parametrize("fmt,i", [("bf16", i) for i in range(len(BF16))] + [("fp8", i) for i in range(len(FP8))])
def test_residual(moe, fmt, i):
    c = (BF16 if fmt == "bf16" else FP8)[i]
    say(f"[expert residual] {fmt} {c}")
    r = Routed(moe, 600 + i, **{k: c[k] for k in ("tokens", "experts", "top_k", "pad", "masked", "skew") if k in c})
    k, f, name = c["k"], c["f"], c["act"]
    more = {}
    if fmt == "bf16":
        x, w = r.packed(k), weights(r, f, k)
        x64, w64 = (lambda a, b: x[a:b].double()), (lambda e: w[e].double())
    else:
        x = (100 * r.randn(r.rows, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        w = (100 * r.randn(r.experts, f, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        xs = torch.rand(r.rows, k // 128, generator=r.g, device="cuda") / 100
        ws = (0.2 + torch.rand(r.experts, f // 128, k // 128, generator=r.g, device="cuda")) / (100 * k ** 0.5)
        x[~r.live] = 0x7F  # NaN codes
        xs[~r.live] = float("nan")
        more = dict(x_scales=xs, w_scales=ws)
        x64, w64 = (lambda a, b: ref.dequant_rows(x[a:b], xs[a:b])), (lambda e: ref.dequant_weights(w[e], ws[e]))
    bias = r.randn(r.experts, f) if c.get("bias") else None
    residual = r.packed(f, 3.0)
    op = moe.expert_op(k, f, act=name, fmt=fmt)
    y, z = r.sentinel(f), r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, op, x, w, y, bias=bias, residual=residual, preact=z, **more)
    torch.cuda.synchronize()
    r.check_rest(y, "y")
    r.check_rest(z, "preact")
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        rz, ry, tz, ty = ref.forward(x64(a, b), w64(e), None if bias is None else bias[e].double(), False, name,
                                     residual[a:b].double())
        assert_within(z[a:b], rz, tz, f"preact of expert {e}")
        assert_within(y[a:b], ry, ty, f"y of expert {e}")
    # without the kept pre-activation, and with y in the residual's place: the same bits
    alone = r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, op, x, w, alone, bias=bias, residual=residual, **more)
    assert torch.equal(alone.view(torch.int16), y.view(torch.int16))
    for kept in (None, r.sentinel(f)):
        same = residual.clone()
        moe.moe_expert_linear(r.p, r.plan, op, x, w, same, bias=bias, residual=same, preact=kept, **more)
        torch.cuda.synchronize()
        assert torch.equal(same[r.live].view(torch.int16), y[r.live].view(torch.int16))
        assert bool(torch.isnan(same[~r.live]).all()), "a row without a token was written"
        if kept is not None:
            assert torch.equal(kept.view(torch.int16), z.view(torch.int16))
