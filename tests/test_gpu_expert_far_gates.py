"""GPU: the activations and their slopes far from zero, where exp leaves the range
of fp32 and the sigmoid becomes 0 or 1 (and the tanh form's slope takes its own branch),
in the gated block, the linear layer and both backward passes.

Bounds (u = 2^-23).  s = 1 / (1 + exp(-t)), t = z (SiLU) or 1.5957 (z + 0.0447 z^3).
t carries at most 8 roundings, so exp(-t) is off by at most 9 |t| u relative to it,
and s by d = (9 |t| + 16) u with the sum, the reciprocal and the products around it;
past |t| = 128 s is 0 or 1 exactly.  A sigmoid below 2^-126 may be flushed
to zero.  1 - s, for t > 0, is off by at most 2^-22 + d e with e = exp(-t), and by at most
e once 1 + e is 1 (t > 18)."""
import math

import pytest
import torch

from expert_reference import BF16, assert_within
from gpu_helpers import say
from test_gpu_expert import Routed

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -23, 2.0 ** -126
C2 = 2 * math.sqrt(2 / math.pi)


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


def act_and_slope(z, name):
    """(value, its bound, slope, its bound) in 64 bits."""
    if name == "relu":
        zero = torch.zeros_like(z)
        return z.clamp(min=0), zero, (z > 0).double(), zero
    t, dt = (z, torch.ones_like(z)) if name == "silu" else (C2 * (z + 0.044715 * z ** 3), C2 * (1 + 0.134145 * z * z))
    e = torch.exp(-t)
    s = 1 / (1 + e)
    d = (9 * t.abs().clamp(max=128) + 16) * U
    value, value_tol = z * s, d * (z * s).abs() + z.abs() * TINY
    # slope = s + z t' s (1 - s); past the ends s (1 - s) is 0, whatever z t' is
    weight = torch.where(t.abs() > 1000, 0.0, z * dt)
    rest = torch.where(t > 0, e / (1 + e), 1 - s)
    off = torch.where(t > 18, e, torch.where(t > 0, 2.0 ** -22 + d * e, 0.0))
    slope = s + weight * s * rest
    tol = 2 * d * (s + (weight * s * rest).abs()) + weight.abs() * off + TINY * (1 + weight.abs())
    return value, value_tol, slope, tol


def gates():
    near = torch.arange(-1024, 1025) / 8.0  # -128 .. 128, exact in bf16 up to 32 and rounded beyond
    edge = torch.tensor([15.875, 16.0, 16.125, 86.5, 87.0, 87.5, 88.0, 88.5, 89.0, 104.0, 500.0, 1e3, 1e4, 1e10, 1e15, 1e30])
    z = torch.cat([near, edge, -edge, torch.tensor([0.0, -0.0])]).bfloat16()
    return torch.cat([z, z.new_zeros(-z.numel() % 8)])


@pytest.mark.parametrize("name", ["silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("fmt,rows", [("bf16", 5), ("bf16", 200), ("fp8", 5), ("fp8", 200)])
def test_forward(moe, name, fmt, rows):
    """Weights of zero: z is the bias, to the bit."""
    say(f"[expert far gates] forward {name} {fmt} {rows} rows")
    z = gates()
    z = torch.cat([z, z.new_zeros(-z.numel() % 128)]).cuda().float()
    k, f, fp8 = 128, z.numel(), fmt == "fp8"
    r = Routed(moe, 800, rows, 2, 1)
    up = 1.0 + torch.rand(f, generator=r.g, device="cuda")
    kind = torch.uint8 if fp8 else torch.bfloat16
    x = torch.ones(r.rows, k, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else torch.ones(r.rows, k, dtype=kind, device="cuda")

    def scales(n):
        return dict(x_scales=torch.ones(r.rows, k // 128, device="cuda"),
                    w_scales=torch.ones(2, n // 128, k // 128, device="cuda")) if fp8 else {}

    value, tol, _, _ = act_and_slope(z.double(), name)
    y, kept = r.sentinel(f), r.sentinel(2 * f)
    moe.moe_expert_glu(r.p, r.plan, moe.expert_op(k, f, name, fmt), x, torch.zeros(2, 2 * f, k, dtype=kind, device="cuda"),
                       y, bias=torch.cat([z, up]).repeat(2, 1).contiguous(), preact=kept, **scales(2 * f))
    lin = r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, moe.expert_op(k, f, name, fmt), x, torch.zeros(2, f, k, dtype=kind, device="cuda"),
                          lin, bias=z.repeat(2, 1).contiguous(), **scales(f))
    torch.cuda.synchronize()
    assert torch.equal(kept[:, :f].float(), z.expand(rows, f))
    for got, want, t, what in ((y, value * up.double(), tol * up.double() + U * (value * up.double()).abs(), "h"),
                               (lin, value, tol, "y")):
        bound = t + BF16 * (want.abs() + t)
        assert_within(got, want.expand(rows, f), bound.expand(rows, f), f"{what} of {name}")


@pytest.mark.parametrize("name", ["silu", "gelu_tanh", "relu"])
def test_backward(moe, name):
    say(f"[expert far gates] backward {name}")
    z = gates().cuda()
    k, f = 64, z.numel()
    r = Routed(moe, 801, 40, 2, 1)
    d = (1 + torch.rand(r.rows, f, generator=r.g, device="cuda")).bfloat16()
    up = (1 + torch.rand(r.rows, f, generator=r.g, device="cuda")).bfloat16()
    value, vt, slope, st = act_and_slope(z.double().expand(r.rows, f), name)
    op, zrows = moe.expert_op(k, f, name), z.expand(r.rows, f)
    dz, lin = r.sentinel(2 * f), r.sentinel(f)
    moe.moe_expert_glu_backward(r.p, r.plan, op, d, torch.cat([zrows, up], 1).contiguous(), None, None, dz, None, None)
    moe.moe_expert_linear_backward(r.p, r.plan, op, d, None, None, None, None, preact=zrows.contiguous(), dz=lin)
    torch.cuda.synchronize()
    d64, u64 = d.double(), up.double()
    for got, want, tol, what in ((dz[:, :f], d64 * u64 * slope, d64 * u64 * st, "gate"),
                                 (dz[:, f:], d64 * value, d64 * vt, "up"), (lin, d64 * slope, d64 * st, "linear")):
        tol = tol + 2 * U * want.abs()
        assert_within(got, want, tol + BF16 * (want.abs() + tol), f"dz ({what}) of {name}")
