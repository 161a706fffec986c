"""Plain 64-bit references of the experts' operators and of the combine's
gradients, and the bounds their kernels are held to (no tests here).

Bounds.  A result is rounded once to bf16: half a step, 2^-8 relative.  A sum
of n fp32 products carries at most (n + c) * 2^-23 of the sum of the products'
magnitudes (a rounding of at most 2^-23 per addition in any order, truncation
included; c counts the bias, scale and residual operations).
"""
import math

import torch

BF16 = 2.0 ** -8   # half a step
F32 = 2.0 ** -23   # a whole fp32 step: rounding or truncation
C = math.sqrt(2 / math.pi)


def act(z, name):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(C * (z + 0.044715 * z ** 3)))
    if name == "relu":
        return torch.clamp(z, min=0)
    return z


def slope(z, name):
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu_tanh":
        t = torch.tanh(C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def dequant_rows(codes, scales):
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    return v * scales.double().repeat_interleave(128, dim=-1)


def dequant_weights(codes, scales):
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    return v * scales.double().repeat_interleave(128, dim=-1).repeat_interleave(128, dim=-2)


def forward(x, w, bias, glu, name, residual=None):
    """(z, y, bound of z, bound of y) of one expert's rows; double inputs."""
    k = x.shape[1]
    z = x @ w.T
    mag = x.abs() @ w.abs().T
    if bias is not None:
        z = z + bias
        mag = mag + bias.abs()
    dz = (k + 8) * F32 * mag  # of the fp32 z
    if not glu:
        # |act'| <= 1.13; the activation itself: exp of an argument rounded at
        # |a| 2^-24, then a few operations
        a = act(z, name)
        dy = 1.13 * dz + 2.0 ** -18 * z.abs() * (name != "none")
        y = a if residual is None else a + residual
        if residual is not None:
            dy = dy + F32 * (a.abs() + residual.abs())
        return z, y, dz + BF16 * z.abs(), dy + BF16 * (y.abs() + dy)
    f = z.shape[1] // 2
    g, u = z[:, :f], z[:, f:]
    a = act(g, name)
    da = 1.13 * dz[:, :f] + 2.0 ** -18 * g.abs()
    y = a * u
    dy = da * u.abs() + a.abs() * dz[:, f:] + da * dz[:, f:]
    return z, y, dz + BF16 * z.abs(), dy + BF16 * (y.abs() + dy)


def grad(d, z, glu, name):
    """(dz, bound before rounding) from the result's gradient and the kept z."""
    if glu:
        f = z.shape[1] // 2
        g, u = z[:, :f], z[:, f:]
        dz = torch.cat([d * u * slope(g, name), d * act(g, name)], 1)
        # a slope's and a value's own error: as of the activation above, per unit
        tol = torch.cat([2.0 ** -17 * (d * u).abs(), 2.0 ** -18 * (d * g).abs()], 1)
        return dz, tol + 2 * F32 * dz.abs()
    if name == "none":
        return d, torch.zeros_like(d)
    dz = d * slope(z, name)
    return dz, 2.0 ** -17 * d.abs() + 2 * F32 * dz.abs()


def product_bound(a, b, n):
    """Bound of bf16(a @ b) with n products in each sum."""
    return (n + 2) * F32 * (a.abs() @ b.abs()) * (1 + BF16) + BF16 * (a @ b).abs()


def assert_within(got, ref, tol, what):
    """Elementwise, with the same infinities and NaNs."""
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaNs differ"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got - ref).abs()[fine]
    over = err > tol.expand_as(ref)[fine] + 1e-37
    if bool(over.any()):
        at = int(torch.nonzero(over)[0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} past the bound, first "
                             f"{got[fine][at].item()} for {ref[fine][at].item()}, bound "
                             f"{tol.expand_as(ref)[fine][at].item()}")
