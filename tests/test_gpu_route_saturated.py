"""GPU: the sigmoid router's gradient where its scores are near 0 or 1: the slope s (1 - s) keeps its
bits on both sides (logits up to 80 either way), element by element against 64 bits.

Bounds, in fp32 steps of 2^-23 relative.  exp(-|l|): log2 e is held to 0.23 |l| 2^-24 of the result,
the hardware's exp2 adds one step, the last operation half a one: (1.5 + |l| / 8).  The larger of s
and 1 - s: a sum, a reciprocal and half of that: 3.  The smaller one, their product: 5 + |l| / 8.
The slope times a gradient: (10 + |l| / 8).  Renormalised, with X the largest |l| chosen: a
weight is off by twice a score and a sum over the lanes (13 + X / 4), the weighted mean by as
much and a sum again, and both meet the slope: (42 + X) of w (|d| + sum |d| w) (1 - s)."""
import numpy as np
import pytest
import torch

from gpu_helpers import say

pytestmark = pytest.mark.gpu
F32, BF16 = 2.0 ** -23, 2.0 ** -8  # a step; half a step


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


def gradient(l, ids, dw, ds, renormalize, scale):
    """(dlogits, bound) in 64 bits; 1 - s is formed as a sigmoid of its own."""
    l = l.astype(np.float64)
    s, rest = 1 / (1 + np.exp(-l)), 1 / (1 + np.exp(l))
    rows = np.arange(len(l))[:, None]
    want, tol = np.zeros_like(l), np.zeros_like(l)
    if ds is not None:
        want += ds * s * rest
        tol += (10 + np.abs(l) / 8) * F32 * np.abs(ds) * s * rest
    if dw is not None:
        u, si, ri = dw.astype(np.float64) * scale, s[rows, ids], rest[rows, ids]
        if renormalize:
            w = si / si.sum(1, keepdims=True)
            part = w * (u - (u * w).sum(1, keepdims=True)) * ri
            most = np.abs(l[rows, ids]).max(1, keepdims=True)
            far = (42 + most) * F32 * w * (np.abs(u) + (np.abs(u) * w).sum(1, keepdims=True)) * ri
        else:
            part = u * si * ri
            far = (10 + np.abs(l[rows, ids]) / 8) * F32 * np.abs(part)
        np.put_along_axis(want, ids, np.take_along_axis(want, ids, 1) + part, 1)
        np.put_along_axis(tol, ids, np.take_along_axis(tol, ids, 1) + far, 1)
    return want, tol + F32 * np.abs(want) + 2.0 ** -118


# one of each number of lanes and of experts a lane
@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (33, 24, 4), (20, 100, 8), (9, 200, 16), (7, 256, 20), (5, 500, 8),
                                   (3, 1000, 30)])
@pytest.mark.parametrize("logits", ["fp32", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("given", ["weights", "scores", "both"])
def test_slope_of_saturated_scores(moe, n, e, k, logits, renormalize, given):
    say(f"[route saturated] {n} x {e}, k {k}, {logits}, renormalize {renormalize}, {given}")
    rng = np.random.default_rng(n * 7 + e)
    l = (rng.choice([-1.0, 1.0], (n, e)) * rng.choice([8, 10, 12, 14, 16, 17, 20, 40, 80], (n, e))
         * rng.uniform(0.9, 1.0, (n, e))).astype(np.float32)
    t = torch.from_numpy(l).cuda()
    if logits == "bf16":
        t = t.bfloat16()
        l = t.float().cpu().numpy()
    # (among the chosen ones at least one that is not small: their sum stays in fp32's range)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    if renormalize:
        l[np.arange(n), ids[:, 0]] = np.abs(l[np.arange(n), ids[:, 0]])
        t = torch.from_numpy(l).cuda().to(t.dtype)
    dw = rng.standard_normal((n, k)).astype(np.float32) if given != "scores" else None
    ds = rng.standard_normal((n, e)).astype(np.float32) if given != "weights" else None
    p = moe.problem(n, 8, k, e, 1)
    r = moe.router("sigmoid", logits, renormalize=renormalize, scale=2.5)
    dl = torch.full_like(t, -7.0)
    moe.moe_route_backward(p, r, t, torch.from_numpy(ids).cuda(), dl,
                           dweights=None if dw is None else torch.from_numpy(dw).cuda(),
                           dscores=None if ds is None else torch.from_numpy(ds).cuda())
    got = dl.double().cpu().numpy()
    want, tol = gradient(l, ids, dw, ds, renormalize, 2.5)
    if logits == "bf16":
        tol = tol + BF16 * (np.abs(want) + tol)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{(err / tol).max()} of the bound"


def test_both_sides_alike(moe):
    """Without dweights the gradient is the slope, which is even: l and -l give the same bits."""
    n, e = 64, 96
    g = torch.Generator("cuda").manual_seed(1)
    l = 30 * torch.rand(n, e, generator=g, device="cuda")
    p, r = moe.problem(n, 8, 2, e, 1), moe.router("sigmoid")
    a, b, ds = torch.empty_like(l), torch.empty_like(l), torch.ones_like(l)
    moe.moe_route_backward(p, r, l, None, a, dscores=ds)
    moe.moe_route_backward(p, r, -l, None, b, dscores=ds)
    assert torch.equal(a, b) and bool((a > 0).all())
