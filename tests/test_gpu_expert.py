"""GPU: the experts' products (gated block, linear layer), their gradients and
the combine's gradients against plain 64-bit references, element by element,
with bounds derived in expert_reference.py.  Rows that hold no token are
poisoned in every input (NaN) and must come back untouched in every output."""
import numpy as np
import pytest
import torch

import expert_reference as ref
from expert_reference import assert_within
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


class Routed:
    """A routing, its plan, and the rows that hold a token."""

    def __init__(self, moe, seed, tokens, experts, top_k, pad=1, masked=0.0, skew=0.0, cap=0, only=None,
                 hidden=64):
        self.g = torch.Generator("cuda").manual_seed(seed)
        logits = self.randn(tokens, experts) + skew * self.randn(experts)
        if only is not None:  # some experts never chosen
            logits[:, [e for e in range(experts) if e not in only]] = -1e9
        ids = logits.topk(top_k, dim=1).indices.int()
        if masked:
            ids[torch.rand(tokens, top_k, generator=self.g, device="cuda") < masked] = -1
        self.p = moe.problem(tokens, hidden, top_k, experts, 1, pad_multiple=pad, expert_capacity=cap)
        self.plan = moe.alloc_plan(self.p)
        moe.moe_dispatch_plan(self.p, ids.contiguous(), self.plan)
        self.ids, self.rows, self.experts = ids, moe.moe_max_rows(self.p), experts
        off = self.plan.expert_offsets.cpu().numpy()
        cnt = self.plan.expert_counts.cpu().numpy()
        self.ranges = [(int(off[e]), int(off[e] + min(cnt[e], off[e + 1] - off[e]))) for e in range(experts)]
        self.live = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for a, b in self.ranges:
            self.live[a:b] = True

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def packed(self, cols, scale=1.0, dtype=torch.bfloat16):
        """Random rows, NaN where no token is."""
        t = (scale * self.randn(self.rows, cols)).to(dtype)
        t[~self.live] = float("nan")
        return t

    def sentinel(self, cols):
        return torch.full((self.rows, cols), -77.0, dtype=torch.bfloat16, device="cuda")

    def check_rest(self, out, what):
        assert bool((out[~self.live] == -77.0).all()), f"{what}: a row without a token was written"


# tokens, experts, top_k, K, F and what is special
SIZES = [
    dict(tokens=1, experts=8, top_k=2, k=64, f=8),
    dict(tokens=1, experts=1, top_k=1, k=8, f=8),
    dict(tokens=3, experts=5, top_k=3, k=72, f=24, bias=True),
    dict(tokens=17, experts=4, top_k=2, k=200, f=136, act="gelu_tanh", bias=True),
    dict(tokens=40, experts=2, top_k=2, k=128, f=264, act="relu", pad=16),
    dict(tokens=129, experts=3, top_k=2, k=520, f=72, masked=0.3, skew=1.0, bias=True),
    dict(tokens=200, experts=64, top_k=6, k=256, f=128, pad=128),
    dict(tokens=257, experts=1, top_k=1, k=136, f=392, act="none"),
    dict(tokens=300, experts=7, top_k=1, k=328, f=520, act="gelu_tanh", only=(2, 5)),
    dict(tokens=600, experts=4, top_k=2, k=512, f=256, cap=100, bias=True),
    dict(tokens=1000, experts=6, top_k=2, k=1032, f=328, pad=7, masked=0.1),
    dict(tokens=64, experts=300, top_k=8, k=64, f=64),
    dict(tokens=90, experts=1024, top_k=4, k=64, f=40),
    dict(tokens=33, experts=4, top_k=2, k=256, f=256, masked=1.0),
    dict(tokens=2500, experts=3, top_k=1, k=264, f=520, skew=2.0, bias=True),
    # few weights and many rows: dw in parts
    dict(tokens=6000, experts=2, top_k=1, k=136, f=72, skew=1.0, bias=True),
    # past the small tiles: enough tiles of 128 x 128, and of 256 x 256, in every product
    dict(tokens=2500, experts=3, top_k=1, k=776, f=1032, bias=True),
    dict(tokens=2000, experts=8, top_k=2, k=1400, f=1552, masked=0.05, skew=0.3, act="gelu_tanh", bias=True),
    dict(tokens=1100, experts=64, top_k=6, k=1032, f=264, pad=16),
    # a long contraction with few rows an expert or few tiles: split over the waves, with
    # uneven shares, and with more tiles than workgroups
    dict(tokens=1, experts=4, top_k=1, k=2048, f=24),
    dict(tokens=70, experts=5, top_k=2, k=2120, f=136, masked=0.1, act="gelu_tanh", bias=True),
    dict(tokens=500, experts=1, top_k=1, k=2056, f=264),
    dict(tokens=160, experts=96, top_k=6, k=2304, f=200, pad=16, skew=0.5, bias=True),
]


def routed(moe, c, seed):
    keys = ("tokens", "experts", "top_k", "pad", "masked", "skew", "cap", "only")
    return Routed(moe, seed, **{k: c[k] for k in keys if k in c})


def weights(r, n, k):
    return (r.randn(r.experts, n, k) / k ** 0.5).bfloat16()


@pytest.mark.parametrize("glu", [True, False], ids=["glu", "linear"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_forward(moe, i, glu):
    c = SIZES[i]
    say(f"[expert forward] {c} glu={glu}")
    r = routed(moe, c, 100 + i)
    k, f, name = c["k"], c["f"], c.get("act", "silu")
    n = 2 * f if glu else f
    x, w = r.packed(k), weights(r, n, k)
    bias = r.randn(r.experts, n) if c.get("bias") else None
    residual = r.packed(f) if not glu and i % 2 == 0 else None
    op = moe.expert_op(k, f, act=name)
    y, z = r.sentinel(f), r.sentinel(n)
    if glu:
        moe.moe_expert_glu(r.p, r.plan, op, x, w, y, bias=bias, preact=z)
    else:
        moe.moe_expert_linear(r.p, r.plan, op, x, w, y, bias=bias, residual=residual, preact=z)
    torch.cuda.synchronize()
    r.check_rest(y, "y")
    r.check_rest(z, "preact")
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        rz, ry, tz, ty = ref.forward(x[a:b].double(), w[e].double(), None if bias is None else bias[e].double(),
                                     glu, name, None if residual is None else residual[a:b].double())
        assert_within(z[a:b], rz, tz, f"preact of expert {e}")
        assert_within(y[a:b], ry, ty, f"y of expert {e}")
    # without the optional output: the same results
    y2 = r.sentinel(f)
    if glu:
        moe.moe_expert_glu(r.p, r.plan, op, x, w, y2, bias=bias)
    else:
        moe.moe_expert_linear(r.p, r.plan, op, x, w, y2, bias=bias, residual=residual)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))


FP8_SIZES = [
    dict(tokens=1, experts=4, top_k=2, k=128, f=128),
    dict(tokens=5, experts=3, top_k=2, k=384, f=256, bias=True),
    dict(tokens=150, experts=4, top_k=2, k=512, f=384, act="gelu_tanh", masked=0.2),
    dict(tokens=700, experts=2, top_k=1, k=256, f=128, pad=128, bias=True),
    dict(tokens=64, experts=128, top_k=8, k=256, f=128, act="relu"),
    # enough tiles: workgroups that take tile after tile, and one workgroup a tile
    dict(tokens=300, experts=64, top_k=6, k=384, f=256, pad=16, bias=True),
    dict(tokens=3000, experts=4, top_k=1, k=512, f=768, skew=0.5, bias=True),
    # split over the waves: uneven shares of the steps, more tiles than workgroups
    dict(tokens=3, experts=2, top_k=2, k=2048, f=256, bias=True),
    dict(tokens=200, experts=40, top_k=2, k=2176, f=384, masked=0.1),
    dict(tokens=40, experts=2, top_k=2, k=2432, f=128, act="none", bias=True),
]


@pytest.mark.parametrize("glu", [True, False], ids=["glu", "linear"])
@pytest.mark.parametrize("i", range(len(FP8_SIZES)))
def test_forward_fp8(moe, i, glu):
    c = FP8_SIZES[i]
    say(f"[expert forward fp8] {c} glu={glu}")
    r = routed(moe, c, 200 + i)
    k, f, name = c["k"], c["f"], c.get("act", "silu")
    n = 2 * f if glu else f
    x = (100 * r.randn(r.rows, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    xs = torch.rand(r.rows, k // 128, generator=r.g, device="cuda") / 100
    x[~r.live] = 0x7F  # NaN codes
    xs[~r.live] = float("nan")
    w = (100 * r.randn(r.experts, n, k)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = (0.2 + torch.rand(r.experts, n // 128, k // 128, generator=r.g, device="cuda")) / (100 * k ** 0.5)
    bias = r.randn(r.experts, n) if c.get("bias") else None
    op = moe.expert_op(k, f, act=name, fmt="fp8")
    y, z = r.sentinel(f), r.sentinel(n)
    call = moe.moe_expert_glu if glu else moe.moe_expert_linear
    call(r.p, r.plan, op, x, w, y, x_scales=xs, w_scales=ws, bias=bias, preact=z)
    torch.cuda.synchronize()
    r.check_rest(y, "y")
    r.check_rest(z, "preact")
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        rz, ry, tz, ty = ref.forward(ref.dequant_rows(x[a:b], xs[a:b]), ref.dequant_weights(w[e], ws[e]),
                                     None if bias is None else bias[e].double(), glu, name)
        assert_within(z[a:b], rz, tz, f"preact of expert {e}")
        assert_within(y[a:b], ry, ty, f"y of expert {e}")


@pytest.mark.parametrize("glu", [True, False], ids=["glu", "linear"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_backward(moe, i, glu):
    c = SIZES[i]
    say(f"[expert backward] {c} glu={glu}")
    r = routed(moe, c, 300 + i)
    k, f, name = c["k"], c["f"], c.get("act", "silu")
    if not glu and i % 3 == 0:
        name = "none"
    n = 2 * f if glu else f
    kept = glu or name != "none"
    d, x, w = r.packed(f), r.packed(k), weights(r, n, k)
    z = r.packed(n, 2.0) if kept else None
    op = moe.expert_op(k, f, act=name)
    dz = r.sentinel(n) if kept else None
    dx = r.sentinel(k)
    dw = torch.full((r.experts, n, k), -77.0, dtype=torch.bfloat16, device="cuda")
    db = torch.full((r.experts, n), -77.0, device="cuda")
    ws = moe.alloc_expert_workspace(r.p, op)
    ws.fill_(0xFF)
    if glu:
        moe.moe_expert_glu_backward(r.p, r.plan, op, d, z, x, w, dz, dx, dw, dbias=db, workspace=ws)
    else:
        moe.moe_expert_linear_backward(r.p, r.plan, op, d, x, w, dx, dw, preact=z, dz=dz, dbias=db, workspace=ws)
    torch.cuda.synchronize()
    if kept:
        r.check_rest(dz, "dz")
    r.check_rest(dx, "dx")
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            assert not bool(dw[e].any()) and not bool(db[e].any()), f"expert {e} without rows"
            continue
        rdz, tol = ref.grad(d[a:b].double(), z[a:b].double() if kept else None, glu, name)
        if kept:
            assert_within(dz[a:b], rdz, tol + ref.BF16 * (rdz.abs() + tol), f"dz of expert {e}")
        m = b - a
        assert_within(db[e], rdz.sum(0), tol.sum(0) + (m + 2) * ref.F32 * rdz.abs().sum(0), f"dbias of expert {e}")
        used = (dz if kept else d)[a:b].double()  # the products read the rounded dz
        xe, we = x[a:b].double(), w[e].double()
        assert_within(dx[a:b], used @ we, ref.product_bound(used, we, n), f"dx of expert {e}")
        assert_within(dw[e], used.T @ xe, ref.product_bound(used.T, xe, m), f"dw of expert {e}")


COMBINE = [dict(tokens=1, experts=1, top_k=1, hidden=8), dict(tokens=7, experts=4, top_k=3, hidden=72),
           dict(tokens=130, experts=16, top_k=4, hidden=520, masked=0.4),
           dict(tokens=64, experts=64, top_k=6, hidden=4096, pad=128),
           dict(tokens=33, experts=256, top_k=8, hidden=7168), dict(tokens=20, experts=40, top_k=37, hidden=136),
           dict(tokens=500, experts=4, top_k=2, hidden=1032, cap=120), dict(tokens=9, experts=9, top_k=2, hidden=64, masked=1.0),
           dict(tokens=5, experts=80, top_k=64, hidden=264, masked=0.1)]


@pytest.mark.parametrize("i", range(len(COMBINE)))
def test_combine_backward(moe, i):
    c = COMBINE[i]
    say(f"[combine backward] {c}")
    r = Routed(moe, 400 + i, **c)
    h, n, k = c["hidden"], c["tokens"], c["top_k"]
    y, dout = r.packed(h), r.randn(n, h).bfloat16()
    wts = r.randn(n, k)
    dy, dw = r.sentinel(h), torch.full((n, k), -77.0, device="cuda")
    moe.moe_combine_backward(r.p, r.plan, y, wts, dout, dy, dw)
    torch.cuda.synchronize()
    slot = r.plan.slot.long()
    live = slot >= 0
    rows = y[slot.clamp(min=0)].double()
    d64 = dout.double()[:, None, :]
    want = torch.where(live, (torch.where(live[..., None], rows, 0.0) * d64).sum(-1), 0.0)
    mag = (torch.where(live[..., None], rows, 0.0) * d64).abs().sum(-1)
    assert_within(dw, want, (h + 2) * ref.F32 * mag, "dweights")
    expect = torch.full_like(dy, -77.0)
    expect[slot[live]] = (wts[..., None] * dout.float()[:, None, :])[live].bfloat16()
    assert torch.equal(dy.view(torch.int16), expect.view(torch.int16))
    # the unweighted combine's gradient: copies, and no gradient of weights
    dy2 = r.sentinel(h)
    moe.moe_combine_backward(r.p, r.plan, None, None, dout, dy2)
    torch.cuda.synchronize()
    expect[slot[live]] = dout[:, None, :].expand(n, k, h)[live]
    assert torch.equal(dy2.view(torch.int16), expect.view(torch.int16))
