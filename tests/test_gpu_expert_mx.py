"""GPU: the experts' products with MX-FP4 weights, from MX-FP4 and FP8 rows, against plain
64-bit references, element by element.  Rows that hold no token are poisoned in every input
(codes of 6, NaN scales) and must come back untouched in every output.

Bounds: those of the other products (expert_reference.py).  An addition of the scaled
instruction, of 128 products and the sum so far, is off by up to 2^-20 of the largest term: K / 128
of them (K / 64 of FP8 rows, in two halves) by less than the (K + 8) 2^-23 of the sum of
magnitudes that the reference allows (2^-20 = 8 * 2^-23, and K / 64 * 8 < K)."""
import numpy as np
import pytest
import torch

import expert_reference as ref
import more_reference as mref
from expert_reference import assert_within
from gpu_helpers import say
from test_gpu_expert import Routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


TABLE = torch.tensor(mref.E2M1)


def mx_value(codes, scales):
    """float64, on the device; scale byte 255: NaN."""
    t = TABLE.to(codes.device)
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).reshape(*codes.shape[:-1], -1)
    x = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return v * x.repeat_interleave(32, -1)


def mx_weights(moe, r, n, k):
    """Random weights [E, n, K], quantised by the library."""
    w = (r.randn(r.experts, n, k) / k ** 0.5).bfloat16()
    codes = torch.empty(r.experts, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(r.experts, n, k // 32, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(w, codes, scales)
    return codes, scales


def mx_rows(moe, r, k, scale=1.0):
    x = (scale * r.randn(r.rows, k)).bfloat16()
    codes = torch.empty(r.rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(r.rows, k // 32, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, codes, scales)
    codes[~r.live], scales[~r.live] = 0x77, 255
    return codes, scales


def fp8_rows(r, k):
    x = r.randn(r.rows, k).view(r.rows, -1, 128)
    scales = x.abs().amax(-1) / 448
    codes = (x / scales[..., None]).to(torch.float8_e4m3fn).view(r.rows, k).view(torch.uint8).clone()
    codes[~r.live], scales[~r.live] = 0x7F, float("nan")
    return codes, scales


def check_quantised(codes, scales, y, dy, what):
    """MX-FP4 results against the unquantised values y, each off by at most dy."""
    got = mx_value(codes, scales)
    rows = y.shape[0]
    b, d = y.view(rows, -1, 32), dy.view(rows, -1, 32)
    high, low = (b.abs() + d).amax(-1), (b.abs() - d).amax(-1).clamp(min=0)
    x = scales.double() - 127

    def exponent(v):
        return torch.where(v > 0, torch.floor(torch.log2(v.clamp(min=1e-300))) - 2, -127.0).clamp(min=-127)

    assert bool(((exponent(low) <= x) & (x <= exponent(high))).all()), f"{what}: a block's scale"
    unit = torch.exp2(x)[..., None]
    a = b.abs() / unit
    # distance to the nearest of the grid's values, then once for the value's error and once
    # for where that moves the nearest
    grid = TABLE[:8].to(y.device)
    near = (a[..., None] - grid).abs().amin(-1)
    err = (got.view_as(b) - b).abs()
    over = err > near * unit + 2 * d + 1e-37
    assert not bool(over.any()), f"{what}: {int(over.sum())} codes past the bound"


# tokens, experts, top_k, K, F and what is special
SIZES = [
    dict(tokens=1, experts=8, top_k=2, k=64, f=8),
    dict(tokens=1, experts=1, top_k=1, k=32, f=8),
    dict(tokens=3, experts=5, top_k=3, k=96, f=24, bias=True),
    dict(tokens=17, experts=4, top_k=2, k=224, f=136, act="gelu_tanh", bias=True),
    dict(tokens=40, experts=2, top_k=2, k=128, f=264, act="relu", pad=16),
    dict(tokens=129, experts=3, top_k=2, k=544, f=72, masked=0.3, skew=1.0, bias=True),
    dict(tokens=200, experts=64, top_k=6, k=256, f=128, pad=128),
    dict(tokens=257, experts=1, top_k=1, k=160, f=392, act="none"),
    dict(tokens=300, experts=7, top_k=1, k=352, f=520, act="gelu_tanh", only=(2, 5)),
    dict(tokens=600, experts=4, top_k=2, k=512, f=256, cap=100, bias=True),
    dict(tokens=1000, experts=6, top_k=2, k=1056, f=328, pad=7, masked=0.1),
    dict(tokens=64, experts=300, top_k=8, k=64, f=64),
    dict(tokens=33, experts=4, top_k=2, k=256, f=256, masked=1.0),
    dict(tokens=2500, experts=3, top_k=1, k=288, f=520, skew=2.0, bias=True),
    # past the small tiles
    dict(tokens=2500, experts=3, top_k=1, k=800, f=1032, bias=True),
    dict(tokens=2000, experts=8, top_k=2, k=1408, f=1552, masked=0.05, skew=0.3, act="gelu_tanh", bias=True),
    dict(tokens=1100, experts=64, top_k=6, k=1024, f=264, pad=16),
    # a long contraction with few rows an expert or few tiles
    dict(tokens=1, experts=4, top_k=1, k=2048, f=24),
    dict(tokens=70, experts=5, top_k=2, k=2144, f=136, masked=0.1, act="gelu_tanh", bias=True),
    dict(tokens=500, experts=1, top_k=1, k=4096 + 32, f=264),
    dict(tokens=160, experts=96, top_k=6, k=2304, f=192, pad=16, skew=0.5, bias=True),
    dict(tokens=5, experts=3, top_k=1, k=7168, f=64),
]


def routed(moe, c, seed):
    keys = ("tokens", "experts", "top_k", "pad", "masked", "skew", "cap", "only")
    return Routed(moe, seed, **{k: c[k] for k in keys if k in c})


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
@pytest.mark.parametrize("glu", [True, False], ids=["glu", "linear"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_forward(moe, i, glu, fmt):
    c = dict(SIZES[i])
    if fmt == "fp8":
        c["k"] = -(-c["k"] // 128) * 128
    say(f"[expert mx] {c} glu={glu} {fmt}")
    r = routed(moe, c, 100 + i)
    k, f, name = c["k"], c["f"], c.get("act", "silu")
    n = 2 * f if glu else f
    x, xs = mx_rows(moe, r, k) if fmt == "mxfp4" else fp8_rows(r, k)
    w, ws = mx_weights(moe, r, n, k)
    bias = r.randn(r.experts, n) if c.get("bias") else None
    residual = r.packed(f) if not glu and i % 2 == 0 else None
    op = moe.expert_op(k, f, act=name, fmt=fmt)
    y = r.sentinel(f)
    if glu:
        moe.moe_expert_glu_mx(r.p, r.plan, op, x, xs, w, ws, y, bias=bias)
    else:
        moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, y, bias=bias, residual=residual)
    torch.cuda.synchronize()
    r.check_rest(y, "y")
    q = qs = None
    if glu and f % 32 == 0:
        q = torch.full((r.rows, f // 2), 0x5A, dtype=torch.uint8, device="cuda")
        qs = torch.full((r.rows, f // 32), 0x5A, dtype=torch.uint8, device="cuda")
        moe.moe_expert_glu_mx(r.p, r.plan, op, x, xs, w, ws, q, h_scales=qs, bias=bias)
        torch.cuda.synchronize()
        assert bool((q[~r.live] == 0x5A).all()) and bool((qs[~r.live] == 0x5A).all())
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        X = mx_value(x[a:b], xs[a:b]) if fmt == "mxfp4" else ref.dequant_rows(x[a:b], xs[a:b])
        _, ry, _, ty = ref.forward(X, mx_value(w[e], ws[e]), None if bias is None else bias[e].double(), glu, name,
                                   None if residual is None else residual[a:b].double())
        assert_within(y[a:b], ry, ty, f"y of expert {e}")
        if q is not None:
            check_quantised(q[a:b], qs[a:b], ry, ty, f"h of expert {e}")


@pytest.mark.parametrize("c", [dict(tokens=6, experts=3, k=256, f=128), dict(tokens=90, experts=2, k=384, f=256),
                               dict(tokens=400, experts=16, k=1536, f=520), dict(tokens=900, experts=2, k=128, f=2048),
                               dict(tokens=12, experts=2, k=2176, f=128)])
def test_fp8_rows_of_any_code(moe, c):
    """Codes from 2^-9 to 448 beside each other: no product is cut, in any tile."""
    say(f"[expert mx] any code {c}")
    r = Routed(moe, 500 + c["k"], c["tokens"], c["experts"], 1)
    k, f = c["k"], c["f"]
    x = torch.randint(0, 256, (r.rows, k), generator=r.g, device="cuda", dtype=torch.int32).to(torch.uint8)
    x = torch.where((x & 0x7F) == 0x7F, torch.zeros_like(x), x)
    xs = 0.5 + torch.rand(r.rows, k // 128, generator=r.g, device="cuda")
    w = torch.randint(0, 256, (r.experts, f, k // 2), generator=r.g, device="cuda", dtype=torch.int32).to(torch.uint8)
    ws = torch.randint(110, 118, (r.experts, f, k // 32), generator=r.g, device="cuda").to(torch.uint8)
    y, rest, op = r.sentinel(f), r.sentinel(f), moe.expert_op(k, f, fmt="fp8")
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, y)
    # with -y for the residual: what the rounding took off, so that the sum itself is seen
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, rest, residual=-y)
    for e, (a, b) in enumerate(r.ranges):
        X, W = ref.dequant_rows(x[a:b], xs[a:b]), mx_value(w[e], ws[e])
        z, tol = X @ W.T, (k + 8) * ref.F32 * (X.abs() @ W.abs().T)
        assert_within(y[a:b], z, tol + ref.BF16 * (z.abs() + tol), f"y of expert {e}")
        left = z - y[a:b].double()
        assert_within(rest[a:b], left, tol + ref.F32 * z.abs() + ref.BF16 * (left.abs() + tol), f"rest of expert {e}")


def test_exact_sums(moe):
    """Codes and scales whose products and sums fp32 holds: y is their one rounding, in every
    form of the rows' length and format."""
    for k in (32, 64, 96, 128, 160, 256, 288, 1056, 2048, 2080):
        for fmt in ("mxfp4", "fp8"):
            if fmt == "fp8" and k % 128:
                continue
            say(f"[expert mx] exact k {k} {fmt}")
            r = Routed(moe, k, 70, 5, 2)
            f = 40

            def codes(*shape):
                return torch.randint(0, 256, shape, generator=r.g, device="cuda", dtype=torch.int32).to(torch.uint8)

            def powers(*shape):
                return torch.randint(125, 130, shape, generator=r.g, device="cuda").to(torch.uint8)

            w, ws = codes(r.experts, f, k // 2), powers(r.experts, f, k // 32)
            if fmt == "mxfp4":
                x, xs = codes(r.rows, k // 2), powers(r.rows, k // 32)
                x[~r.live], xs[~r.live] = 0x77, 255
            else:
                table = torch.tensor([0x00, 0x38, 0xB8, 0x3C, 0xBC, 0x40, 0xC0], dtype=torch.uint8, device="cuda")
                x = table[torch.randint(0, 7, (r.rows, k), generator=r.g, device="cuda")]
                xs = torch.exp2(torch.randint(-2, 3, (r.rows, k // 128), generator=r.g, device="cuda").float())
            y = r.sentinel(f)
            op = moe.expert_op(k, f, fmt=fmt)
            moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, y)
            rest = r.sentinel(f)
            moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, rest, residual=-y)
            for e, (a, b) in enumerate(r.ranges):
                X = mx_value(x[a:b], xs[a:b]) if fmt == "mxfp4" else ref.dequant_rows(x[a:b], xs[a:b])
                z = X @ mx_value(w[e], ws[e]).T
                assert torch.equal(y[a:b].float(), z.float().bfloat16().float())
                assert torch.equal(rest[a:b].float(), (z - y[a:b].double()).float().bfloat16().float())


@pytest.mark.parametrize("k", [128, 160, 224, 288, 1056, 2080])
def test_a_nan_block_stays_in_its_row(moe, k):
    """A NaN scale in the first or last block of a row or of a weight's row reaches that row's (that
    column's) results and no other's, whatever the rows' length."""
    r = Routed(moe, 7, 60, 3, 1)
    f = 48
    x, xs = mx_rows(moe, r, k)
    w, ws = mx_weights(moe, r, f, k)
    y = r.sentinel(f)
    op = moe.expert_op(k, f, fmt="mxfp4")
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, y)
    rows = [a for a, b in r.ranges if b > a] + [b - 1 for a, b in r.ranges if b > a]
    bad_x, bad_w = xs.clone(), ws.clone()
    for n, i in enumerate(rows):
        bad_x[i, 0 if n % 2 else -1] = 255
    bad_w[1, 5, 0] = bad_w[1, 47, -1] = bad_w[0, 0, -1] = bad_w[2, 0, 0] = 255
    out = r.sentinel(f)
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, bad_x, w, bad_w, out)
    torch.cuda.synchronize()
    r.check_rest(out, "y")
    want = torch.zeros_like(y, dtype=torch.bool)
    want[rows] = True
    for e, cols in ((0, [0]), (1, [5, 47]), (2, [0])):
        a, b = r.ranges[e]
        for col in cols:
            want[a:b, col] = True
    want[~r.live] = False
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], y[~want])


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_nan_results_become_nan_blocks(moe, fmt):
    """A result that is not finite makes its 32-value block the NaN block, and the next product's row NaN."""
    r = Routed(moe, 3, 40, 2, 1)
    k, f = 256, 96
    x, xs = mx_rows(moe, r, k) if fmt == "mxfp4" else fp8_rows(r, k)
    w, ws = mx_weights(moe, r, 2 * f, k)
    bias = torch.zeros(2, 2 * f, device="cuda")
    bias[1, f + 40] = float("inf")
    q = torch.zeros(r.rows, f // 2, dtype=torch.uint8, device="cuda")
    qs = torch.zeros(r.rows, f // 32, dtype=torch.uint8, device="cuda")
    moe.moe_expert_glu_mx(r.p, r.plan, moe.expert_op(k, f, "silu", fmt), x, xs, w, ws, q, h_scales=qs, bias=bias)
    down, dscales = mx_weights(moe, r, 16, f)
    y = r.sentinel(16)
    moe.moe_expert_linear_mx(r.p, r.plan, moe.expert_op(f, 16, fmt="mxfp4"), q, qs, down, dscales, y)
    (a0, b0), (a1, b1) = r.ranges
    assert bool((qs[a1:b1, 1] == 255).all()) and not bool((qs[a1:b1, [0, 2]] == 255).any())
    assert not bool((qs[a0:b0] == 255).any()) and not bool(q[a1:b1, 16:32].any())
    assert bool(torch.isnan(y[a1:b1]).all()) and bool(torch.isfinite(y[a0:b0]).all())
