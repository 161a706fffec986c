"""GPU: the experts' operators as they are used together and at the edges: a whole
expert layer forward and backward, FP8 rows as the dispatch writes them,
captured and replayed graphs, other streams, repeated runs, values that are not
finite, plan arrays that describe no routing, no tokens at all."""
import numpy as np
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


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


class Layer:
    """dispatch -> gated block -> linear layer -> combine, and back."""

    def __init__(self, moe, r, hidden, ffn, act="silu"):
        self.moe, self.r, self.h, self.f = moe, r, hidden, ffn
        n, e, rows = r.p.n_tokens, r.experts, r.rows
        self.x = r.randn(n, hidden).bfloat16()
        self.gates = torch.softmax(r.randn(n, r.p.top_k), 1)
        self.w1, self.w2 = weights(r, 2 * ffn, hidden), weights(r, hidden, ffn)
        self.b1, self.b2 = r.randn(e, 2 * ffn), r.randn(e, hidden)
        self.dout = r.randn(n, hidden).bfloat16()
        self.op1, self.op2 = moe.expert_op(hidden, ffn, act), moe.expert_op(ffn, hidden)
        self.ws1 = moe.alloc_expert_workspace(r.p, self.op1)
        self.ws2 = moe.alloc_expert_workspace(r.p, self.op2)

        def rows_of(c):
            return torch.zeros(rows, c, dtype=torch.bfloat16, device="cuda")

        self.xp, self.pre, self.hid, self.y = rows_of(hidden), rows_of(2 * ffn), rows_of(ffn), rows_of(hidden)
        self.dy, self.dh, self.dz, self.dxp = rows_of(hidden), rows_of(ffn), rows_of(2 * ffn), rows_of(hidden)
        self.out, self.dx = torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.dgates = torch.zeros_like(self.gates)
        self.dw1, self.dw2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        self.db1, self.db2 = torch.zeros_like(self.b1), torch.zeros_like(self.b2)

    RESULTS = ("xp", "pre", "hid", "y", "out", "dy", "dgates", "dh", "dw2", "db2", "dz", "dxp", "dw1", "db1", "dx")

    def run(self):
        m, r = self.moe, self.r
        p, plan = r.p, r.plan
        m.moe_dispatch(p, plan, self.x, self.xp, None)
        m.moe_expert_glu(p, plan, self.op1, self.xp, self.w1, self.hid, bias=self.b1, preact=self.pre)
        m.moe_expert_linear(p, plan, self.op2, self.hid, self.w2, self.y, bias=self.b2)
        m.moe_combine(p, plan, self.y, self.gates, self.out)
        m.moe_combine_backward(p, plan, self.y, self.gates, self.dout, self.dy, self.dgates)
        m.moe_expert_linear_backward(p, plan, self.op2, self.dy, self.hid, self.w2, self.dh, self.dw2,
                                     dbias=self.db2, workspace=self.ws2)
        m.moe_expert_glu_backward(p, plan, self.op1, self.dh, self.pre, self.xp, self.w1, self.dz, self.dxp,
                                  self.dw1, dbias=self.db1, workspace=self.ws1)
        m.moe_combine(p, plan, self.dxp, None, self.dx)  # the dispatch's gradient

    def results(self):
        return {k: getattr(self, k).clone() for k in self.RESULTS}


@pytest.mark.parametrize("kw", [dict(tokens=300, experts=6, top_k=2, pad=16, masked=0.1),
                                dict(tokens=40, experts=16, top_k=4), dict(tokens=900, experts=2, top_k=1, skew=1.0)])
def test_a_layer_forward_and_backward(moe, kw):
    say(f"[expert layer] {kw}")
    h, f = 264, 136
    r = Routed(moe, 11, hidden=h, **kw)
    L = Layer(moe, r, h, f)
    L.run()
    torch.cuda.synchronize()
    slot = r.plan.slot.long()
    live = slot >= 0
    # the whole layer in 64 bits, from the same inputs
    x, gates, dout = L.x.double(), L.gates.double(), L.dout.double()
    src = r.plan.packed_src.long()
    y = torch.zeros(r.rows, h, dtype=torch.float64, device="cuda")
    dxp = torch.zeros_like(y)
    dy = torch.zeros_like(y)
    dy[slot[live]] = (gates[..., None] * dout[:, None, :])[live]
    total = 0.0
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        xe, w1, w2 = x[src[a:b]], L.w1[e].double(), L.w2[e].double()
        z, hid, _, _ = ref.forward(xe, w1, L.b1[e].double(), True, "silu")
        y[a:b] = hid @ w2.T + L.b2[e].double()
        dh = dy[a:b] @ w2
        dz, _ = ref.grad(dh, z, True, "silu")
        dxp[a:b] = dz @ w1
        # rounded on the way: z, h (forward), dy, dh, dz (backward), each 2^-8 at most
        # of its value; through sums of independent terms they add like noise,
        # so the norms stay within a few steps
        for got, want, what in ((L.dw1[e], dz.T @ xe, "dw1"), (L.dw2[e], dy[a:b].T @ hid, "dw2"),
                                (L.db1[e], dz.sum(0), "db1"), (L.db2[e], dy[a:b].sum(0), "db2")):
            err = (got.double() - want).norm() / want.norm()
            assert err < 5 * ref.BF16, (e, what, float(err))
            total += float(err)
    out = (gates[..., None] * torch.where(live[..., None], y[slot.clamp(min=0)], 0.0)).sum(1)
    dx = torch.where(live[..., None], dxp[slot.clamp(min=0)], 0.0).sum(1)
    dg = torch.where(live, (y[slot.clamp(min=0)] * dout[:, None, :]).sum(-1), 0.0)
    for got, want, what in ((L.out, out, "out"), (L.dx, dx, "dx"), (L.dgates, dg, "dgates")):
        err = (got.double() - want).norm() / want.norm()
        assert err < 5 * ref.BF16, (what, float(err))
    say(f"[expert layer] summed relative errors of the weights' gradients {total:.4f}")


def test_gradients_against_differences(moe):
    """<dw, d> and <dx, d> against a central difference of the 64-bit loss along d.
    dz is rounded (2^-8 of each term), dw and dx are rounded once more."""
    k, f = 136, 72
    r = Routed(moe, 12, 200, 3, 2, masked=0.1)
    x, w, d = r.packed(k), weights(r, 2 * f, k), r.packed(f)
    op = moe.expert_op(k, f, "gelu_tanh")
    y, z = r.sentinel(f), r.sentinel(2 * f)
    moe.moe_expert_glu(r.p, r.plan, op, x, w, y, preact=z)
    dz, dx, dw = r.sentinel(2 * f), r.sentinel(k), torch.empty_like(w)
    moe.moe_expert_glu_backward(r.p, r.plan, op, d, z, x, w, dz, dx, dw,
                                workspace=moe.alloc_expert_workspace(r.p, op))
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(r.ranges):
        xe, we, de = x[a:b].double(), w[e].double(), d[a:b].double()

        def loss(xe, we):
            return (de * ref.forward(xe, we, None, True, "gelu_tanh")[1]).sum()

        for what, got, v in (("dx", dx[a:b].double(), xe), ("dw", dw[e].double(), we)):
            u, eps = r.randn(*v.shape).double(), 1e-5
            pair = [loss(xe + s * eps * u, we) if what == "dx" else loss(xe, we + s * eps * u) for s in (1, -1)]
            num = (pair[0] - pair[1]) / (2 * eps)
            # of each term of got * u: the kept z's rounding moves the slopes (2^-8, and at
            # most |z| of that again), dz's and the result's 2^-8 each; as noise over v's elements
            bound = 6 * ref.BF16 * (got * u).norm() * 3
            assert abs((got * u).sum() - num) < bound, (e, what, float((got * u).sum()), float(num), float(bound))


def test_fp8_rows_as_the_dispatch_writes_them(moe):
    h, f = 384, 128
    r = Routed(moe, 13, 150, 5, 3, pad=8, masked=0.1, hidden=h)
    p8 = moe.problem(150, h, 3, 5, 1, pad_multiple=8, fmt="fp8")
    x = r.randn(150, h).bfloat16()
    x[7] = 0  # blocks without a value: scale 0
    codes, scales = moe.alloc_payload(p8)
    codes.fill_(0x7F)
    scales.fill_(float("nan"))
    moe.moe_dispatch(p8, r.plan, x, codes, scales)
    w = (100 * r.randn(5, 2 * f, h)).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(5, 2 * f // 128, h // 128, generator=r.g, device="cuda") / 2000
    y = r.sentinel(f)
    op = moe.expert_op(h, f, "silu", "fp8")
    moe.moe_expert_glu(p8, r.plan, op, codes, w, y, x_scales=scales, w_scales=ws)
    torch.cuda.synchronize()
    r.check_rest(y, "y")
    for e, (a, b) in enumerate(r.ranges):
        xe = ref.dequant_rows(codes[a:b], scales[a:b])
        _, ry, _, ty = ref.forward(xe, ref.dequant_weights(w[e].view(torch.uint8), ws[e]), None, True, "silu")
        assert_within(y[a:b], ry, ty, f"y of expert {e}")


@pytest.mark.parametrize("kw,h,f", [(dict(tokens=64, experts=16, top_k=2), 256, 128),
                                    (dict(tokens=1500, experts=4, top_k=2, pad=8), 520, 264)])
def test_captured_and_replayed(moe, kw, h, f):
    """Two graphs of the same layer shape with their own buffers, replayed in turn
    with eager work between and new inputs in place; every replay against
    the eager results, bit for bit."""
    layers = [Layer(moe, Routed(moe, 20 + i, hidden=h, **kw), h, f) for i in range(2)]
    side = torch.cuda.Stream()
    graphs = []
    for L in layers:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.run()
        graphs.append(g)
    for turn in range(4):
        say(f"[expert graph] turn {turn}")
        for L in layers:
            L.x.copy_(L.r.randn(*L.x.shape))
            L.dout.copy_(L.r.randn(*L.dout.shape))
            L.w1.mul_(1.25)
        for g in graphs:
            g.replay()
        got = [L.results() for L in layers]
        torch.cuda.synchronize()
        for L, res in zip(layers, got):
            for k in L.RESULTS:
                getattr(L, k).fill_(0)
            L.run()
            torch.cuda.synchronize()
            for k, v in L.results().items():
                assert torch.equal(bits(res[k]), bits(v)), (turn, k)


def test_two_streams_and_repeats(moe):
    """Two layers at once on streams of their own, again and again: every run the same
    bits as the first, alone on the default stream."""
    h, f = 264, 392
    layers = [Layer(moe, Routed(moe, 30 + i, 700, 5, 2, hidden=h, skew=1.0), h, f) for i in range(2)]
    for L in layers:
        L.run()
    torch.cuda.synchronize()
    first = [L.results() for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for turn in range(3):
        for L, s in zip(layers, streams):
            for k in L.RESULTS:
                getattr(L, k).zero_()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                L.run()
        torch.cuda.synchronize()
        for L, want in zip(layers, first):
            for k, v in L.results().items():
                assert torch.equal(bits(v), bits(want[k])), (turn, k)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_values_that_are_not_finite_stay_where_they_are(moe, bad, fmt):
    """A row's NaN or infinity reaches that row alone (and its expert's dw), an
    expert's weights' its rows alone."""
    k, f = 256, 128
    r = Routed(moe, 40, 200, 4, 2)
    (a0, _), (a1, b1) = r.ranges[0], r.ranges[1]

    def run(row, weight):
        g = torch.Generator("cuda").manual_seed(5)
        x = torch.randn(r.rows, k, generator=g, device="cuda")
        w = torch.randn(4, 2 * f, k, generator=g, device="cuda")
        y = torch.zeros(r.rows, f, dtype=torch.bfloat16, device="cuda")
        if fmt == "bf16":
            x, w = x.bfloat16(), w.bfloat16()
            if row:
                x[a0 + 3, 17] = bad
            if weight:
                w[1, 5, 9] = bad
            moe.moe_expert_glu(r.p, r.plan, moe.expert_op(k, f, "silu"), x, w, y)
        else:
            x8, w8 = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w))
            xs = torch.ones(r.rows, k // 128, device="cuda")
            ws = torch.full((4, 2 * f // 128, k // 128), 0.01, device="cuda")
            if row:
                xs[a0 + 3, 1] = bad
            if weight:
                ws[1, 0, 1] = bad
            moe.moe_expert_glu(r.p, r.plan, moe.expert_op(k, f, "silu", fmt="fp8"), x8, w8, y, x_scales=xs, w_scales=ws)
        torch.cuda.synchronize()
        return y

    clean = run(False, False)
    assert bool(torch.isfinite(clean).all())
    y = run(True, False)
    others = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    others[a0 + 3] = False
    assert torch.equal(bits(y[others]), bits(clean[others]))
    assert not bool(torch.isfinite(y[a0 + 3]).all())
    y = run(False, True)
    others = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    others[a1:b1] = False
    assert torch.equal(bits(y[others]), bits(clean[others]))
    assert not bool(torch.isfinite(y[a1:b1]).all())


def test_an_expert_without_rows_may_hold_anything(moe):
    r = Routed(moe, 41, 64, 5, 2, only=(0, 2, 4))
    k, f = 72, 40
    x, w, d = r.packed(k), weights(r, 2 * f, k), r.packed(f)
    w[1] = w[3] = float("nan")
    op = moe.expert_op(k, f, "silu")
    y, z = r.sentinel(f), r.sentinel(2 * f)
    moe.moe_expert_glu(r.p, r.plan, op, x, w, y, preact=z)
    dz, dx, dw = r.sentinel(2 * f), r.sentinel(k), torch.full_like(w, float("nan"))
    db = torch.full((5, 2 * f), float("nan"), device="cuda")
    moe.moe_expert_glu_backward(r.p, r.plan, op, d, z, x, w, dz, dx, dw, dbias=db,
                                workspace=moe.alloc_expert_workspace(r.p, op))
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y[r.live]).all()) and bool(torch.isfinite(dx[r.live]).all())
    assert bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())
    assert not bool(dw[1].any()) and not bool(dw[3].any()) and not bool(db[3].any())


def test_no_tokens(moe):
    p, op = moe.problem(0, 64, 1, 3, 1), moe.expert_op(64, 40, "silu")
    plan = moe.alloc_plan(p)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_plan(p, torch.empty(0, 1, dtype=torch.int32, device="cuda"), plan)
    w = torch.ones(3, 80, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_glu(p, plan, op, empty, w, empty)
    dw, db = torch.ones_like(w), torch.ones(3, 80, device="cuda")
    moe.moe_expert_glu_backward(p, plan, op, empty, empty, empty, w, empty, empty, dw, dbias=db,
                                workspace=moe.alloc_expert_workspace(p, op))
    moe.moe_combine_backward(p, plan, empty, torch.empty(0, 1, device="cuda"), empty, empty,
                             torch.empty(0, 1, device="cuda"))
    torch.cuda.synchronize()
    assert not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("kind", ["negative", "huge", "backwards", "minimum"])
def test_plan_arrays_that_describe_no_routing(moe, kind):
    """Whatever offsets and counts hold, nothing outside the buffers is written: each
    output lies between guards."""
    r = Routed(moe, 42, 100, 6, 2)
    k, f = 136, 72
    bad = {"negative": (-5, -7), "huge": (1 << 30, 1 << 30), "backwards": (None, None),
           "minimum": (-(1 << 31), (1 << 31) - 1)}[kind]
    off, cnt = r.plan.expert_offsets, r.plan.expert_counts
    if kind == "backwards":
        off.copy_(off.flip(0))
    else:
        off.fill_(bad[0])
        cnt.fill_(bad[1])
        off[2] = 40
        off[4] = 1 << 30
    held = []

    def guarded(shape, dtype=torch.bfloat16, fill=1.0):
        n = int(np.prod(shape))
        raw = torch.full((n + 8192,), 55.0, dtype=dtype, device="cuda")
        raw[4096:4096 + n] = fill
        held.append((raw, n))
        return raw[4096:4096 + n].view(shape)

    op = moe.expert_op(k, f, "silu")
    x, w = guarded((r.rows, k)), guarded((6, 2 * f, k))
    y, z, dz = guarded((r.rows, f)), guarded((r.rows, 2 * f)), guarded((r.rows, 2 * f))
    dx, dw, db = guarded((r.rows, k)), guarded((6, 2 * f, k)), guarded((6, 2 * f), torch.float32)
    moe.moe_expert_glu(r.p, r.plan, op, x, w, y, preact=z)
    n = moe.moe_expert_workspace_bytes(r.p, op)
    ws = torch.full((n + 512,), 77, dtype=torch.uint8, device="cuda")
    moe.moe_expert_glu_backward(r.p, r.plan, op, y, z, x, w, dz, dx, dw, dbias=db, workspace=ws[256:256 + n])
    torch.cuda.synchronize()
    for raw, n_ in held:
        assert bool((raw[:4096] == 55).all()) and bool((raw[4096 + n_:] == 55).all())
    assert bool((ws[:256] == 77).all()) and bool((ws[256 + n:] == 77).all())


def test_residual_in_place(moe):
    r = Routed(moe, 43, 130, 3, 2, pad=4)
    k, f = 200, 136
    x, w, res = r.packed(k), weights(r, f, k), r.packed(f)
    op = moe.expert_op(k, f, "relu")
    y = r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, op, x, w, y, residual=res)
    same = res.clone()
    moe.moe_expert_linear(r.p, r.plan, op, x, w, same, residual=same)
    torch.cuda.synchronize()
    assert torch.equal(bits(same[r.live]), bits(y[r.live]))


def test_parts_of_the_gradients(moe):
    """dx, dw and dbias one at a time: the same bits as together."""
    r = Routed(moe, 44, 180, 4, 2)
    k, f = 136, 72
    x, w, d, z = r.packed(k), weights(r, 2 * f, k), r.packed(f), r.packed(2 * f)
    op, ws = moe.expert_op(k, f, "silu"), None
    ws = moe.alloc_expert_workspace(r.p, op)

    def run(want):
        dz = r.sentinel(2 * f)
        dx = r.sentinel(k) if "dx" in want else None
        dw = torch.zeros_like(w) if "dw" in want else None
        db = torch.zeros(4, 2 * f, device="cuda") if "db" in want else None
        moe.moe_expert_glu_backward(r.p, r.plan, op, d, z, x if dw is not None else None,
                                    w if dx is not None else None, dz, dx, dw, dbias=db,
                                    workspace=None if dw is None and db is None else ws)
        torch.cuda.synchronize()
        return {"dz": dz, "dx": dx, "dw": dw, "db": db}

    whole = run(("dx", "dw", "db"))
    for part in ("dx", "dw", "db"):
        got = run((part,))
        assert torch.equal(bits(got["dz"]), bits(whole["dz"]))
        assert torch.equal(bits(got[part]), bits(whole[part]))


def test_offsets_past_32_bits(moe):
    """Rows, results and weights of more than 4 GiB: the last expert's last rows."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    tokens, experts, k, f = 150_000, 3, 16_384, 24
    r = Routed(moe, 50, tokens, experts, 1, hidden=8)
    a, b = r.ranges[-1]
    assert b == tokens and b * k * 2 > 1 << 32
    tail = slice(b - 40, b)
    x = torch.empty(r.rows, k, dtype=torch.bfloat16, device="cuda").normal_(generator=r.g)
    w = weights(r, f, k)
    y = r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, moe.expert_op(k, f), x, w, y)
    torch.cuda.synchronize()
    _, ry, _, ty = ref.forward(x[tail].double(), w[-1].double(), None, False, "none")
    assert_within(y[tail], ry, ty, "y of rows past 4 GiB")
    # and as results: dx of the same size, with dw over all of the expert's rows
    d, dw = r.randn(r.rows, f).bfloat16(), torch.empty_like(w)
    dx = torch.full((r.rows, k), -77.0, dtype=torch.bfloat16, device="cuda")
    op = moe.expert_op(k, f)
    moe.moe_expert_linear_backward(r.p, r.plan, op, d, x, w, dx, dw, workspace=moe.alloc_expert_workspace(r.p, op))
    torch.cuda.synchronize()
    dt = d[tail].double()
    assert_within(dx[tail], dt @ w[-1].double(), ref.product_bound(dt, w[-1].double(), f), "dx past 4 GiB")
    dc, xc = d[a:b, :8].double(), x[a:b, -64:].double()
    assert_within(dw[-1, :8, -64:], dc.T @ xc, ref.product_bound(dc.T, xc, b - a), "dw over rows past 4 GiB")
    del x, dx, dw
    # weights: 70 experts of 64 MiB, the last one's result
    r = Routed(moe, 51, 20, 70, 2, only=(0, 69), hidden=8)
    k, f = 4096, 8192
    w = torch.empty(70, f, k, dtype=torch.bfloat16, device="cuda").normal_(0, k ** -0.5, generator=r.g)
    x, y = r.packed(k), r.sentinel(f)
    moe.moe_expert_linear(r.p, r.plan, moe.expert_op(k, f), x, w, y)
    torch.cuda.synchronize()
    for e in (0, 69):
        a, b = r.ranges[e]
        _, ry, _, ty = ref.forward(x[a:b].double(), w[e].double(), None, False, "none")
        assert_within(y[a:b], ry, ty, f"y of expert {e}")
