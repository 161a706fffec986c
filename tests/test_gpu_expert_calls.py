"""GPU: calls of the experts' operators that are allowed and come seldom: the stream
given by hand, FP8 layers and split weights' gradients captured into two graphs and
replayed in turn, a token that names one expert twice."""
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


class Step:
    """A gated block and, for bf16, its gradients, with buffers of its own; `change`
    puts new inputs in place."""

    def __init__(self, moe, seed, tokens, experts, top_k, k, f, fmt):
        self.moe, self.fmt, self.k, self.f = moe, fmt, k, f
        self.r = r = Routed(moe, seed, tokens, experts, top_k, masked=0.05)
        self.op = moe.expert_op(k, f, "silu", fmt)
        self.h, self.z = r.sentinel(f), r.sentinel(2 * f)
        self.out = [self.h, self.z]
        if fmt == "fp8":
            self.x = torch.zeros(r.rows, k, dtype=torch.uint8, device="cuda")
            self.xs, self.ws = torch.ones(r.rows, k // 128, device="cuda"), torch.ones(experts, 2 * f // 128, k // 128, device="cuda")
            self.w = (16 * r.randn(experts, 2 * f, k)).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.x, self.w, self.d = torch.zeros(r.rows, k, dtype=torch.bfloat16, device="cuda"), weights(r, 2 * f, k), r.packed(f)
            self.dz, self.dx, self.dw = r.sentinel(2 * f), r.sentinel(k), torch.zeros_like(self.w)
            self.db = torch.zeros(experts, 2 * f, device="cuda")
            self.work = moe.alloc_expert_workspace(r.p, self.op)
            self.out += [self.dz, self.dx, self.dw, self.db]
        self.change()

    def change(self):
        v = self.r.randn(self.r.rows, self.k)
        if self.fmt == "fp8":
            self.x.copy_((16 * v).to(torch.float8_e4m3fn).view(torch.uint8))
            self.xs.uniform_(0.001, 0.01, generator=self.r.g)
        else:
            self.x.copy_(v)

    def run(self, **kw):
        m, r = self.moe, self.r
        more = dict(x_scales=self.xs, w_scales=self.ws) if self.fmt == "fp8" else {}
        m.moe_expert_glu(r.p, r.plan, self.op, self.x, self.w, self.h, preact=self.z, **more, **kw)
        if self.fmt == "bf16":
            m.moe_expert_glu_backward(r.p, r.plan, self.op, self.d, self.z, self.x, self.w, self.dz, self.dx, self.dw,
                                      dbias=self.db, workspace=self.work, **kw)

    def results(self):
        return [t.clone() for t in self.out]


FORMS = [("fp8", 6, 3, 2, 2176, 128), ("fp8", 900, 2, 1, 256, 1024), ("fp8", 300, 64, 6, 384, 256),
         ("bf16", 6000, 2, 1, 136, 72), ("bf16", 9, 4, 2, 2056, 40)]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_captured_and_replayed(moe, form):
    """(FP8: K in four, one tile a workgroup, tile after tile; bf16: dw in eleven parts
    joined in the workspace, K in four.)  Every replay against the eager results, bit for bit."""
    fmt, tokens, experts, top_k, k, f = form
    steps = [Step(moe, 1200 + i, tokens, experts, top_k, k, f, fmt) for i in range(2)]
    side, graphs = torch.cuda.Stream(), []
    for s in steps:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(4):
        say(f"[expert calls] {form} turn {turn}")
        for s in steps:
            s.change()
        for g in graphs:
            g.replay()
        got = [s.results() for s in steps]
        torch.cuda.synchronize()
        for s, res in zip(steps, got):
            for t in s.out:
                t.fill_(-77.0)
            s.run()
            torch.cuda.synchronize()
            for a, b in zip(res, s.results()):
                assert torch.equal(bits(a)[s.r.live] if a.shape[0] == s.r.rows else bits(a),
                                   bits(b)[s.r.live] if b.shape[0] == s.r.rows else bits(b)), (form, turn)


@pytest.mark.parametrize("form", FORMS[2:4], ids=lambda f: "-".join(map(str, f)))
def test_the_stream_given_by_hand(moe, form):
    """Work on the given stream, in its order: behind the inputs that it writes."""
    fmt, tokens, experts, top_k, k, f = form
    s = Step(moe, 1210, tokens, experts, top_k, k, f, fmt)
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    kept, side = s.x.clone(), torch.cuda.Stream()
    for turn in range(3):
        say(f"[expert calls] stream {form} turn {turn}")
        s.x.zero_()
        for t in s.out:
            t.fill_(-77.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            s.x.copy_(kept)
        s.run(stream=side)
        side.synchronize()
        for a, b in zip(s.results(), want):
            assert torch.equal(bits(a), bits(b))


def test_one_expert_twice(moe):
    """A token that names an expert twice has two rows there (the plan reports it); each
    has its own result and its own gradient."""
    say("[expert calls] one expert twice")
    n, k, f = 40, 136, 72
    r = Routed(moe, 1220, n, 5, 3)
    ids = r.ids.clone()
    ids[::3, 1] = ids[::3, 0]
    plan = moe.alloc_plan(r.p)
    moe.moe_dispatch_plan(r.p, ids, plan)
    torch.cuda.synchronize()
    assert plan.read_status() & moe.STATUS_DUP_ID
    slot = plan.slot.long()
    live = slot >= 0
    assert slot[live].unique().numel() == int(live.sum())
    tokens, wts, dout = r.randn(n, k).bfloat16(), r.randn(n, 3), r.randn(n, f).bfloat16()
    x = torch.full((r.rows, k), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[slot[live]] = tokens[:, None].expand(n, 3, k)[live]
    w, op = weights(r, 2 * f, k), moe.expert_op(k, f, "silu")
    h, z = r.sentinel(f), r.sentinel(2 * f)
    moe.moe_expert_glu(r.p, plan, op, x, w, h, preact=z)
    p = moe.problem(n, f, 3, 5, 1)  # the combine's columns are h's
    dy, dg = r.sentinel(f), torch.full((n, 3), -77.0, device="cuda")
    moe.moe_combine_backward(p, plan, h, wts, dout, dy, dg)
    torch.cuda.synchronize()
    for t in range(n):
        for j in range(3):
            if not live[t, j]:
                assert dg[t, j] == 0
                continue
            row = slot[t, j]
            _, rh, _, th = ref.forward(tokens[t:t + 1].double(), w[ids[t, j]].double(), None, True, "silu")
            assert_within(h[row:row + 1], rh, th, "h")
            assert torch.equal(bits(dy[row]), bits((wts[t, j] * dout[t].float()).bfloat16()))
            q = h[row].double() * dout[t].double()
            assert_within(dg[t, j], q.sum(), (f + 2) * ref.F32 * q.abs().sum(), "dweights")
