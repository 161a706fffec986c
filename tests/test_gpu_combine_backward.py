"""GPU: the combine's gradients in each of the kernel's forms: k that the kernel knows
at compile time (1, 2, 4, 6, 8) and any other (slots in batches of eight), a
token to a workgroup (H > 512) or to a wave.  Element by element against 64 bits; rows that
no slot names are NaN in expert_out and stay as they were in dy."""
import pytest
import torch

import expert_reference as ref
from expert_reference import assert_within
from gpu_helpers import say
from test_gpu_expert import Routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


WIDE = [dict(top_k=k, hidden=h, masked=m) for k, h, m in (
    (1, 1544, 0.2), (2, 520, 0.0), (4, 4104, 0.1), (6, 776, 0.3), (8, 520, 0.5),
    # any other k: one batch of slots, whole batches, a last one of one or three
    (3, 520, 0.2), (5, 4104, 0.0), (7, 1032, 0.1), (9, 776, 0.2), (11, 1032, 0.1), (16, 520, 0.1), (37, 648, 0.2),
    (64, 776, 0.1))]
NARROW = [dict(top_k=k, hidden=h, masked=m) for k, h, m in (
    (1, 512, 0.2), (2, 88, 0.0), (2, 512, 0.1), (4, 512, 0.2), (6, 264, 0.0), (8, 88, 0.3), (3, 512, 0.1), (9, 512, 0.2),
    (11, 8, 0.1), (64, 40, 0.2))]


@pytest.mark.parametrize("tokens", [1, 2, 131])
@pytest.mark.parametrize("c", WIDE + NARROW, ids=lambda c: f"k{c['top_k']}-h{c['hidden']}")
def test_combine_backward(moe, c, tokens):
    say(f"[combine backward] {tokens} tokens {c}")
    h, n, k = c["hidden"], tokens, c["top_k"]
    r = Routed(moe, 700 + k + h, tokens=n, experts=max(k, 5) + 3, pad=3, **c)
    y, dout, wts = r.packed(h), r.randn(n, h).bfloat16(), r.randn(n, k)
    dy, dw = r.sentinel(h), torch.full((n, k), -77.0, device="cuda")
    moe.moe_combine_backward(r.p, r.plan, y, wts, dout, dy, dw)
    torch.cuda.synchronize()
    slot = r.plan.slot.long()
    live = slot >= 0
    d64 = dout.double()[:, None, :]
    products = torch.where(live[..., None], y[slot.clamp(min=0)].double(), 0.0) * d64
    assert_within(dw, products.sum(-1), (h + 2) * ref.F32 * products.abs().sum(-1), "dweights")
    expect = torch.full_like(dy, -77.0)
    # one fp32 product, rounded once: the same bits
    expect[slot[live]] = (wts[..., None] * dout.float()[:, None, :])[live].bfloat16()
    assert torch.equal(dy.view(torch.int16), expect.view(torch.int16))
    # without the gradient of the weights: the same rows
    alone = r.sentinel(h)
    moe.moe_combine_backward(r.p, r.plan, None, wts, dout, alone)
    torch.cuda.synchronize()
    assert torch.equal(alone.view(torch.int16), expect.view(torch.int16))
