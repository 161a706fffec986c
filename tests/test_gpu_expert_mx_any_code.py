"""GPU: FP8 rows whose codes lie from 2^-9 to 448 beside each other, with MX-FP4 weights: no product is cut,
in each of the four tiles (bound, and proof that a cut would pass it: any_code_reference.py)."""
import pytest
import torch

import any_code_reference as any_code
import expert_reference as ref
from expert_reference import assert_within
from gpu_helpers import say
from test_gpu_expert import Routed
from test_gpu_expert_mx import mx_value

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


@pytest.mark.parametrize("c", any_code.CASES, ids=lambda c: any_code.tile(**c) + f", {c['k']}")
def test_no_product_is_cut(moe, c):
    say(f"[expert mx] any code {c}")
    r = Routed(moe, 900 + c["k"], c["tokens"], c["experts"], 1)
    k, f = c["k"], c["f"]
    x, xs, w, ws = (t.cuda() for t in any_code.inputs(c, r.rows))
    y, rest, op = r.sentinel(f), r.sentinel(f), moe.expert_op(k, f, fmt="fp8")
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, y)
    # with -y for the residual: what the rounding took off, so that the sum itself is seen
    moe.moe_expert_linear_mx(r.p, r.plan, op, x, xs, w, ws, rest, residual=-y)
    for e, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        X, W = ref.dequant_rows(x[a:b], xs[a:b]), mx_value(w[e], ws[e])
        z, tol = X @ W.T, any_code.BOUND * (X.abs() @ W.abs().T)
        assert_within(y[a:b], z, tol + ref.BF16 * (z.abs() + tol), f"y of expert {e}")
        left = z - y[a:b].double()
        assert_within(rest[a:b], left, tol + ref.F32 * z.abs() + ref.BF16 * (left.abs() + tol), f"rest of expert {e}")
