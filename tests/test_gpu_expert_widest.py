"""GPU: the widest layers that the experts' calls accept: 2^20 columns of x or of the
result (rows of up to 4 MiB), and an expert's weights of 2 GiB less a few rows, where
byte offsets come near 2^31.  Last rows, last columns and a sample between, against
64 bits, with the bounds of expert_reference.py."""
import pytest
import torch

import expert_reference as ref
from expert_reference import assert_within
from gpu_helpers import say
from test_gpu_expert import Routed

pytestmark = pytest.mark.gpu

# many rows and few (K in four), wide on either side, and both wide; rows past one tile
CASES = [dict(tokens=300, experts=2, k=1 << 20, f=8), dict(tokens=5, experts=2, k=1 << 20, f=8),
         dict(tokens=300, experts=2, k=8, f=1 << 20), dict(tokens=3, experts=1, k=8, f=1 << 20),
         dict(tokens=300, experts=1, k=16384, f=32760), dict(tokens=9, experts=1, k=16384, f=32760),
         dict(tokens=300, experts=1, k=32760, f=16384)]


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


def sample(g, n):
    """Columns: the first 16, the last 80, and 32 between."""
    some = torch.randint(0, n, (32,), generator=g, device="cuda")
    return torch.cat([torch.arange(min(16, n), device="cuda"), some, torch.arange(max(n - 80, 0), n, device="cuda")]).unique()


@pytest.mark.parametrize("i", range(len(CASES)))
def test_the_widest(moe, i):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    c = CASES[i]
    say(f"[expert widest] {c}")
    r = Routed(moe, 1100 + i, c["tokens"], c["experts"], 1, hidden=8)
    k, f, e = c["k"], c["f"], c["experts"]

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=r.g)

    op = moe.expert_op(k, f, "silu")
    assert moe.moe_check_expert_op(r.p, op) == 0
    x, w, d = normal(r.rows, k), normal(e, 2 * f, k, std=k ** -0.5), normal(r.rows, f)

    def unwritten(*shape, dtype=torch.bfloat16):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    h, z = unwritten(r.rows, f), unwritten(r.rows, 2 * f)
    moe.moe_expert_glu(r.p, r.plan, op, x, w, h, preact=z)
    dz, dx, dw = unwritten(r.rows, 2 * f), unwritten(r.rows, k), unwritten(e, 2 * f, k)
    db = unwritten(e, 2 * f, dtype=torch.float32)
    moe.moe_expert_glu_backward(r.p, r.plan, op, d, z, x, w, dz, dx, dw, dbias=db, workspace=moe.alloc_expert_workspace(r.p, op))
    torch.cuda.synchronize()
    cols, ks = sample(r.g, f), sample(r.g, k)
    both = torch.cat([cols, cols + f])
    for n, (a, b) in enumerate(r.ranges):
        if a == b:
            continue
        rz, rh, tz, th = ref.forward(x[a:b].double(), w[n][both].double(), None, True, "silu")
        assert_within(z[a:b][:, both], rz, tz, f"z of expert {n}")
        assert_within(h[a:b][:, cols], rh, th, f"h of expert {n}")
        rdz, tol = ref.grad(d[a:b][:, cols].double(), z[a:b][:, both].double(), True, "silu")
        assert_within(dz[a:b][:, both], rdz, tol + ref.BF16 * (rdz.abs() + tol), f"dz of expert {n}")
        assert_within(db[n][both], rdz.sum(0), tol.sum(0) + (b - a + 2) * ref.F32 * rdz.abs().sum(0), f"dbias of expert {n}")
        used = dz[a:b].double()  # the products read the rounded dz
        wk = w[n][:, ks].double()
        assert_within(dx[a:b][:, ks], used @ wk, ref.product_bound(used, wk, 2 * f), f"dx of expert {n}")
        u, xk = used[:, both].T, x[a:b][:, ks].double()
        assert_within(dw[n][both][:, ks], u @ xk, ref.product_bound(u, xk, b - a), f"dw of expert {n}")
    for out in (h, z, dz, dx, dw, db):  # written whole
        assert not bool(torch.isnan(out).any())
    say("[expert widest] done")
