"""Routing, MX-FP4 quantisation and the products with MX-FP4 weights refuse malformed calls on
the host (no GPU work: every call here returns before anything is launched)."""
import ctypes
import os

import pytest

ref = ctypes.byref
FAKE = 1 << 20  # never dereferenced: every call fails its checks first
OK, EINVAL, EALIGN, EOVERFLOW = 0, -1, -2, -3


@pytest.fixture(scope="module")
def moe():
    from combine_topk_ids_amd import _build
    if not os.path.exists(_build.LIB):
        _build.build(force=False)
    import combine_topk_ids_amd.moe as m
    return m


def full_plan(moe):
    return moe.Plan(*([FAKE] * 7))


@pytest.mark.parametrize("field,value", [
    ("score", 2), ("score", -1), ("logits", 2), ("n_groups", 0), ("n_groups", 3), ("n_groups", 16), ("top_groups", 0),
    ("top_groups", 5), ("top_groups", 1), ("group_top", 0), ("group_top", 3), ("renormalize", 2),
    ("scale", float("nan")), ("scale", float("inf"))])
def test_malformed_routers(moe, field, value):
    p = moe.problem(16, 8, 3, 8, 1)
    r = moe.router("sigmoid", n_groups=4, top_groups=2, group_top=2)
    assert moe.moe_check_router(p, r) == OK
    setattr(r, field, value)  # (one group of two holds fewer than k = 3)
    assert moe.moe_check_router(p, r) == EINVAL
    assert moe.lib.moe_route(ref(p), ref(r), *[FAKE] * 5, None) == EINVAL
    assert moe.lib.moe_route_backward(ref(p), ref(r), *[FAKE] * 5, None) == EINVAL


def test_route_refusals(moe):
    p, r = moe.problem(16, 8, 3, 8, 1), moe.router()
    assert moe.lib.moe_check_router(ref(p), None) == EINVAL
    bad = moe.problem(16, 8, 9, 8, 1)
    assert moe.moe_check_router(bad, r) == EINVAL

    def fwd(*a):
        return moe.lib.moe_route(ref(p), ref(r), *a, None)

    def bwd(*a):
        return moe.lib.moe_route_backward(ref(p), ref(r), *a, None)

    assert fwd(None, None, FAKE, FAKE, None) == EINVAL
    assert fwd(FAKE, None, None, FAKE, None) == EINVAL
    for i in range(5):
        assert fwd(*[FAKE + 2 if j == i else FAKE for j in range(5)]) == EALIGN
    assert bwd(None, FAKE, FAKE, FAKE, FAKE) == EINVAL
    assert bwd(FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert bwd(FAKE, FAKE, None, None, FAKE) == EINVAL  # nothing to go back from
    assert bwd(FAKE, None, FAKE, FAKE, FAKE) == EINVAL  # weights' gradients without their IDs
    for i in range(5):
        assert bwd(*[FAKE + 2 if j == i else FAKE for j in range(5)]) == EALIGN
    r.logits = 1  # bf16: two bytes will do for logits and their gradient
    assert fwd(FAKE + 1, None, FAKE, FAKE, None) == EALIGN
    assert bwd(FAKE, FAKE, FAKE, FAKE, FAKE + 1) == EALIGN


def test_quantize_refusals(moe):
    q = moe.lib.moe_quantize_mxfp4
    assert q(-1, 32, FAKE, FAKE, FAKE, None) == EINVAL
    assert q(1, 0, FAKE, FAKE, FAKE, None) == EINVAL
    assert q(1, -32, FAKE, FAKE, FAKE, None) == EINVAL
    assert q(1, 48, FAKE, FAKE, FAKE, None) == EINVAL
    assert q(1 << 41, 32, FAKE, FAKE, FAKE, None) == EOVERFLOW
    for i in range(3):
        assert q(4, 32, *[None if j == i else FAKE for j in range(3)], None) == EINVAL
    assert q(4, 32, FAKE + 8, FAKE, FAKE, None) == EALIGN
    assert q(4, 32, FAKE, FAKE + 4, FAKE, None) == EALIGN
    assert q(0, 32, None, None, None, None) == OK  # nothing to do


@pytest.mark.parametrize("field,value,code", [
    ("in_dim", 0, EINVAL), ("in_dim", -32, EINVAL), ("in_dim", 48, EINVAL), ("out_dim", 0, EINVAL), ("out_dim", 12, EINVAL),
    ("act", -1, EINVAL), ("act", 4, EINVAL), ("fmt", 0, EINVAL), ("fmt", 3, EINVAL), ("in_dim", 1 << 21, EOVERFLOW),
    ("out_dim", 1 << 21, EOVERFLOW)])
def test_malformed_mx_ops(moe, field, value, code):
    p, op, pl = moe.problem(64, 256, 2, 8, 4), moe.expert_op(256, 128, "silu", "mxfp4"), full_plan(moe)
    assert moe.moe_check_expert_mx_op(p, op) == OK
    setattr(op, field, value)
    assert moe.moe_check_expert_mx_op(p, op) == code
    assert moe.lib.moe_expert_glu_mx(ref(p), ref(pl), ref(op), *[FAKE] * 7, None) == code
    assert moe.lib.moe_expert_linear_mx(ref(p), ref(pl), ref(op), *[FAKE] * 7, None) == code


def test_mx_sizes(moe):
    p = moe.problem(64, 256, 2, 8, 4)
    check = moe.moe_check_expert_mx_op
    assert check(p, moe.expert_op(32, 8, fmt="mxfp4")) == OK
    assert check(p, moe.expert_op(160, 8, fmt="fp8")) == EINVAL  # FP8 rows: whole 128-value blocks
    assert check(p, moe.expert_op(128, 8, fmt="fp8")) == OK
    assert check(p, moe.expert_op(16384, 32768, fmt="mxfp4")) == EOVERFLOW
    assert moe.lib.moe_check_expert_mx_op(None, ref(moe.expert_op(32, 8, fmt="mxfp4"))) == EINVAL
    assert moe.lib.moe_check_expert_mx_op(ref(p), None) == EINVAL
    bad = moe.problem(64, 256, 9, 8, 4)
    assert check(bad, moe.expert_op(32, 8, fmt="mxfp4")) == EINVAL


def test_mx_argument_refusals(moe):
    p, pl = moe.problem(64, 256, 2, 8, 4), full_plan(moe)
    op = moe.expert_op(256, 128, "silu", "mxfp4")

    def glu(*a, op=op, plan=pl):
        return moe.lib.moe_expert_glu_mx(ref(p), ref(plan) if plan else None, ref(op), *a, None)

    def lin(*a, op=op):
        return moe.lib.moe_expert_linear_mx(ref(p), ref(pl), ref(op), *a, None)

    # x, x_scales, w, w_scales, bias, h, h_scales
    for i in (0, 1, 2, 3, 5):
        assert glu(*[None if j == i else FAKE for j in range(7)]) == EINVAL
    for i, off in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 8), (5, 8)):
        assert glu(*[FAKE + off if j == i else FAKE for j in range(7)]) == EALIGN
    assert glu(*[FAKE] * 7, plan=None) == EINVAL
    for field in ("expert_counts", "expert_offsets"):
        part = full_plan(moe)
        setattr(part, field, None)
        assert glu(*[FAKE] * 7, plan=part) == EINVAL
    # a quantised result has whole blocks
    assert glu(*[FAKE] * 7, op=moe.expert_op(256, 72, "silu", "mxfp4")) == EINVAL
    # x, x_scales, w, w_scales, bias, residual, y
    for i in (0, 1, 2, 3, 6):
        assert lin(*[None if j == i else FAKE for j in range(7)]) == EINVAL
    for i, off in ((0, 8), (1, 2), (2, 8), (3, 2), (4, 8), (5, 8), (6, 8)):
        assert lin(*[FAKE + off if j == i else FAKE for j in range(7)]) == EALIGN


def test_binding_refusals(moe):
    """Tensors on the host, of another type or too small never reach the library."""
    import torch
    p, r = moe.problem(4, 8, 2, 8, 1), moe.router()
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_route(p, r, f, i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_route_backward(p, r, f, i, f, dweights=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_quantize_mxfp4(torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.uint8),
                               torch.zeros(2, dtype=torch.uint8))
