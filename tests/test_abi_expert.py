"""The experts' entry points and the combine's backward pass refuse malformed
calls on the host (no GPU work: every call here returns before anything is
launched), and the sizes they report."""
import ctypes
import os

import pytest

ref = ctypes.byref
FAKE = 1 << 20  # never dereferenced: every call fails its checks first
EINVAL, EALIGN, EOVERFLOW = -1, -2, -3


@pytest.fixture(scope="module")
def moe():
    from combine_topk_ids_amd import _build
    if not os.path.exists(_build.LIB):
        _build.build(force=False)
    import combine_topk_ids_amd.moe as m
    return m


def full_plan(moe):
    return moe.Plan(*([FAKE] * 7))


@pytest.mark.parametrize("field,value,code", [
    ("in_dim", 0, EINVAL), ("in_dim", -8, EINVAL), ("in_dim", 12, EINVAL), ("out_dim", 0, EINVAL),
    ("out_dim", 4, EINVAL), ("act", -1, EINVAL), ("act", 4, EINVAL), ("fmt", 2, EINVAL), ("fmt", 3, EINVAL),
    ("fmt", 7, EINVAL), ("in_dim", 1 << 21, EOVERFLOW), ("out_dim", 1 << 21, EOVERFLOW),
])
def test_malformed_ops(moe, field, value, code):
    p, op, pl = moe.problem(64, 256, 2, 8, 4), moe.expert_op(256, 128, "silu"), full_plan(moe)
    assert moe.moe_check_expert_op(p, op) == 0
    setattr(op, field, value)
    assert moe.moe_check_expert_op(p, op) == code
    assert moe.moe_expert_workspace_bytes(p, op) == 0
    with pytest.raises(moe.MoeError):
        moe.alloc_expert_workspace(p, op)
    glu, lin = moe.lib.moe_expert_glu, moe.lib.moe_expert_linear
    assert glu(ref(p), ref(pl), ref(op), *[FAKE] * 7, None) == code
    assert lin(ref(p), ref(pl), ref(op), *[FAKE] * 8, None) == code
    for back in (moe.lib.moe_expert_glu_backward, moe.lib.moe_expert_linear_backward):
        assert back(ref(p), ref(pl), ref(op), *[FAKE] * 9, None) == code


def test_sizes_too_large_for_the_offsets(moe):
    p = moe.problem(64, 256, 2, 8, 4)
    assert moe.moe_check_expert_op(p, moe.expert_op(16384, 32768 - 8)) == 0
    assert moe.moe_check_expert_op(p, moe.expert_op(16384, 32768)) == EOVERFLOW  # in * out = 2^29
    # many rows of a wide layer: more workgroups than a launch may have
    big = moe.problem(1 << 22, 64, 8, 8, 8)
    assert moe.moe_check_expert_op(big, moe.expert_op(64, 64)) == 0
    assert moe.moe_check_expert_op(big, moe.expert_op(8192, 8192)) == EOVERFLOW


def test_an_invalid_problem_is_refused_first(moe):
    p, op = moe.problem(64, 256, 2, 8, 4), moe.expert_op(256, 128)
    p.top_k = 9
    assert moe.moe_check_expert_op(p, op) == EINVAL
    assert moe.lib.moe_combine_backward(ref(p), ref(full_plan(moe)), *[FAKE] * 5, None) == EINVAL
    assert moe.moe_check_expert_op(moe.problem(64, 256, 2, 8, 4), op) == 0
    assert moe.lib.moe_check_expert_op(None, ref(op)) == EINVAL
    assert moe.lib.moe_check_expert_op(ref(moe.problem(64, 256, 2, 8, 4)), None) == EINVAL


def test_workspace_holds_the_column_sums(moe):
    """One row of 2 * out_dim fp32 sums for every 16-row chunk of every expert: an
    expert's n rows touch at most n / 16 + 1 chunks."""
    p, op = moe.problem(1000, 256, 3, 8, 4, pad_multiple=16), moe.expert_op(256, 72)
    need = (moe.moe_max_rows(p) // 16 + 8) * 2 * 72 * 4
    got = moe.moe_expert_workspace_bytes(p, op)
    assert need <= got <= need + 4096 and got % 256 == 0
    # few weights and many rows: dw's parts too, 2 experts x 144 x 136 of fp32, 16 of them
    p, op = moe.problem(20000, 64, 1, 2, 1), moe.expert_op(136, 72)
    need = (moe.moe_max_rows(p) // 16 + 2) * 2 * 72 * 4 + 16 * 2 * 144 * 136 * 4
    assert need <= moe.moe_expert_workspace_bytes(p, op) <= need + 4096


def test_forward_refusals(moe):
    p, pl = moe.problem(64, 256, 2, 8, 4), full_plan(moe)
    glu, lin = moe.lib.moe_expert_glu, moe.lib.moe_expert_linear
    op, op8 = moe.expert_op(256, 128, "silu"), moe.expert_op(256, 128, "silu", "fp8")

    def g(plan=pl, o=op, x=FAKE, xs=None, w=FAKE, ws=None, b=None, h=FAKE, z=None):
        return glu(ref(p), ref(plan), ref(o), x, xs, w, ws, b, h, z, None)

    def f(plan=pl, o=op, x=FAKE, xs=None, w=FAKE, ws=None, b=None, r=None, y=FAKE, z=None):
        return lin(ref(p), ref(plan), ref(o), x, xs, w, ws, b, r, y, z, None)

    for call, out in ((g, "h"), (f, "y")):
        for missing in ("x", "w", out):
            assert call(**{missing: None}) == EINVAL, missing
        # scales with bf16, none with FP8
        assert call(xs=FAKE) == EINVAL and call(ws=FAKE) == EINVAL
        assert call(o=op8) == EINVAL and call(o=op8, xs=FAKE) == EINVAL and call(o=op8, ws=FAKE) == EINVAL
        for name in ("x", "w", "b", "z", out):
            assert call(**{name: FAKE + 8}) == EALIGN, name
        assert call(o=op8, xs=FAKE + 2, ws=FAKE) == EALIGN
        for hole in (0, 1):  # counts, offsets
            fields = [FAKE] * 7
            fields[hole] = 0
            assert call(plan=moe.Plan(*fields)) == EINVAL
        # FP8 needs whole scale blocks
        assert call(o=moe.expert_op(256, 64, "silu", "fp8"), xs=FAKE, ws=FAKE) == EINVAL
        assert call(o=moe.expert_op(192, 128, "silu", "fp8"), xs=FAKE, ws=FAKE) == EINVAL
    assert f(r=FAKE + 8) == EALIGN
    assert glu(ref(p), None, ref(op), FAKE, None, FAKE, None, None, FAKE, None, None) == EINVAL


def test_backward_refusals(moe):
    p, pl = moe.problem(64, 256, 2, 8, 4), full_plan(moe)
    op, none = moe.expert_op(256, 128, "silu"), moe.expert_op(256, 128, "none")
    names = ("dy", "z", "x", "w", "dz", "dx", "dw", "db", "ws")

    def call(fn, o=op, **given):
        v = {n: FAKE for n in names}
        v.update(given)
        return fn(ref(p), ref(pl), ref(o), *[v[n] for n in names], None)

    glu, lin = moe.lib.moe_expert_glu_backward, moe.lib.moe_expert_linear_backward
    for fn in (glu, lin):
        assert call(fn, moe.expert_op(256, 128, "silu", "fp8")) == EINVAL  # forward passes only
        for missing in ("dy", "z", "dz"):
            assert call(fn, **{missing: None}) == EINVAL, missing
        assert call(fn, x=None) == EINVAL  # dw needs the rows
        assert call(fn, w=None) == EINVAL  # dx needs the weights
        # dw and dbias need the workspace
        assert call(fn, ws=None, dw=None) == EINVAL and call(fn, ws=None, db=None) == EINVAL
        for n in names:
            assert call(fn, **{n: FAKE + 2}) == EALIGN, n
    # without activation dz is dy: neither a kept z nor a dz of its own
    assert call(lin, none) == EINVAL
    assert call(lin, none, z=None) == EINVAL and call(lin, none, dz=None) == EINVAL


def test_combine_backward_refusals(moe):
    p, pl = moe.problem(64, 256, 2, 8, 4), full_plan(moe)
    names = ("y", "w", "dout", "dy", "dw")

    def call(plan=pl, **given):
        v = {n: FAKE for n in names}
        v.update(given)
        return moe.lib.moe_combine_backward(ref(p), ref(plan), *[v[n] for n in names], None)

    assert call(y=None) == EINVAL  # dweights needs the rows
    assert call(w=None) == EINVAL  # no gradient of weights the combine did not take
    assert call(dout=None) == EINVAL and call(dy=None) == EINVAL
    fields = [FAKE] * 7
    fields[4] = 0
    assert call(plan=moe.Plan(*fields)) == EINVAL  # slots
    for n in ("y", "dout", "dy"):
        assert call(**{n: FAKE + 8}) == EALIGN
    assert call(w=FAKE + 2) == EALIGN and call(dw=FAKE + 2) == EALIGN


def test_host_tensors_are_refused(moe):
    torch = pytest.importorskip("torch")
    p, op = moe.problem(4, 64, 1, 2, 1), moe.expert_op(64, 64, "silu")
    plan = moe.alloc_plan(p, device="cpu")
    t = torch.zeros(4096 * 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_expert_glu(p, plan, op, t, t, t)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_expert_linear(p, plan, op, t, t, t)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_expert_linear_backward(p, plan, op, t, t, t, t, t, preact=t, dz=t)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_combine_backward(p, plan, t, torch.zeros(4), t, t)
