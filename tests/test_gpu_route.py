"""GPU: routing and its gradient against the 64-bit references, element by element (the
choices exactly, weights and gradients within bounds derived in more_reference.py)."""
import numpy as np
import pytest
import torch

import more_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8  # half a step


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


# tokens, experts, k, groups, groups kept
SIZES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 5, 5, 1, 1), (7, 64, 8, 1, 1), (130, 60, 3, 1, 1), (65, 128, 8, 1, 1),
         (33, 256, 8, 8, 4), (20, 256, 16, 4, 1), (9, 256, 17, 1, 1), (5, 257, 5, 1, 1), (4, 300, 20, 10, 3),
         (3, 512, 8, 16, 2), (2, 1024, 64, 32, 4), (40, 72, 6, 9, 2), (50, 12, 4, 12, 5), (3, 1000, 10, 1, 1),
         (6, 1024, 1, 1024, 1), (17, 130, 7, 2, 1), (300, 16, 4, 4, 2), (21, 6, 2, 3, 3), (70, 250, 12, 25, 20)]


def router(moe, r):
    return moe.router(r["score"], r.get("logits", "fp32"), r.get("n_groups", 1), r.get("top_groups", 1),
                      r.get("group_top", 1), r.get("renormalize", True), r.get("scale", 1.0))


def make_logits(rng, n, e, kind):
    l = rng.standard_normal((n, e)).astype(np.float32)
    if kind == "ties":
        l = np.round(l * 2) / 2
    elif kind == "masked":
        l = np.round(l * 4) / 4
        l[rng.random((n, e)) < 0.4] = -np.inf
        l[rng.random(n) < 0.3] = -np.inf
    elif kind == "wide":
        l *= 20
    return l


def to_type(l, kind):
    t = torch.from_numpy(np.ascontiguousarray(l)).cuda()
    return t.bfloat16() if kind == "bf16" else t


def run(moe, l, r, k, bias=None, scores=False):
    n, e = l.shape
    p = moe.problem(n, 8, k, e, 1)
    ids = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), -7.0, device="cuda")
    s = torch.full((n, e), -7.0, device="cuda") if scores else None
    moe.moe_route(p, router(moe, r), l, ids, w, bias=bias, scores=s)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), None if s is None else s.cpu().numpy()


def check_close(got, want, tol, what):
    with np.errstate(invalid="ignore"):
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs differ"
        err = np.abs(np.where(np.isnan(want), 0, got.astype(np.float64) - want))
        assert (err <= np.where(np.isnan(tol), 0, tol)).all(), f"{what}: {np.nanmax(err / tol)} of the bound"


@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "wide"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_forward(moe, i, kind):
    n, e, k, groups, kept = SIZES[i]
    rng = np.random.default_rng(100 * i + len(kind))
    for j, (score, logits, with_bias) in enumerate([("softmax", "fp32", False), ("sigmoid", "fp32", True),
                                                    ("softmax", "bf16", True), ("sigmoid", "bf16", False)]):
        r = dict(score=score, logits=logits, n_groups=groups, top_groups=kept, group_top=1 + (i + j) % 2,
                 renormalize=(i + j) % 3 > 0, scale=(1.0, 2.5)[j % 2])
        say(f"[route] {n} x {e}, k {k}, {kind}, bias {with_bias}, {r}")
        t = to_type(make_logits(rng, n, e, kind), logits)
        l = t.float().cpu().numpy()
        bias = None
        if with_bias:
            b = (0.2 * rng.standard_normal(e)).astype(np.float32)
            if kind == "masked":
                b[rng.random(e) < 0.1] = -np.inf
            bias = torch.from_numpy(b).cuda()
        ids, w, s = run(moe, t, r, k, bias, scores=j % 2 == 0)
        want = ref.choose(l, None if bias is None else b, r, k)
        assert np.array_equal(ids, want), (ids[(ids != want).any(1)][:3], want[(ids != want).any(1)][:3])
        check_close(w, *ref.gates(l, ids, r), "weights")
        if s is not None:
            rs = ref.scores(l, score)
            arg = np.abs(np.where(np.isfinite(l), l, 0)).max(1, keepdims=True)
            check_close(s, rs, (e + 10 + 4 * arg) * ref.F32 * np.abs(rs) + 2.0 ** -125, "scores")


def test_without_weights(moe):
    """The IDs alone, and the same as with the rest."""
    t = torch.randn(50, 40, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    r = dict(score="softmax")
    ids = torch.zeros(50, 4, dtype=torch.int32, device="cuda")
    moe.moe_route(moe.problem(50, 8, 4, 40, 1), router(moe, r), t, ids, None)
    assert np.array_equal(ids.cpu().numpy(), run(moe, t, r, 4)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k", [(64, 16), (256, 8), (700, 30)])
def test_order_finer_than_fp32(moe, score, e, k):
    """Keys that fp32 scores cannot tell apart: neighbouring fp32 logits, and with a bias a hair
    (2^-40 of it and less) between the keys."""
    rng = np.random.default_rng(e)
    n = 24
    step = np.stack([rng.permutation(e) for _ in range(n)])
    l = (1.0 + step * 2.0 ** -23).astype(np.float32)
    order = np.argsort(-step, axis=1)[:, :k]
    ids, _, _ = run(moe, torch.from_numpy(l).cuda(), dict(score=score), k)
    assert np.array_equal(ids, order)
    bias = torch.full((e,), 0.375, device="cuda")
    ids, _, _ = run(moe, torch.from_numpy(l).cuda(), dict(score=score), k, bias)
    assert np.array_equal(ids, order)
    # biases that cancel the scores up to their rounding to fp32
    l = rng.standard_normal((1, e)).astype(np.float32)
    b = (0.5 - ref.scores(l, score)[0]).astype(np.float32)
    want = ref.choose(l, b, dict(score=score), k)
    ids, _, _ = run(moe, torch.from_numpy(l).cuda(), dict(score=score), k, torch.from_numpy(b).cuda())
    assert np.array_equal(ids, want)


def test_groups_finer_than_fp32(moe):
    """Sums of two that fp32 cannot tell apart decide between groups."""
    rng = np.random.default_rng(8)
    n, groups, each = 40, 8, 32
    l = rng.standard_normal((n, groups, each)).astype(np.float32) - 3
    step = np.stack([rng.permutation(groups) for _ in range(n)])
    l[:, :, 5] = 1.0
    l[:, :, 9] = 1.0 + step * 2.0 ** -23
    l = l.reshape(n, -1)
    for score in ("sigmoid", "softmax"):
        for bias in (None, np.full(groups * each, 0.25, dtype=np.float32)):
            r = dict(score=score, n_groups=groups, top_groups=3, group_top=2)
            ids, _, _ = run(moe, torch.from_numpy(l).cuda(), r, 6, None if bias is None else torch.from_numpy(bias).cuda())
            assert np.array_equal(ids, ref.choose(l, bias, r, 6))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_nan_and_infinite_logits(moe, score, with_bias):
    """A NaN ranks first and shows in its own token's weights only."""
    rng = np.random.default_rng(9)
    l = rng.standard_normal((12, 48)).astype(np.float32)
    clean = l.copy()
    l[1, 30] = np.nan
    l[3, [40, 7]] = np.nan
    l[5] = np.nan
    l[7, 11] = -np.nan
    l[9, 20] = np.inf
    b = (0.1 * rng.standard_normal(48)).astype(np.float32) if with_bias else None
    bias = None if b is None else torch.from_numpy(b).cuda()
    r = dict(score=score, n_groups=4, top_groups=2, group_top=2)
    ids, w, s = run(moe, torch.from_numpy(l).cuda(), r, 5, bias, scores=True)
    assert np.array_equal(ids, ref.choose(l, b, r, 5))
    bad = [1, 3, 5, 7] + [9] * (score == "softmax")
    for t in range(12):
        assert np.isnan(w[t]).any() == (t in bad), t
        assert np.isnan(s[t]).any() == (t in bad), t
    ids0, w0, s0 = run(moe, torch.from_numpy(clean).cuda(), r, 5, bias, scores=True)
    good = [t for t in range(12) if t not in (1, 3, 5, 7, 9)]
    assert np.array_equal(ids[good], ids0[good]) and np.array_equal(w[good], w0[good])
    assert np.array_equal(s[good], s0[good])


def test_far_logits(moe):
    """Scores that leave fp32's range: weights stay those of the chosen ones."""
    l = np.array([[-200.0, -201, -500, -1e30], [1e30, 3, 2, 1], [3e38, 3e38, -3e38, 0], [-90, -91, -92, -93],
                  [95, 94, -95, -94]], dtype=np.float32)
    for r in (dict(score="softmax"), dict(score="softmax", renormalize=False), dict(score="sigmoid", renormalize=False)):
        ids, w, _ = run(moe, torch.from_numpy(l).cuda(), r, 2)
        assert np.array_equal(ids, ref.choose(l, None, r, 2))
        check_close(w, *ref.gates(l, ids, r), "weights")
    # sigmoid scores that are zero in fp32: weights of 0, and no NaN
    ids, w, _ = run(moe, torch.from_numpy(l).cuda(), dict(score="sigmoid"), 2)
    assert ids.tolist() == [[0, 1], [0, 1], [0, 1], [0, 1], [0, 1]]
    assert (w[0] == 0).all() and not np.isnan(w).any() and abs(w[4].sum() - 1) < 1e-6


@pytest.mark.parametrize("e", [37, 64, 256])
def test_rows_that_start_anywhere(moe, e):
    """Logits, scores and gradients whose rows start on no whole vector."""
    n, k = 9, 3
    g = torch.Generator("cuda").manual_seed(e)
    base = torch.randn(n * e + 3, generator=g, device="cuda")
    for off in (1, 2, 3):
        for kind in ("fp32", "bf16"):
            flat = base if kind == "fp32" else base.bfloat16()
            l = flat[off:off + n * e].view(n, e)
            r = dict(score="softmax", logits=kind)
            a = run(moe, l, r, k, scores=True)
            b = run(moe, l.clone(), r, k, scores=True)
            for x, y in zip(a, b):
                assert np.array_equal(x, y)


# ---- the gradient -------------------------------------------------------------------


def run_backward(moe, l, ids, r, dw, ds):
    n, e = l.shape
    p = moe.problem(n, 8, ids.shape[1], e, 1)
    dl = torch.full_like(l, -7.0)
    moe.moe_route_backward(p, router(moe, r), l, torch.from_numpy(ids).cuda(), dl,
                           dweights=None if dw is None else torch.from_numpy(dw).cuda(),
                           dscores=None if ds is None else torch.from_numpy(ds).cuda())
    torch.cuda.synchronize()
    return dl.float().cpu().numpy()


@pytest.mark.parametrize("kind", ["plain", "masked", "wide"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_backward(moe, i, kind):
    n, e, k, _, _ = SIZES[i]
    rng = np.random.default_rng(1000 * i + len(kind))
    for j, (score, logits, renormalize, given) in enumerate([
            ("softmax", "fp32", True, "both"), ("sigmoid", "fp32", True, "weights"), ("softmax", "bf16", False, "both"),
            ("sigmoid", "bf16", False, "both"), ("softmax", "fp32", True, "weights"), ("softmax", "fp32", False, "weights"),
            ("sigmoid", "fp32", False, "weights"), ("softmax", "fp32", True, "scores"), ("sigmoid", "bf16", True, "both")]):
        r = dict(score=score, logits=logits, renormalize=renormalize, scale=(1.0, 2.5)[j % 2])
        say(f"[route backward] {n} x {e}, k {k}, {kind}, {given}, {r}")
        t = to_type(make_logits(rng, n, e, kind), logits)
        l = t.float().cpu().numpy()
        ids = ref.choose(l, None, r, k)
        if kind == "plain":
            ids[rng.random((n, k)) < 0.2] = -1
        dw = rng.standard_normal((n, k)).astype(np.float32) if given != "scores" else None
        ds = rng.standard_normal((n, e)).astype(np.float32) if given != "weights" else None
        got = run_backward(moe, t, ids, r, dw, ds)
        want, tol = ref.route_gradient(l, ids, dw, ds, r)
        if logits == "bf16":
            tol = tol + BF16 * (np.abs(want) + tol)
        check_close(got, want, tol, "dlogits")


def test_backward_of_odd_ids(moe):
    """IDs that repeat within a token count each time; IDs outside [0, E) and their dweights (NaN
    here) are left out."""
    rng = np.random.default_rng(4)
    n, e, k = 20, 40, 6
    l = rng.standard_normal((n, e)).astype(np.float32)
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    ids[:, 3] = ids[:, 0]
    ids[4:8] = 11
    ids[9, 1], ids[10, 2], ids[11, 5] = e, -5, 2 ** 31 - 1
    dw, ds = rng.standard_normal((n, k)).astype(np.float32), rng.standard_normal((n, e)).astype(np.float32)
    nan = dw.copy()
    nan[9, 1] = nan[10, 2] = nan[11, 5] = np.nan
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            r = dict(score=score, renormalize=renormalize)
            want, tol = ref.route_gradient(l, ids, dw, ds, r)
            check_close(run_backward(moe, torch.from_numpy(l).cuda(), ids, r, nan, ds), want, tol, str(r))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(moe, score):
    """Forward and backward together: differences of the kernel's own weights and scores (fp32:
    2^-21 of them, over steps of 2^-6; third derivatives below 10 add 2^-12 / 6 of that)."""
    g = torch.Generator("cuda").manual_seed(6)
    n, e, k, h = 5, 24, 4, 2.0 ** -6
    l = torch.randn(n, e, generator=g, device="cuda")
    dw, ds = torch.randn(n, k, generator=g, device="cuda"), torch.randn(n, e, generator=g, device="cuda")
    r = dict(score=score)
    ids = run(moe, l, r, k)[0]
    got = run_backward(moe, l, ids, r, dw.cpu().numpy(), ds.cpu().numpy())

    def loss(l):
        i, w, s = run(moe, l, r, k, scores=True)
        # the choice's order may change; its members may not
        at = np.argsort(i, axis=1), np.argsort(ids, axis=1)
        assert np.array_equal(np.take_along_axis(i, at[0], 1), np.take_along_axis(ids, at[1], 1))
        w = np.take_along_axis(w, at[0], 1).astype(np.float64)
        return (w * np.take_along_axis(dw.cpu().numpy(), at[1], 1)).sum(1) + (s.astype(np.float64) * ds.cpu().numpy()).sum(1)

    # chosen experts well above the rest, so that a step keeps the choice
    for t in range(n):
        l[t, torch.from_numpy(ids[t]).long().cuda()] += 1.0
    got = run_backward(moe, l, ids, r, dw.cpu().numpy(), ds.cpu().numpy())
    for i in range(e):
        up, down = l.clone(), l.clone()
        up[:, i] += h
        down[:, i] -= h
        d = (loss(up) - loss(down)) / (2 * h)
        assert np.allclose(d, got[:, i], rtol=0, atol=30 * 2.0 ** -21 / h + 10 * h * h / 6 * 30)


def test_many_tokens(moe):
    """More tokens than a launch has groups of lanes: each alone gives the same bits."""
    n, e, k = 70001, 64, 4
    g = torch.Generator("cuda").manual_seed(2)
    l = torch.randn(n, e, generator=g, device="cuda").bfloat16()
    r = dict(score="sigmoid", logits="bf16")
    ids, w, s = run(moe, l, r, k, scores=True)
    some = [0, 1, 63, 64, 4095, 65535, 65536, 70000]
    one = run(moe, l[some].contiguous(), r, k, scores=True)
    assert np.array_equal(ids[some], one[0]) and np.array_equal(w[some], one[1]) and np.array_equal(s[some], one[2])
    lf = l.float()
    top = torch.sort(lf, dim=1, descending=True, stable=True).indices[:, :k].int().cpu().numpy()
    assert np.array_equal(ids, top)
