"""CPU: the 64-bit references of routing and MX-FP4 against differences, against the oracle's
encoder and against cases worked out by hand."""
import numpy as np
import pytest

import more_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(5)
    n, e, k = 3, 7, 3
    r = dict(score=score, renormalize=renormalize, scale=1.5)
    l = rng.standard_normal((n, e))
    ids = np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    ids[1, 2] = -1
    dw, ds = rng.standard_normal((n, k)), rng.standard_normal((n, e))

    def loss(l):
        w = ref.gates(l, ids, r)[0]
        return (w * dw).sum(1) + (ref.scores(l, score) * ds).sum(1)

    got, _ = ref.route_gradient(l, ids, dw, ds, r)
    for i in range(e):
        h = np.zeros((n, e))
        h[:, i] = 1e-5
        # central differences: h^2 of third derivatives (below 10), rounding 1e-16 / h
        assert np.allclose((loss(l + h) - loss(l - h)) / 2e-5, got[:, i], rtol=0, atol=1e-8)


def test_choice_by_hand():
    r = dict(score="sigmoid", n_groups=2, top_groups=1, group_top=2)
    l = np.array([[3.0, -9.0, 1.0, 1.0], [-np.inf] * 4, [np.nan, 0, 5, 5], [2.0, -np.inf, 1.0, -3.0]])
    # sums of two: .95 + 0 against .73 + .73; nothing; the NaN's group; one expert alone, .88 against .78
    assert ref.choose(l, None, r, 2).tolist() == [[2, 3], [-1, -1], [0, 1], [0, -1]]
    assert ref.choose(l[:1], None, dict(r, group_top=1), 2).tolist() == [[0, 1]]
    bias = np.array([0, 2.0, 0, -np.inf])
    assert ref.choose(l[:1], bias, dict(score="sigmoid"), 4).tolist() == [[1, 0, 2, -1]]


def test_mx_encode_is_the_oracles(orc):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.integers(-140, 120, (40, 1)))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    bits[5, :32] = 0
    plan = orc.plan(np.zeros((40, 1), dtype=np.int32), 1, 1, 1, 40, 64)
    pay, sc = orc.dispatch("mxfp4", bits, plan)
    value = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales = ref.mx_encode(value)
    assert np.array_equal(np.asarray(pay).view(np.uint8).reshape(40, -1), codes)
    assert np.array_equal(np.asarray(sc).view(np.uint8).reshape(40, -1), scales)
    # half a step of the block's grid: 1 unit in the last place above 4, and what passes 6
    err = np.abs(ref.mx_value(codes, scales) - value)
    unit = np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=1)
    assert (err <= np.maximum(np.abs(value) - 6 * unit, unit)).all()
