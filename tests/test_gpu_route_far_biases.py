"""GPU: biases as large as fp32 goes.  Keys are scores plus biases in 64 bits: sums of two
biased scores that cancel, or that pass the largest fp32 number, order the groups as they
do there."""
import numpy as np
import pytest
import torch

import more_reference as ref
from gpu_helpers import say
from test_gpu_route import moe, run  # noqa: F401 (moe is a fixture)

pytestmark = pytest.mark.gpu

# experts, groups: lanes that hold one group whole, groups that start inside a lane, one by one
SHAPES = [(32, 4), (64, 8), (256, 8), (60, 4), (21, 7), (12, 12), (1000, 10)]


def both(moe, l, b, r, k):
    ids, _, _ = run(moe, torch.from_numpy(l).cuda(), r, k, torch.from_numpy(b).cuda())
    want = ref.choose(l, b, r, k)
    assert np.array_equal(ids, want), (ids[(ids != want).any(1)][:3], want[(ids != want).any(1)][:3])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", SHAPES)
def test_sums_that_cancel(moe, score, e, groups):  # noqa: F811
    """Every other group's two best are a large bias and its negative (2^20 to 2^27: a unit of fp32
    is 1/8 to 16, of 64 bits 2^-32 and less), the others' are their scores."""
    rng = np.random.default_rng(e + groups)
    each = e // groups
    for power in (20, 24, 27):
        say(f"[route far biases] cancel {score} {e} {groups} 2^{power}")
        l = (2 * rng.standard_normal((50, e))).astype(np.float32)
        b = np.zeros((groups, each), dtype=np.float32)
        b[::2] = -2.0 ** power
        b[::2, 0] = 2.0 ** power
        for top in (1, 2):
            r = dict(score=score, n_groups=groups, top_groups=max(1, groups // 2), group_top=top)
            both(moe, l, b.reshape(-1), r, 2 if each * r["top_groups"] > 1 else 1)


@pytest.mark.parametrize("sign", [1, -1, 0])
@pytest.mark.parametrize("e,groups", SHAPES)
def test_sums_past_the_largest_number(moe, e, groups, sign):  # noqa: F811
    rng = np.random.default_rng(7 * e + groups)
    for score in ("softmax", "sigmoid"):
        say(f"[route far biases] overflow {score} {e} {groups} {sign}")
        l = rng.standard_normal((20, e)).astype(np.float32)
        b = (rng.uniform(1.6e38, 3.4e38, e) * (sign or rng.choice([-1, 1], e))).astype(np.float32)
        for top in (1, 2):
            r = dict(score=score, n_groups=groups, top_groups=max(1, groups // 3), group_top=top)
            both(moe, l, b, r, 2 if e // groups * r["top_groups"] > 1 else 1)
