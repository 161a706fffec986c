"""CPU: the inputs of the FP8 rows of any code would show a cut product in each tile."""
import pytest

import any_code_reference as any_code


def test_each_tile_once():
    assert {any_code.tile(**c) for c in any_code.CASES} == {"16x64, K in four", "16x64", "64x128", "128x256"}


@pytest.mark.parametrize("c", any_code.CASES, ids=lambda c: any_code.tile(**c) + f", {c['k']}")
def test_a_cut_would_pass_the_bound(c):
    x, xs, w, ws = any_code.inputs(c, c["tokens"])
    some = 64
    past = 0
    for t in range(0, 8):
        lost, mag = any_code.cut_error(x[t], xs[t], w[0][:some].numpy(), ws[0][:some].numpy())
        # twice the bound: not less than the bound even where what is kept errs the other way
        past += int((lost > 2 * any_code.BOUND * mag).sum())
    assert past > 8 * some // 4
