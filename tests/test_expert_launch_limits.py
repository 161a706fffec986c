"""CPU: a layer that the experts' calls accept is one that the device can launch: no
grid reaches 2^32 threads in a dimension.  The widest is that of dz, a workgroup of 256
threads for every 16 rows of an expert and 512 columns, in whole rounds of 8."""
import os
import random
import shutil
import subprocess

import pytest

EOVERFLOW = -3
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    from combine_topk_ids_amd import _build
    if not os.path.exists(_build.LIB):
        _build.build(force=False)
    import combine_topk_ids_amd.moe as m
    return m


def dz_threads(pairs, experts, out_dim):
    tiles = (pairs + min(pairs, experts) * 15) // 16 * -(-out_dim // 512)
    return -(-tiles // 8) * 8 * 256


def test_the_largest_dz_grid(moe):
    def check(rows, experts=1, dim=8):
        return moe.moe_check_expert_op(moe.problem(rows, 8, 1, experts, 1), moe.expert_op(dim, dim, "silu"))

    most = 16 * ((1 << 24) - 8)  # rows of one expert
    assert dz_threads(most, 1, 8) < 1 << 32 <= dz_threads(most + 1, 1, 8)
    assert check(most) == 0
    for rows in (most + 1, most + 17, most + 50):
        assert check(rows) == EOVERFLOW, rows
    assert moe.moe_expert_workspace_bytes(moe.problem(most + 1, 8, 1, 1, 1), moe.expert_op(8, 8, "silu")) == 0
    # more experts: a partial chunk each, until the tiles of the products are too many first
    for experts in (2, 3, 16, 200):
        for rows in range(most - 16 * experts - 64, most + 1, 7):
            fits = dz_threads(rows, experts, 8) < 1 << 32 and rows // 64 + experts < 1 << 22
            assert (check(rows, experts) == 0) == fits, (rows, experts)


def test_accepted_layers_can_be_launched(moe):
    rng = random.Random(5)
    accepted = 0
    for _ in range(20000):
        rows = max(1, (1 << rng.randint(10, 28)) + rng.randint(-600, 600))
        experts, top_k = rng.choice((1, 1, 2, 8, 64, 1024)), 1
        cap = rng.choice((0, 0, 0, 1 << rng.randint(4, 24)))
        p = moe.problem(rows, 8, top_k, experts, 1, expert_capacity=cap)
        op = moe.expert_op(8 * rng.choice((1, 2, 7, 64, 1000)), 8 * rng.choice((1, 2, 3, 7, 8, 64, 65, 1000)), "silu")
        if moe.moe_check_expert_op(p, op) != 0:
            continue
        accepted += 1
        pairs = min(rows * top_k, moe.moe_max_rows(p))
        assert dz_threads(pairs, experts, op.out_dim) < 1 << 32, (rows, experts, cap, op.in_dim, op.out_dim)
    assert accepted > 2000


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_bound_is_the_launchs_own(tmp_path):
    """expert_grad_workgroups, which the launch and the check share, is that grid."""
    src = tmp_path / "grid.cpp"
    src.write_text("""
#include <stdio.h>
#include "host_checks.hpp"
int main() {
  long long n, e, out;
  while (scanf("%lld %lld %lld", &n, &e, &out) == 3) {
    moe_problem p = {};
    p.n_tokens = n; p.hidden = 8; p.top_k = 1; p.n_experts = (int)e; p.ep = 1; p.pad_multiple = 1;
    printf("%lld\\n", (long long)moe::expert_grad_workgroups(p, (int)out) * moe::kGradThreads);
  }
}
""")
    exe, csrc = str(tmp_path / "grid"), os.path.join(ROOT, "combine_topk_ids_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "host_checks.cpp"), str(src), "-o", exe],
                   check=True)
    cases = [(n, e, out) for n in (0, 1, 15, 16, 17, 1000, 268435328, 268435391) for e in (1, 3, 64, 1024)
             for out in (8, 512, 520, 1 << 20)]
    res = subprocess.run([exe], input="\n".join("%d %d %d" % c for c in cases), capture_output=True, text=True, check=True)
    assert [int(v) for v in res.stdout.split()] == [dz_threads(*c) for c in cases]
