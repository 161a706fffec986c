"""CPU: routing, quantisation and the products with MX-FP4 weights, lane by lane under the address sanitizer
(tests/emulate): no access outside its memory, every barrier met by all, no stage of LDS read before it has
landed or freed while it is read, and the results right, over random sizes up to the largest that are accepted."""
import os
import subprocess

import pytest

import emulate_build

pytestmark = pytest.mark.skipif(emulate_build.CLANG is None, reason="needs clang")


@pytest.fixture(scope="module")
def programs(tmp_path_factory):
    """Built side by side: {name: path}."""
    from concurrent.futures import ThreadPoolExecutor
    to = tmp_path_factory.mktemp("emulate")
    what = {"route": ("route", ()), "glu": ("expert_mx", ("-DGATED=true",)), "linear": ("expert_mx", ("-DGATED=false",))}
    with ThreadPoolExecutor(len(what)) as pool:
        made = {k: pool.submit(emulate_build.build, str(to / k), v[0], v[1]) for k, v in what.items()}
    return {k: f.result() for k, f in made.items()}


def run(exe, seed, cases):
    # (the lanes' stacks live as long as the program)
    res = subprocess.run([exe, str(seed), str(cases)], capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert res.returncode == 0 and res.stdout.endswith("no failures\n"), res.stdout[-600:] + res.stderr[-3000:]


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_routing_and_quantisation(programs, seed):
    run(programs["route"], seed, 60)


@pytest.mark.parametrize("form", ["glu", "linear"])
@pytest.mark.parametrize("seed", [1])
def test_products_with_mx_weights(programs, form, seed):
    run(programs[form], seed, 4)
