"""Build libmoe.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe.so")
SOURCES = ["host_checks.cpp", "api.hip", "plan.hip", "dispatch.hip", "combine.hip", "exchange.hip",
           "routing_map.hip", "combine_backward.hip", "expert_forward.hip", "expert_backward.hip",
           "route.hip", "quantize.hip", "expert_mx.hip"]
ARCH = os.environ.get("MOE_OFFLOAD_ARCH", "gfx950")


# keep the compiler from emitting packed-fp32 VALU forms
NO_PACKED = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def compile_command(source: str, out: str) -> list[str]:
    return ["hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", *NO_PACKED,
            "-Wall", "-Wno-unused-command-line-argument", "-I", os.path.join(ROOT, "include"),
            "-x", "hip", "-c", os.path.join(CSRC, source), "-o", out]


def link_command(objects: list[str], out: str) -> list[str]:
    return ["hipcc", f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", out, *objects]


TEST_KERNELS = os.path.join(ROOT, "tests", "kernels")
TEST_LIB = os.path.join(TEST_KERNELS, "libfp8_path_check.so")


def build_test_kernels(force: bool = True) -> str:
    """Compile the test-support kernels that check libmoe's device code paths
    exhaustively (tests/kernels/*.hip) into tests/kernels/libfp8_path_check.so."""
    if not force and os.path.exists(TEST_LIB):
        return TEST_LIB
    tmp = TEST_LIB + ".tmp%d" % os.getpid()
    cmd = ["hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", *NO_PACKED,
           "-Wno-unused-command-line-argument", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
           "-o", tmp, os.path.join(TEST_KERNELS, "fp8_path_check.hip")]
    subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE)
    os.replace(tmp, TEST_LIB)
    return TEST_LIB


def build(force: bool = True, verbose: bool = False) -> str:
    """Compile every HIP source, side by side, and link combine_topk_ids_amd/libmoe.so."""
    if not force and os.path.exists(LIB):
        return LIB
    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, cwd=PKG, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)

    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory(dir=PKG) as to, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(to, s + ".o") for s in SOURCES]
        list(pool.map(run, [compile_command(s, o) for s, o in zip(SOURCES, objects)]))
        run(link_command(objects, tmp))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_test_kernels(force=True))
