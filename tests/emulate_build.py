"""Builds a kernel's source for the CPU, lane by lane (tests/emulate; no tests here)."""
import os
import re
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_topk_ids_amd", "csrc")
EMULATE = os.path.join(ROOT, "tests", "emulate")
CLANG = shutil.which("amdclang++") or shutil.which("clang++")


def _once(pattern, to, text, what):
    text, n = re.subn(pattern, to, text, flags=re.S)
    assert n == 1, f"{what}: {n} places"
    return text


def for_cpu(name, text, units):
    """What the host compiler takes of a source: launches, LDS and the four functions in assembly."""
    text = re.sub(r"(\w+(?:<[^<>;]*>)?)<<<(.+?), (.+?), 0, stream>>>\((.*?)\);",
                  r"emu::launch(\2, \3, [=] { \1(\4); });", text)
    text = re.sub(r"__shared__ (?:__align__\(\d+\) )?(\w+) (\w+)\[(.*?)\];", r'\1 *\2 = emu::shared<\1>("\2", \3);',
                  text)
    if name == "expert_tile.hpp":
        text = text.replace("#define MOE_LDS __attribute__((address_space(3)))", "#define MOE_LDS")
        body = r"(__device__ __forceinline__ void %s\(i32x4 r, lds_ptr to, %s\) \{\n).*?\n\}\n"
        text = _once(body % ("load_lds16", r"const uint32_t \(&o\)\[L\]"), r"\1  emu::load_lds<STRIDE, 16>(r, to, o);\n}\n",
                     text, "load_lds16")
        text = _once(body % ("load_lds4", r"uint32_t o"),
                     r"\1  const uint32_t a[1] = {o};\n  emu::load_lds<0, 4>(r, to, a);\n}\n", text, "load_lds4")
        text = _once(r'  asm volatile\("s_waitcnt vmcnt\(%0\)[^;]*;', "  emu::wait_and_meet(N);", text, "wait_and_meet")
        text = _once(r'  asm volatile\("" : "\+v"\(l\)\);', "", text, "late_lane_id")
        text = _once(r"constexpr int kComputeUnits = 256;",
                     f"constexpr int kComputeUnits = {units};", text, "compute units")
    return text


def build(to, kernel, defines=(), units=16):
    """The program of tests/emulate/<kernel>.cpp, under the address sanitizer; `units`: the card's compute units."""
    os.makedirs(to, exist_ok=True)
    for name in os.listdir(CSRC):
        if name.endswith((".hpp", ".hip")):
            with open(os.path.join(CSRC, name)) as f:
                text = for_cpu(name, f.read(), units)
            with open(os.path.join(to, name.replace(".hip", ".inc")), "w") as f:
                f.write(text)
    exe = os.path.join(to, kernel)
    subprocess.run([CLANG, "-std=c++20", "-O1", "-gline-tables-only", *defines, "-fno-omit-frame-pointer", "-fsanitize=address",
                    "-Wno-unknown-attributes", "-Wno-psabi", "-ffp-contract=off", "-I", to, "-I", EMULATE,
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(EMULATE, kernel + ".cpp"),
                    os.path.join(CSRC, "host_checks.cpp"), "-o", exe], check=True)
    return exe
