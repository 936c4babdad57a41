"""Builds the HIP library tiled_gemm_epilogues_amd/libtge.so for gfx950 with hipcc.

The kernel source is compiled once per (input, output) type pair, in parallel, and linked with
the host API into one shared library that exports the C ABI declared in include/gemm.h.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtge.so")

PAIRS = ["F32_F32", "F16_F16", "F16_F32", "BF16_BF16", "BF16_F32", "I8_I32"]
FAST_PAIRS = ["F16_F16", "F16_F32", "BF16_BF16", "BF16_F32", "I8_I32"]
SKINNY_PAIRS = ["F16_F16", "F16_F32", "BF16_BF16", "BF16_F32", "I8_I32"]
GROUPED_PAIRS = ["F16_F16", "F16_F32", "BF16_BF16", "BF16_F32"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         # never let the compiler form packed fp32 VALU instructions
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include")]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"build step failed: {' '.join(cmd)}")
    return r


def steps():
    """The compile commands, one per object (the object is each command's last word)."""
    out = []

    def add(source, obj, *defines, host=False):
        out.append([HIPCC, *FLAGS, *defines, *(["-x", "hip"] if host else []), "-c",
                    os.path.join(CSRC, source), "-o", os.path.join(BUILD, obj + ".o")])

    for name, pairs in (("gemm_kernels", PAIRS), ("gemm_fast", FAST_PAIRS), ("gemm_skinny", SKINNY_PAIRS)):
        for pair in pairs:
            add(name + ".hip", f"{name}_{pair.lower()}", f"-DTGE_PAIR_{pair}")
    # the same kernels on products grouped by expert (float types)
    for name, pairs in (("gemm_kernels", GROUPED_PAIRS + ["F32_F32"]), ("gemm_fast", GROUPED_PAIRS)):
        for pair in pairs:
            add(name + ".hip", f"grouped_{name}_{pair.lower()}", f"-DTGE_PAIR_{pair}", "-DTGE_GROUPED")
    for pair in GROUPED_PAIRS:
        for name in ("gemm_rows16", "gemm_quant"):
            add(name + ".hip", f"{name}_{pair.lower()}", f"-DTGE_PAIR_{pair}")
    for name in ("gemm_complex", "gemm_diag", "gemm_repack"):
        add(name + ".hip", name)
    for name in ("gemm_api", "grouped_api", "quant_api"):
        add(name + ".cpp", name, host=True)
    return out


def build(verbose=False, jobs=None):
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(8, os.cpu_count() or 1)
    cmds = steps()
    with cf.ThreadPoolExecutor(jobs) as ex:
        list(ex.map(lambda c: _run(c, verbose), cmds))
    objs = [s[-1] for s in cmds]
    tmp = LIB + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
