"""The plan and run logic of a layer's products, layer norm and routing (layer_api.cpp, norm_api.cpp,
route_api.cpp; host code, no GPU) under AddressSanitizer and UndefinedBehaviorSanitizer: driven over random and
edge-case descriptions and pointers, with kernel stand-ins that check what the kernels rely on."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
CLANGXX = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(HIPCC) or not os.path.exists(CLANGXX), reason="no hipcc")
def test_layer_plan_logic_under_asan(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-fno-sanitize-recover=undefined"]
    objs = []
    for src in (os.path.join(ROOT, "tiled_gemm_epilogues_amd", "csrc", "layer_api.cpp"),
                os.path.join(ROOT, "tiled_gemm_epilogues_amd", "csrc", "norm_api.cpp"),
                os.path.join(ROOT, "tiled_gemm_epilogues_amd", "csrc", "route_api.cpp"),
                os.path.join(ROOT, "tests", "asan", "layer_stubs.cpp"),
                os.path.join(ROOT, "tests", "asan", "layer_driver.cpp")):
        obj = tmp_path / (os.path.basename(src) + ".o")
        r = subprocess.run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
                            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                            "-I", os.path.join(ROOT, "include"), *san, "-c", src, "-o", str(obj)],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-3000:]
        objs.append(str(obj))
    exe = tmp_path / "layer_driver"
    subprocess.run([CLANGXX, "-fsanitize=address,undefined", "-o", str(exe), *objs, "-L/opt/rocm/lib",
                    "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([str(exe)], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " 0 failures" in r.stdout, r.stdout
