"""The host side of the MXFP4 calls and of the gradients of permute and un-permute (api.hip's checks and the
launchers' arithmetic) under AddressSanitizer and UndefinedBehaviorSanitizer, with refused and random arguments
(tests/sanitize/abi_driver_mxfp4.cpp).  CPU only: the driver refuses to run where a GPU is visible."""
import concurrent.futures as cf
import glob
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "group_gemm_amd", "csrc")
OBJ = os.path.join(ROOT, "group_gemm_amd", "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
# instrumented on the host: the checks, and the launchers whose sizes reach them from the random arguments.  (The
# product's launchers are compiled as they are in the library: their kernels take most of a minute.)
CHECKED = ("api.hip", "mxfp4.hip", "unpermute_grad.hip")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_mxfp4_and_gradient_validation_under_asan_and_ubsan(tmp_path):
    kernels = [o for o in glob.glob(os.path.join(OBJ, "*.hip.o")) if os.path.basename(o)[:-2] not in CHECKED]
    if not kernels:
        pytest.skip("the library has not been built (python -m group_gemm_amd.build)")
    common = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-w", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    srcs = [os.path.join(CSRC, s) for s in CHECKED] + [os.path.join(ROOT, "tests", "sanitize", "abi_driver_mxfp4.cpp")]

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, *common, *SAN, "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    with cf.ThreadPoolExecutor(len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "abi_driver_mxfp4")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, *kernels, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=900)
    if run.returncode == 77:
        pytest.skip(run.stdout.strip())
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-3000:]
    assert "0 failures" in run.stdout
    print(run.stdout)
