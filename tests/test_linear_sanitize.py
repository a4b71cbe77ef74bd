"""The host layer of linear attention and rotary positions under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): their sources with the sanitizers on the
host side alone, linked with a driver (tests/linear_sanitize) that checks
refusals, sizes and calls without work over random problems.  No call reaches
HIP."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_frame_amd", "csrc")
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
HIP_SOURCES = ["gdn_decode.hip", "gdn_linear.hip", "gdn_linear_grad.hip", "gdn_rotary.hip"]
HOST_SOURCES = ["gdn_linear_api.cpp", "gdn_profile.cpp", os.path.join(ROOT, "tests", "linear_sanitize", "check_linear.cpp")]


def _compile(cmd):
    return subprocess.run(cmd, capture_output=True, text=True)


@pytest.mark.slow
def test_linear_host_layer_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    common = ["-O1", "-g", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *san]
    device = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    jobs, objs = [], []
    for src in HIP_SOURCES + HOST_SOURCES:
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        jobs.append([HIPCC, *common, *(device if src in HIP_SOURCES else []), "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    with ThreadPoolExecutor(max_workers=4) as ex:
        for r in ex.map(_compile, jobs):
            assert r.returncode == 0, r.stdout + r.stderr
    exe = str(tmp_path / "check_linear")
    r = _compile([HIPCC, "--offload-arch=gfx950", *san, "-o", exe, *objs])
    assert r.returncode == 0, r.stdout + r.stderr
    symbols = subprocess.run(["nm", exe], capture_output=True, text=True).stdout
    assert "__asan_report" in symbols and "__ubsan_handle" in symbols, "driver was not instrumented"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "linear host checks passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
