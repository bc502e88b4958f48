"""The host code of the paged cache's entries (gdn_paged_api.hip) and the attention's
plan under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU
(sanitize/paged_driver.cpp): workspaces of exactly the queried sizes, splits that cover
all keys and tiles that cover all rows, over a grid of sizes."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrence_fwd_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_paged_host_code_under_asan_ubsan(tmp_path):
    flags = ["-O1", "-g", "-std=c++17", "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
             "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-I" + os.path.join(ROOT, "include")]
    srcs = [(os.path.join(CSRC, "gdn_paged_api.hip"), []), (os.path.join(CSRC, "gdn_prefix_plan.hip"), []),
            (os.path.join(ROOT, "tests", "sanitize", "paged_driver.cpp"), ["-x", "hip"])]
    objs = []
    for src, extra in srcs:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        r = subprocess.run([HIPCC, *flags, *extra, "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
    exe = str(tmp_path / "paged_san")
    r = subprocess.run([HIPCC, "-fsanitize=address,undefined", "-fno-gpu-sanitize", "--offload-arch=gfx950", *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
                                UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1"))
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert r.stdout.startswith("ok:")
