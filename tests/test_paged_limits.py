"""The attention over pages at its limits: sizes just inside are accepted and make launches
that a device can hold, those just outside are refused, and every item of the prefix has one
part of the work (sanitize/paged_limits_driver.cpp).  No GPU is touched."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrence_fwd_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ("gdn_paged_api.hip", "gdn_paged_append.hip", "gdn_prefix_attn.hip", "gdn_prefix_attn_many.hip", "gdn_prefix_plan.hip")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_limits(tmp_path):
    flags = ["--cuda-host-only", "-O1", "-std=c++17", "--offload-arch=gfx950", "-I" + os.path.join(ROOT, "include")]
    srcs = [(os.path.join(CSRC, s), []) for s in SOURCES]
    srcs.append((os.path.join(ROOT, "tests", "sanitize", "paged_limits_driver.cpp"), ["-x", "hip"]))
    procs, objs = [], []
    for src, extra in srcs:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen([HIPCC, *flags, *extra, "-c", src, "-o", objs[-1]], stdout=subprocess.PIPE,
                                      stderr=subprocess.PIPE, text=True))
    for p in procs:
        err = p.communicate(timeout=600)[1]
        assert p.returncode == 0, err[-4000:]
    exe = str(tmp_path / "limits")
    # (what is left open is the device code's images, of which there are none)
    r = subprocess.run(["g++", "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert r.stdout.startswith("ok:")
