"""Every launch of the decay operator and of the query/key norm keeps to what a
launch can hold, at the largest sizes that the entries accept: their host code and
launchers, built for the host alone, with the runtime's launch replaced by one that
looks at the grid (sanitize/grid_driver.cpp).  No GPU is touched."""
import glob
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrence_fwd_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_grids_of_the_largest_sizes(tmp_path):
    flags = ["--cuda-host-only", "-O1", "-std=c++17", "--offload-arch=gfx950", "-I" + os.path.join(ROOT, "include")]
    srcs = [(s, []) for s in sorted(glob.glob(os.path.join(CSRC, "gdn_decay*.hip"))) +
            [os.path.join(CSRC, "gdn_norm_rope.hip")]]
    srcs.append((os.path.join(ROOT, "tests", "sanitize", "grid_driver.cpp"), ["-x", "hip"]))
    procs, objs = [], []
    for src, extra in srcs:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen([HIPCC, *flags, *extra, "-c", src, "-o", objs[-1]], stdout=subprocess.PIPE,
                                      stderr=subprocess.PIPE, text=True))
    for p in procs:
        err = p.communicate(timeout=600)[1]
        assert p.returncode == 0, err[-4000:]
    exe = str(tmp_path / "grids")
    # (the device code's images are the only symbols left open: there are none)
    r = subprocess.run(["g++", "-no-pie", "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert r.stdout.startswith("ok:")
    print(r.stdout)
