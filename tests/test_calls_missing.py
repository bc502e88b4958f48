"""A short way (_calls.so) that cannot be loaded is said at the import of the binding, which
is whole without it; one that can be says nothing."""
import os
import shutil
import subprocess
import sys

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_recurrence_fwd_amd")
SCRIPT = """
import warnings
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    from {name} import binding
print([str(x.message) for x in w if "_calls" in str(x.message)], binding._calls is not None)
"""


@pytest.mark.parametrize("content", [None, b"", b"not a library", "real"])
def test_said_at_import(tmp_path, content):
    name = os.path.basename(PACKAGE)
    built = os.path.join(PACKAGE, "_calls.so")
    if content == "real" and not os.path.exists(built):
        pytest.skip("not built")
    os.mkdir(tmp_path / name)
    for f in os.listdir(PACKAGE):
        if f.endswith(".py") or (content == "real" and f.endswith(".so")):
            shutil.copy(os.path.join(PACKAGE, f), tmp_path / name / f)
    if isinstance(content, bytes):
        (tmp_path / name / "_calls.so").write_bytes(content)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(name=name)], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    said, loaded = r.stdout.strip().rsplit(" ", 1)
    assert loaded == str(content == "real")
    assert (said == "[]") == (content == "real") and (content == "real" or "was not loaded" in said)
