"""What the build needs and when it makes kda_native.so anew."""
import os
import subprocess
import sys

import torch

from linear_attention_rule_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_builds_without_torch(monkeypatch, tmp_path):
    """A C user of libkda.so has nvcc and a host compiler, and may have no torch."""
    build.build()
    ran = []
    monkeypatch.setattr(build, "_run", lambda cmd, target, verbose: ran.append(target))
    monkeypatch.setattr(build, "torch_version", lambda: None)
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "kda_native.so"))
    assert build.build() == build.LIB and ran == []
    assert build.build(force=True) == build.LIB and ran == [build.LIB]


def test_a_process_where_torch_cannot_be_imported_builds():
    build.build()
    code = ("import sys; sys.modules['torch'] = None\n"
            "from linear_attention_rule_b200 import build\n"
            "assert build.torch_version() is None and build.build() == build.LIB")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "no torch" in r.stderr


def test_looking_at_a_build_that_is_up_to_date_does_not_import_torch():
    build.build()
    code = "import sys\nfrom linear_attention_rule_b200 import build\nbuild.build()\nassert 'torch' not in sys.modules"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_another_torch_makes_the_binding_stale(monkeypatch):
    build.build()
    assert build.torch_version() == torch.__version__
    assert not build.native_needs_build()
    for other in ("0.1.0", torch.__version__[:-1], torch.__version__ + "0"):
        monkeypatch.setattr(build, "torch_version", lambda: other)
        assert build.native_needs_build()
