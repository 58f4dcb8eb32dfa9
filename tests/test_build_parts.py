"""The C library and the operators' extension module are built separately."""
from __future__ import annotations

import os
import subprocess
import sys


def test_the_library_needs_no_torch(gemv_lib, tmp_path):
    """The build file run as a script, with neither torch nor its headers to be found."""
    from memory_bound_gemv_02_gb300 import _build
    (tmp_path / "torch.py").write_text("raise ImportError('no torch here')\n")
    r = subprocess.run([sys.executable, os.path.abspath(_build.__file__)], capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [_build.LIB]


def test_an_extension_of_another_torch_is_stale(gemv_lib, tmp_path, monkeypatch):
    from memory_bound_gemv_02_gb300 import _build
    assert not _build._stale_extension()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(_build, "EXTENSION_STAMP", str(stamp))
    assert _build._stale_extension()  # nothing says what it was built against
    stamp.write_text(_build._extension_target())
    assert not _build._stale_extension()
    stamp.write_text("torch 1.0 python cpython-30")
    assert _build._stale_extension() and not _build._stale_library()
