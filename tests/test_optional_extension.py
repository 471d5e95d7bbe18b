"""The binding's extension (_fast_calls.so) is optional: where it cannot be built
or does not load, the library does what it does without it."""
import os
import shutil
import subprocess
import sys

import pytest

from mixture_experts_projections_b200 import build as b

PROGRAM = """
import warnings
from mixture_experts_projections_b200 import rom
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    assert rom.rom_workspace_size(1000, 8) > 0      # the first call of the process
    assert rom.rom_workspace_size(1000, 8) > 0
assert rom._fast is None
print([str(w.message) for w in seen if "checked in Python" in str(w.message)])
"""


@pytest.mark.parametrize("torch_version", [None, "0.0.1", "unknown"])
def test_an_extension_that_does_not_load_is_left_out(tmp_path, torch_version):
    b.build()
    pkg = tmp_path / "mixture_experts_projections_b200"
    pkg.mkdir()
    for f in ("__init__.py", "rom.py", "librom.so"):
        shutil.copy(os.path.join(b.PKG, f), pkg / f)
    if torch_version is None:  # no library at all
        (pkg / "_fast_calls.so").write_bytes(b"not a library")
    else:  # one built against another torch, or that does not say against which
        import torch
        old = torch.__version__.split("+")[0].encode() + b"\0"
        new = torch_version.encode().ljust(len(old) - 1, b"0") + b"\0"
        if torch_version == "unknown":
            old, new = b"torch_version\0", b"torch_versios\0"
        data = open(b.FAST, "rb").read()
        assert old in data
        (pkg / "_fast_calls.so").write_bytes(data.replace(old, new))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("checked in Python") == 1  # said once
    if torch_version:
        assert f"built against torch {torch_version}" in r.stdout


def test_the_library_builds_without_a_compiler_for_the_extension(tmp_path, monkeypatch):
    b.build()
    stale = tmp_path / "_fast_calls.so"
    stale.write_bytes(b"of older sources")
    os.utime(stale, (0, 0))
    real = subprocess.run

    def run(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return real(cmd, **kw)

    monkeypatch.setattr(b, "FAST", str(stale))
    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="g\\+\\+"):
        assert b.build() == b.LIB
    assert not stale.exists()
