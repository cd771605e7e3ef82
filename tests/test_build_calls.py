"""The compiled calls are optional: where they cannot be built the build goes on without them."""
import os
import stat

import pytest

from nvfp4_token_routed_gb300 import build


@pytest.mark.parametrize("gcc", ["fails", "missing", "no headers"])
def test_a_build_without_the_compiled_calls(tmp_path, monkeypatch, capsys, gcc):
    so = tmp_path / "_calls.so"
    so.write_text("of older sources")
    monkeypatch.setattr(build, "CALLS", str(so))
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    if gcc == "fails":
        f = bin_dir / "gcc"
        f.write_text("#!/bin/sh\necho 'calls.c: error' >&2\nexit 1\n")
        f.chmod(f.stat().st_mode | stat.S_IXUSR)
    if gcc == "no headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setenv("PATH", str(bin_dir) + (os.pathsep + "/bin" if gcc == "fails" else ""))
    assert build.build_calls() is None
    assert not so.exists()  # another build's would meet other entry points
    assert "calls.c not built" in capsys.readouterr().err
