"""The build without what only the compiled marshalling needs: the library comes out all the same."""
import os
import subprocess
import sys

import pytest

from bit_weight_only_w2_b200 import build as b


def compiler_missing(monkeypatch):
    monkeypatch.setenv("CXX", "no-such-compiler")


def compiler_failing(monkeypatch):
    monkeypatch.setenv("CXX", "false")


def torch_missing(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)


@pytest.mark.parametrize("without", [compiler_missing, compiler_failing, torch_missing])
def test_build_without_the_marshalling(without, monkeypatch, tmp_path, capsys):
    lib = tmp_path / "_marshal.so"
    lib.write_bytes(b"of other sources")
    os.utime(lib, (0, 0))
    monkeypatch.setattr(b, "MARSHAL_LIB", str(lib))
    monkeypatch.setattr(b, "sources", list)          # (the library as it is)
    without(monkeypatch)
    assert b.build() == b.LIB
    assert list(tmp_path.iterdir()) == []
    assert "_marshal.so was not built" in capsys.readouterr().err


def test_the_tests_collect_without_the_marshalling():
    """Every test file is collected where _marshal.so is missing, but for that module's own."""
    code = ("import sys; sys.modules['bit_weight_only_w2_b200._marshal'] = None; import pytest; "
            "sys.exit(pytest.main(['tests', '--collect-only', '-q', '-p', 'no:cacheprovider']))")
    r = subprocess.run([sys.executable, "-c", code], cwd=b.ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]
    assert "test_adapter_abi.py" in r.stdout and "test_marshal.py" not in r.stdout
