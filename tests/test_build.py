"""The build without a GPU compiler: a stand-in for nvcc writes its output file.  The library needs nvcc alone; where the
operators' Python binding cannot be built (no C compiler, no CPython headers) the library is there all the same."""
import os
import stat
import subprocess
import sys
import warnings

import pytest

from shampoo_roots_gb300 import build as b


def script(path, text):
    path.write_text("#!%s\n%s" % (sys.executable, text))
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


WRITES = "import sys\nopen(sys.argv[sys.argv.index('-o') + 1], 'w').write('%s')\n"


@pytest.fixture
def place(tmp_path, monkeypatch):
    """Targets in a folder of their own, and a PATH that holds the stand-ins only."""
    (tmp_path / "bin").mkdir()
    monkeypatch.setattr(b, "OUT", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setenv("PATH", str(tmp_path / "bin"))
    monkeypatch.setenv("NVCC", script(tmp_path / "bin" / "nvcc", WRITES % "library"))
    return tmp_path


def test_both(place):
    script(place / "bin" / "gcc", WRITES % "binding")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert b.build() == b.OUT
    assert open(b.OUT).read() == "library" and open(b.BINDING).read() == "binding"
    assert sorted(os.listdir(place)) == ["bin", "binding.so", "lib.so"]


@pytest.mark.parametrize("compiler", [None, "import sys\nsys.exit(1)\n"])
def test_library_without_the_binding(place, compiler):
    if compiler:
        script(place / "bin" / "gcc", compiler)
    (place / "binding.so").write_text("of other sources")
    with pytest.warns(UserWarning, match="binding"):
        assert b.build(force=True) == b.OUT
    assert open(b.OUT).read() == "library"
    assert sorted(os.listdir(place)) == ["bin", "lib.so"]          # nothing stale, nothing half made


def test_only_what_is_older_is_made(place):
    script(place / "bin" / "gcc", WRITES % "binding")
    b.build()
    os.remove(b.BINDING)
    open(b.OUT, "w").write("kept")
    b.build()
    assert open(b.OUT).read() == "kept" and open(b.BINDING).read() == "binding"


def test_a_library_that_does_not_compile_raises(place, monkeypatch):
    script(place / "bin" / "gcc", WRITES % "binding")
    monkeypatch.setenv("NVCC", script(place / "bin" / "nvcc2", "import sys\nsys.exit(3)\n"))
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert not os.path.exists(b.OUT)
