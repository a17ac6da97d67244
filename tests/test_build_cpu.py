"""Building without a GPU: the library needs nvcc alone, the binding of the generation
calls torch, its headers and Python's; the one is built where the other cannot be.
Nothing here touches the package's own built files."""
import os
import subprocess
import sys

import pytest

from ffn_long_video_b200 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A library that needs no compiling, a binding that does and whose compiler fails."""
    lib = tmp_path / "libadaspark.so"
    obj = tmp_path / "x.o"
    obj.write_text("")
    lib.write_text("")
    os.utime(obj, (1, 1))
    monkeypatch.setattr(_build, "LIB", str(lib))
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "sources", lambda: ["x"])
    monkeypatch.setattr(_build, "_compile", lambda *a: str(obj))
    monkeypatch.setattr(_build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setenv("CXX", "false")
    return tmp_path


def test_the_library_is_built_without_its_binding(built, capsys):
    assert _build.build() == str(built / "libadaspark.so")
    assert "_calls.so" in capsys.readouterr().err
    with pytest.raises(RuntimeError):
        _build.build_calls()


def test_the_library_is_built_without_torch():
    """In a Python of its own that has no torch, with a library that is up to date."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from ffn_long_video_b200 import _build\n"
            "_build.LIB = sys.executable\n"
            "_build.sources = lambda: ['x']\n"
            "_build._compile = lambda *a: sys.executable\n"
            "print(_build.build())")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == sys.executable and "torch" in r.stderr


@pytest.mark.parametrize("stamp", ["torch", "python", "source"])
def test_a_stale_binding_is_built_again_or_taken_away(built, stamp):
    """One compiled against another torch or Python, or older than its source, is not
    left to be loaded beside a newer library."""
    import torch
    here = f"{torch.__version__} {sys.implementation.cache_tag}"
    calls = built / "_calls.so"
    calls.write_text("")
    (built / "calls.torch").write_text({"torch": "0.0 " + sys.implementation.cache_tag,
                                        "python": torch.__version__ + " other",
                                        "source": here}[stamp])
    if stamp == "source":
        os.utime(calls, (1, 1))
    with pytest.raises(RuntimeError):
        _build.build_calls()
    assert not calls.exists()
    calls.write_text("")
    (built / "calls.torch").write_text(here)
    assert _build.build_calls() == str(calls)      # current: left as it is
