"""What build() takes for up to date."""
import os
import subprocess
import sysconfig
import time

import pytest
import torch

from linear_attention_serving_gated_gb300 import build, kda


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A build that is newer than every source, in a folder of its own."""
    for name in ("LIB", "HOST", "HOST_FOR"):
        path = str(tmp_path / os.path.basename(getattr(build, name)))
        monkeypatch.setattr(build, name, path)
        with open(path, "w") as f:
            f.write(build.made_for())
        os.utime(path, (time.time() + 60,) * 2)
    return tmp_path


def test_up_to_date(built):
    assert not build.stale()
    os.utime(build.LIB, (0, 0))
    assert build.stale()


def test_another_pytorch_or_python_is_not(built, monkeypatch):
    """The binding's checks read PyTorch's tensors by the layout that they were built with."""
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.2.3")
        assert build.stale()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        assert build.stale()
    assert not build.stale()
    os.remove(build.HOST_FOR)
    assert build.stale()


def test_the_name_is_this_pythons():
    assert os.path.basename(build.HOST) == "_host_args" + sysconfig.get_config_var("EXT_SUFFIX")


def test_load_refuses_what_another_pytorch_built(built, monkeypatch):
    monkeypatch.setattr(kda, "_lib", None)
    with open(build.HOST_FOR, "w") as f:
        f.write("PyTorch 1.2.3")
    with pytest.raises(RuntimeError, match=r"built for PyTorch 1\.2\.3.*build\(\)"):
        kda.load()
    os.remove(build.HOST_FOR)
    with pytest.raises(RuntimeError, match="_host_args.so not built"):
        kda.load()


def test_installed_beside_and_renamed(tmp_path):
    """A library that a process has open stays what it is there."""
    old, new = tmp_path / "lib.so", tmp_path / "build" / "lib.so"
    new.parent.mkdir()
    old.write_text("old")
    new.write_text("new")
    with open(old) as mapped:
        build.install(str(new), str(old))
        assert mapped.read() == "old" and os.fstat(mapped.fileno()).st_ino != os.stat(old).st_ino
    assert old.read_text() == "new" and sorted(p.name for p in tmp_path.iterdir()) == ["build", "lib.so"]


def test_build_moves_no_file_onto_a_library():
    with open(build.__file__) as f:
        assert "shutil.move" not in f.read()  # (between file systems it copies into the file that is there)


def test_the_bindings_checks_compile_without_warnings(tmp_path):
    command = build._host_command(str(tmp_path / "x.so"))
    assert "-Wall" in command and "-w" not in command
    said = subprocess.run(command, capture_output=True, text=True)
    assert said.returncode == 0 and said.stdout == said.stderr == ""
