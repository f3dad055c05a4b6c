"""What build() leaves where the paged-cache module cannot be compiled, and when
it compiles it again.  No GPU, and nothing is compiled here but the library."""
import os

import pytest

from clustered_multipole_approximation_b200 import build


@pytest.fixture
def module(tmp_path, monkeypatch):
    """build() with a module of its own, up to date; the list of compilers' commands."""
    build.build()
    lib, key = tmp_path / "_torch_cache.so", tmp_path / "_torch_cache.so.key"
    lib.write_text("a module")
    key.write_text(build._torch_key())
    monkeypatch.setattr(build, "TORCH_LIB", str(lib))
    monkeypatch.setattr(build, "TORCH_KEY", str(key))
    ran = []

    def compiler(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("a new module")
        return type("Done", (), dict(returncode=0, stderr=""))

    monkeypatch.setattr(build.subprocess, "run", compiler)
    return lib, key, ran


def test_a_module_that_is_up_to_date_is_kept(module):
    lib, _, ran = module
    assert build.build() == build.LIB and not ran and lib.read_text() == "a module"


@pytest.mark.parametrize("change", ["another torch", "no key", "no module"])
def test_a_module_of_another_torch_is_built_again(module, change):
    lib, key, ran = module
    if change == "another torch":
        key.write_text("torch 1.0, cpython-30")
    else:
        os.remove(key if change == "no key" else lib)
    build.build()
    assert len(ran) == 1 and lib.read_text() == "a new module" and key.read_text() == build._torch_key()


@pytest.mark.parametrize("why", ["no compiler", "compiler fails", "no headers"])
def test_the_library_does_not_need_the_module(module, monkeypatch, why):
    lib, key, _ = module
    key.write_text("torch 1.0, cpython-30")
    if why == "no compiler":
        monkeypatch.setattr(build.shutil, "which", lambda x: None)
    elif why == "compiler fails":
        monkeypatch.setattr(build.subprocess, "run",
                            lambda *a, **kw: type("Done", (), dict(returncode=1, stderr="Python.h: no such file")))
    else:
        monkeypatch.setattr(build, "_torch_key", lambda: (_ for _ in ()).throw(ImportError("no torch")))
    with pytest.warns(RuntimeWarning, match="paged-cache calls will raise"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not lib.exists()
    with pytest.raises((RuntimeError, ImportError)):
        build.build_torch()


@pytest.mark.parametrize("change", ["no key", "older than its sources"])
def test_a_shipped_module_stays_unless_it_is_of_other_sources(module, monkeypatch, change):
    """A module that came without its key, on a box without a compiler."""
    lib, key, _ = module
    monkeypatch.setattr(build.shutil, "which", lambda x: None)
    if change == "no key":
        os.remove(key)
        assert build.build() == build.LIB and lib.exists()
    else:
        os.utime(lib, (1, 1))
        with pytest.warns(RuntimeWarning, match="paged-cache calls will raise"):
            build.build()
        assert not lib.exists()
