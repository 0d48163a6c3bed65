"""The build on the CPU, with compilers and linker replaced by records of what they are
asked: the C libraries do not wait for torch."""
import os
import warnings

import pytest

from conftest import load_build_module


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with every output in a folder of the test's, and nothing compiled."""
    m = load_build_module()
    for name in ("LIB", "PROBES_LIB", "ATTN_LIB", "BINDING_LIB"):
        monkeypatch.setattr(m, name, str(tmp_path / os.path.basename(getattr(m, name))))
    made = []

    def touch(path, text="x"):
        with open(path, "w") as f:
            f.write(text)
        made.append(os.path.basename(path))
        return path

    def link(sources, lib, build_dir, dflags, verbose):
        return touch(lib)

    def compile_binding(build_dir):
        m._torch_root()
        os.makedirs(build_dir, exist_ok=True)
        return touch(os.path.join(build_dir, "attn_binding.o"))

    monkeypatch.setattr(m, "_link", link)
    monkeypatch.setattr(m, "_compile_binding", compile_binding)
    monkeypatch.setattr(m, "_link_binding", lambda obj: touch(m.BINDING_LIB))
    m.made, m.dir = made, str(tmp_path / "build")
    m.run = lambda **kw: m.build(lib=m.LIB, build_dir=m.dir, **kw)
    return m


C_LIBRARIES = {"libdetfold.so", "libdetfold_probes.so", "libdetfold_attn.so"}


def test_everything_is_built_once(build):
    assert build.run() == build.LIB
    assert set(build.made) == C_LIBRARIES | {"attn_binding.o", "_attn_binding.so"}
    build.made.clear()
    build.run()
    assert build.made == []


def test_without_torch_the_c_libraries_are_built(build, monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    with pytest.warns(RuntimeWarning, match="torch"):
        assert build.run() == build.LIB
    assert set(build.made) == C_LIBRARIES


def test_a_binding_that_does_not_compile_leaves_the_c_libraries(build, monkeypatch):
    def fail(build_dir):
        raise RuntimeError("g++ on attn_binding.cpp failed: no such header")

    monkeypatch.setattr(build, "_compile_binding", fail)
    with open(build.BINDING_LIB, "w") as f:
        f.write("of older sources")
    os.utime(build.BINDING_LIB, (0, 0))
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert build.run() == build.LIB
    assert set(build.made) == C_LIBRARIES
    assert not os.path.exists(build.BINDING_LIB), "a binding of older sources is not left to be loaded"


def test_a_c_library_that_does_not_compile_fails_the_build(build, monkeypatch):
    def fail(*a):
        raise RuntimeError("nvcc failed on fold.cu")

    monkeypatch.setattr(build, "_link", fail)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeError, match="nvcc failed"):
            build.run()


def test_the_binding_is_built_again_for_another_torch_or_python(build, tmp_path, monkeypatch):
    # its code is compiled against one torch's headers and one Python's
    root = tmp_path / "torch"
    root.mkdir()
    (root / "version.py").write_text("__version__ = '2.9.1+cu130'\n")
    monkeypatch.setattr(build, "_torch_root", lambda: str(root))
    both = ["attn_binding.o", "_attn_binding.so"]

    def again():
        build.made.clear()
        build.run()
        return [n for n in build.made if n in both]

    assert again() == both
    assert again() == []
    (root / "version.py").write_text("__version__ = '2.11.0+cu130'\n")
    assert again() == both and not C_LIBRARIES & set(build.made)
    assert again() == []
    other = tmp_path / "elsewhere"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '2.11.0+cu130'\n")
    monkeypatch.setattr(build, "_torch_root", lambda: str(other))
    assert again() == both
    assert again() == []
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert again() == both
    assert again() == []
