"""The in-tree build: what the library needs and what its Python binding needs are kept apart."""
import os

import pytest

from combine_ep_get_05_gb300 import build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build of one small translation unit into an empty directory."""
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libep_gb300.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_ep_binding.so"))
    monkeypatch.setattr(build, "sources", lambda: [os.path.join(build.CSRC, "ep_host.cu")])
    return tmp_path


def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch):
    def no_compiler():
        raise RuntimeError("g++ not found")

    monkeypatch.setattr(build, "host_compiler", no_compiler)
    with pytest.raises(RuntimeError, match="g\\+\\+ not found"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert build.is_stale() and not build._library_is_stale()


def test_a_binding_of_another_torch_or_python_is_stale_and_not_loaded(monkeypatch):
    from combine_ep_get_05_gb300 import _lib

    build.build()
    assert not build.is_stale()
    _lib._native()
    monkeypatch.setattr(_lib, "_binding", None)
    for attribute, value in (("__version__", "1.0.0"), ("version.git_version", "0" * 40)):
        with monkeypatch.context() as m:
            m.setattr(f"torch.{attribute}", value)
            assert build.is_stale() and not build._library_is_stale()
            with pytest.raises(RuntimeError, match="was built for .* and this is .*build it again"):
                _lib._native()
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-399.so")
        assert build.is_stale()
        with pytest.raises(RuntimeError, match="build it again"):
            _lib._native()
    _lib._native()


def test_a_binding_whose_origin_is_unknown_is_stale(elsewhere):
    with open(build.BINDING_PATH, "w"):
        pass
    assert build._binding_is_stale()
    with open(build.BINDING_PATH + ".for", "w") as f:
        f.write(build._installed())
    assert not build._binding_is_stale()
    os.remove(build.BINDING_PATH)
    with pytest.raises(RuntimeError, match="missing"):
        build.check_binding()
