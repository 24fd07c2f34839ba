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
