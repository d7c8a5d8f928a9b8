"""The library and the expert layer's extension module are two builds: what needs the one does not need the other."""
import sysconfig

import pytest

import persistent_tile_scheduled_gb300 as pts
from persistent_tile_scheduled_gb300 import _build, experts, gemm


@pytest.fixture
def built():
    pts.build()


def no_compiler():
    raise RuntimeError("nvcc not found")


def test_the_library_does_not_need_the_module(built, monkeypatch, tmp_path):
    """A missing extension module neither makes the library stale nor keeps it from loading."""
    monkeypatch.setattr(_build, "EXPERTS", str(tmp_path / "none.so"))
    monkeypatch.setattr(_build, "nvcc", no_compiler)
    monkeypatch.setattr(gemm, "_lib", None)
    assert _build.up_to_date() and _build.build() == _build.LIB
    assert pts.load().gemm_status_string(0)


def test_the_module_needs_the_interpreters_headers_and_says_so(built, monkeypatch, tmp_path):
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    monkeypatch.setattr(_build, "EXPERTS", str(tmp_path / "none.so"))
    monkeypatch.setattr(_build, "nvcc", no_compiler)
    with pytest.raises(RuntimeError, match="Python.h"):
        _build.build_experts()
    assert _build.build() == _build.LIB


def test_every_interpreter_has_a_module_of_its_own():
    assert _build.EXPERTS.endswith("pts_experts" + sysconfig.get_config_var("EXT_SUFFIX"))


def test_other_names_do_not_load_the_module(monkeypatch):
    calls = experts._Calls()
    monkeypatch.setattr(experts, "load", no_compiler)
    for name in ("__wrapped__", "expert_sorted"):
        with pytest.raises(AttributeError):
            getattr(calls, name)
