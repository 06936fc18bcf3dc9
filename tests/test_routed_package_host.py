"""The routed products' Python binding and its place in the package and the build, without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

from dense_gemm_sgemm_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_operands_of_two_devices_are_refused():
    # every tensor of a call passes this comparison before anything is allocated or launched
    torch = pytest.importorskip("torch")
    from dense_gemm_sgemm_gb300 import routed

    same = routed._routed.same_device
    same(torch.device("cuda:0"), torch.device("cuda:0"))
    same(torch.device("cuda:1"), torch.device("cuda:1"))
    with pytest.raises(ValueError, match="cuda:1"):
        same(torch.device("cuda:0"), torch.device("cuda:1"))
    with pytest.raises(TypeError):
        same("cuda:0", torch.device("cuda:0"))


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own, with one small source in the library's place."""
    for name in ("LIB_PATH", "BINDING_PATH", "BINDING_ERROR", "BINDING_FOR"):
        if hasattr(build, name):
            monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    source = tmp_path / "one.cu"
    source.write_text('extern "C" __attribute__((visibility("default"))) int one(void) { return 1; }')
    monkeypatch.setattr(build, "_sources", lambda: [str(source)])
    return tmp_path


def test_the_library_builds_without_torch(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert ctypes.CDLL(build.build()).one() == 1
    assert not os.path.exists(build.BINDING_PATH)
    assert "torch" in build.binding_error()


def test_the_library_builds_without_a_host_compiler(elsewhere, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", "false")
    open(build.BINDING_PATH, "w").close()  # one of older sources is not left behind
    assert ctypes.CDLL(build.build(force=True)).one() == 1
    assert not os.path.exists(build.BINDING_PATH)
    assert build.binding_error()


def test_why_there_is_no_binding_is_said_on_import(elsewhere, monkeypatch):
    pytest.importorskip("torch")
    from dense_gemm_sgemm_gb300 import routed

    monkeypatch.setenv("CXX", "false")
    build.build()
    with pytest.raises(ImportError, match="compiling the binding failed"):
        routed._load_binding()


def test_another_torch_makes_the_binding_stale(elsewhere, monkeypatch):
    torch = pytest.importorskip("torch")
    from dense_gemm_sgemm_gb300 import routed

    built = []

    def compile_binding(nvcc, obj):
        built.append(torch.__version__)
        return build.BINDING_SRC, 0, ""

    def link_binding(obj):
        open(build.BINDING_PATH, "w").close()
        build.note_torch()

    monkeypatch.setattr(build, "_compile_binding", compile_binding)
    monkeypatch.setattr(build, "_link_binding", link_binding)
    build.build()
    assert build.up_to_date()
    build.build()
    assert len(built) == 1
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not build.up_to_date()
    with pytest.raises(ImportError, match="99.0"):  # not loaded either
        routed._load_binding()
    build.build()
    assert built[1:] == ["99.0"] and build.up_to_date()


def test_a_failed_binding_is_tried_again_when_torch_changes(elsewhere, monkeypatch):
    torch = pytest.importorskip("torch")
    tried = []
    monkeypatch.setattr(build, "_compile_binding", lambda nvcc, obj: (build.BINDING_SRC, 1, tried.append(1) or "no"))
    build.build()
    build.build()
    assert len(tried) == 1 and build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not build.up_to_date()
    build.build()
    assert len(tried) == 2


def test_star_import_works_without_torch_and_binding():
    code = """
import sys
sys.modules["torch"] = None
from dense_gemm_sgemm_gb300 import *
assert gemm_version() >= 200 and "matmul" in globals()
import dense_gemm_sgemm_gb300 as g
try:
    g.moe_route
except ImportError:
    pass
else:
    raise SystemExit("routed products without torch")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build.ROOT)


def test_routed_names_by_attribute_and_by_name():
    pytest.importorskip("torch")
    import dense_gemm_sgemm_gb300 as g
    from dense_gemm_sgemm_gb300 import moe_route, routed

    assert g.moe_route is moe_route is routed.moe_route
    assert all(getattr(g, name) is getattr(routed, name) for name in routed.__all__)
