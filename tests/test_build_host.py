"""Build configuration (CPU only): every per-source option names a compiled
source, the update kernel's fingerprint covers its sources and options, and
the built library carries a code object for gfx950."""
import os

import pytest

from optimizer_muon_step_amd import build as b


def test_source_flags_name_compiled_sources():
    for src in b.SOURCE_FLAGS:
        assert src in b.SOURCES, src
    for src in b.SOURCES + b.UPDATE_KERNEL_SOURCES:
        assert os.path.exists(os.path.join(b.CSRC, src)), src


def test_update_fingerprint_tracks_options(monkeypatch):
    f0 = b.update_kernel_fingerprint()
    assert f0 == b.update_kernel_fingerprint()
    monkeypatch.setitem(b.SOURCE_FLAGS, "kernels_ns.hip", ["-mllvm", "-some-option"])
    assert b.update_kernel_fingerprint() != f0
    monkeypatch.delitem(b.SOURCE_FLAGS, "kernels_ns.hip")
    assert b.update_kernel_fingerprint() == f0
    # options of other sources do not touch the update kernel
    monkeypatch.setitem(b.SOURCE_FLAGS, "kernels_momentum.hip", ["-mllvm", "-some-option"])
    assert b.update_kernel_fingerprint() == f0


def test_library_holds_gfx950_code():
    if not os.path.exists(b.LIB):
        pytest.skip("libmuon.so not built")
    with open(b.LIB, "rb") as f:
        data = f.read()
    assert b".hip_fatbin" in data                   # the device-code section
    assert b"amdgcn-amd-amdhsa--gfx950" in data     # a code object for gfx950


@pytest.mark.parametrize("missing", ["torch", "compiler", "headers"])
def test_the_library_builds_without_what_only_the_binding_needs(missing, monkeypatch, tmp_path, capsys):
    """libmuon.so and its C ABI need neither torch, nor Python's headers, nor a
    C++ host compiler.  Without one of them the binding's tensor calls are left
    out, with a notice; calls of an earlier build do not stay beside a new library."""
    import shutil
    import sys
    import sysconfig
    stale = tmp_path / "_tensor_calls.so"
    stale.write_bytes(b"")
    monkeypatch.setattr(b, "SOURCES", ["plan_host.cpp"])
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmuon.so"))
    monkeypatch.setattr(b, "TENSOR_CALLS", str(stale))
    monkeypatch.setattr(b, "build_c_example", lambda verbose=False: "")
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif missing == "compiler":
        monkeypatch.setattr(shutil, "which", lambda name: None)
    else:
        paths = sysconfig.get_paths()
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {**paths, "include": str(tmp_path)})
    assert b.build(out=b.LIB) == b.LIB and os.path.exists(b.LIB)
    assert not stale.exists()
    assert "_tensor_calls.so" in capsys.readouterr().err
