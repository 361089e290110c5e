"""CPU checks of the gradient norm, clipping and clipped steps: the host code
under sanitizers, refusals at the C entries and in the binding, and the oracle
against closed forms."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from optimizer_muon_step_amd import _lib
from oracle import grad_oracle as go

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "optimizer_muon_step_amd", "csrc")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from optimizer_muon_step_amd import build
        build.build()
    return _lib.load()


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_host_code_under_address_and_ub_sanitizers(tmp_path):
    exe = tmp_path / "grad_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-I", "/opt/rocm/include", "-I", CSRC, os.path.join(CSRC, "grad_host.cpp"),
           os.path.join(CSRC, "plan_host.cpp"), os.path.join(ROOT, "tests", "native", "grad_check.cpp"),
           "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr


def test_entries_refuse_before_any_hip_call(lib):
    """Addresses that no GPU has: a refusal must come before they are used."""
    g, o = _lib.ptr_array([0x100000]), _lib.ptr_array([0x200000])
    n1 = _lib.int64_array([64])
    import ctypes
    t32 = (ctypes.c_int * 1)(0)
    bad = (ctypes.c_int * 1)(7)
    rec, ws = 0x900000, 0xa00000
    text = lambda: lib.muon_last_error().decode()  # noqa: E731
    assert lib.muon_grad_norm(g, n1, bad, 1, 1.0, 1.0, rec, ws, None) == -1 and "dtypes[0] = 7" in text()
    assert lib.muon_grad_norm(g, n1, t32, 1, -1.0, 1.0, rec, ws, None) == -1 and "max_norm" in text()
    assert lib.muon_grad_norm(g, n1, t32, 1, 1.0, math.nan, rec, ws, None) == -1 and "scale" in text()
    assert lib.muon_grad_norm(g, n1, t32, 1, 1.0, 1.0, None, ws, None) == -1 and "record" in text()
    assert lib.muon_grad_norm(g, n1, t32, 1, 1.0, 1.0, rec, None, None) == -1 and "workspace" in text()
    assert lib.muon_grad_clip(g, o, n1, t32, bad, 1, 1.0, 1.0, rec, ws, None) == -1 and "out_dtypes" in text()
    assert lib.muon_grad_clip(g, _lib.ptr_array([0x100010]), n1, t32, t32, 1, 1.0, 1.0, rec, ws, None) == -1
    assert "overlaps" in text()
    P = [_lib.ptr_array([0x10000 * (k + 1)]) for k in range(4)]
    adamw = lambda **kw: lib.muon_adamw_step_clip(  # noqa: E731
        P[0], P[1], kw.get("t", t32), P[2], P[3], n1, None, 1, kw.get("lr", 1e-3), 0.9, 0.999, 1e-8,
        kw.get("step", 1), kw.get("rec", rec), None)
    assert adamw(step=0) == -1 and "step" in text()
    assert adamw(lr=math.inf) == -1 and "lr" in text()
    assert adamw(t=bad) == -1 and "grad_dtypes" in text()
    assert adamw(rec=0x10004) == -1 and "overlaps" in text()
    shapes = _lib.shape_array([(4, 4)])
    c = _lib.float_array([1.0, 0.0, 0.0])
    assert lib.muon_step_clip(P[0], P[1], P[2], shapes, 1, 0.02, 0.95, 1, c, None, 0x900001, None) == -1
    assert "record" in text()
    assert lib.muon_step_clip(P[0], P[1], P[2], shapes, 1, 0.02, 0.95, 1, c, None, 0x30000, None) == -1
    assert "overlaps" in text()
    # nothing to do: no device needed
    assert lib.muon_adamw_step_clip(None, None, None, None, None, None, None, 0, 1e-3, 0.9, 0.999, 1e-8, 1, rec,
                                    None) == 0
    assert lib.muon_step_clip(P[0], P[1], P[2], shapes, 0, 0.02, 0.95, 1, c, None, rec, None) == 0


def test_binding_refuses():
    import torch

    import optimizer_muon_step_amd as mu
    cpu = torch.zeros(4)
    for call in (lambda: mu.muon_grad_norm([cpu]), lambda: mu.muon_grad_clip([cpu], 1.0),
                 lambda: mu.muon_adamw_step([cpu], [cpu.bfloat16()], [cpu], [cpu], 1e-3)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="expected a tensor"):
        mu.muon_grad_norm([None])
    with pytest.raises(ValueError, match="list of tensors"):
        _lib.load_tensor_calls().grad_norm(3, 1.0, 1.0, None, 0, -1, 0)
    with pytest.raises(TypeError):
        mu.muon_grad_norm([], max_norm="1")
    with pytest.raises(ValueError, match="weight_decay"):
        mu.muon_adamw_step([], [], [], [], 1e-3, weight_decay=[0.1], clip=0)
    with pytest.raises(ValueError, match="weight_decay"):
        mu.muon_adamw_step([], [], [], [], 1e-3, weight_decay="x", clip=0)
    with pytest.raises(ValueError, match="record"):
        mu.muon_adamw_step([], [], [], [], 1e-3, clip=0)
    with pytest.raises(ValueError, match="record"):
        mu.muon_grad_norm([], record=torch.zeros(2))
    with pytest.raises(ValueError, match="bfloat16 or float16, not Double"):
        mu.muon_grad_norm([cpu.double()])
    with pytest.raises(ValueError, match="not Int"):
        mu.muon_grad_clip([cpu.int()], 1.0)
    with pytest.raises(ValueError, match="expected float32"):
        mu.muon_adamw_step([cpu.bfloat16()], [cpu.bfloat16()], [cpu], [cpu], 1e-3)


def test_binding_fails_loudly_without_its_calls(monkeypatch):
    import sys

    import optimizer_muon_step_amd as mu
    monkeypatch.setattr(_lib, "_tensor_calls", None)
    monkeypatch.delattr(mu, "_tensor_calls", raising=False)
    monkeypatch.setitem(sys.modules, "optimizer_muon_step_amd._tensor_calls", None)
    with pytest.raises(RuntimeError, match="no fallback"):
        mu.muon_grad_norm([])


def test_dense_layouts():
    import torch

    import optimizer_muon_step_amd as mu
    t = torch.zeros(4, 5, 6)
    for g in (t, t.permute(2, 0, 1), t[1:3], torch.zeros(1, 5).t(), torch.zeros(3, 1, 7).permute(2, 1, 0),
              torch.zeros(0, 3).t(), torch.zeros(())):  # only the device is wrong
        with pytest.raises(ValueError, match="on the GPU"):
            mu.muon_grad_norm([t, g])
    for g in (t[:, :1].permute(1, 2, 0), torch.zeros(4, 5)[:, :3], torch.zeros(1).expand(4), torch.zeros(8)[::2],
              t.to_sparse(), torch._neg_view(t)):
        with pytest.raises(ValueError, match=r"grads\[0\]: expected a dense tensor"):
            mu.muon_grad_norm([g])
    with pytest.raises(ValueError, match=r"params\[0\]: expected a contiguous tensor"):
        mu.muon_adamw_step([t.permute(2, 0, 1)], [t.half()], [t], [t], 1e-3)


def test_oracle_closed_forms():
    norm, factor = go.norm_factor([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert norm == 5.0 and factor == 1.0 / (5.0 + 1e-6)
    assert go.norm_factor([np.array([3.0, 4.0])], 10.0, 0.5) == (2.5, 0.5)
    assert go.norm_factor([], 0.0) == (0.0, 0.0) and go.norm_factor([]) == (0.0, 1.0)
    assert go.norm_factor([np.array([math.inf])], 1.0) == (math.inf, 0.0)
    n, f = go.norm_factor([np.array([math.nan])])
    assert math.isnan(n) and math.isnan(f)
    # halves and ties of the 16-bit roundings
    assert go.rounded(np.float32(1 + 2.0 ** -8), "bf16") == 1.0 and go.rounded(np.float32(1 + 3 * 2.0 ** -8), "bf16") == 1 + 2.0 ** -6
    assert go.rounded(np.float32(70000), "fp16") == np.inf and go.rounded(np.float32(2.0 ** -25), "fp16") == 0.0


class _Meddler:
    """A number whose reading changes a list of the call that reads it."""

    def __init__(self, change):
        self.change = change

    def __float__(self):
        self.change()
        return 0.5


def test_lists_that_change_while_a_call_reads_them(lib):
    """A call goes by its lists as they were when it read them: their lengths
    and their tensors stay the call's own."""
    import torch

    import optimizer_muon_step_amd as mu
    calls = _lib.load_tensor_calls()
    for k in range(4):
        lists = [[], [], [], []]
        wd = _Meddler(lambda: lists[k].append(torch.zeros(3)))  # noqa: B023
        adamw = lambda: calls.adamw_clip(*lists, wd, 1e-3, 0.9, 0.999, 1e-8, 1, None, -1, 0)  # noqa: B023,E731
        with pytest.raises(ValueError, match="on the GPU|same length"):
            adamw()  # the decays are read first: the lists are as they are now
    # decays that their own reading shortens: the call's are those it was given
    decays = [0.1, 0.2]
    decays[0] = _Meddler(decays.clear)
    with pytest.raises(ValueError, match="one value or one per tensor"):
        calls.adamw_clip([], [], [], [], decays, 1e-3, 0.9, 0.999, 1e-8, 1, None, -1, 0)
    params = []
    coeffs = (_Meddler(lambda: params.append(torch.zeros(3, 3))), 0.0, 0.0)
    mu.muon_step(params, [], [], coeffs=coeffs, updates=[], stream=0)


def test_refused_calls_give_back_their_references(lib):
    import sys

    import torch
    t = torch.zeros(2)
    tensors = [t]
    before = sys.getrefcount(t), sys.getrefcount(tensors)
    for _ in range(3):
        for grads in (tensors, (t,)):
            with pytest.raises(ValueError, match="on the GPU"):
                _lib.load_tensor_calls().grad_norm(grads, 1.0, 1.0, None, 0, -1, 0)
        del grads
    assert (sys.getrefcount(t), sys.getrefcount(tensors)) == before


def test_workspaces_are_kept_only_for_streams_that_stay(monkeypatch):
    """torch's own streams live as long as the process, so a handle of theirs
    names one stream.  Another handle may come to name a later stream while
    the earlier one's norm still runs: its calls share no workspace."""
    import types

    import torch

    import optimizer_muon_step_amd as mu
    zeros, current = torch.zeros, types.SimpleNamespace(stream_id=0)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(mu, "_norm_workspaces", {})
    for handle, stream_id in ((0, 0), (0x5000, 35), (0x5010, 67)):  # the default stream and two of the pool's
        current.stream_id = stream_id
        assert mu._norm_workspace(0, handle) is mu._norm_workspace(0, handle)
        assert mu._norm_workspace(0, handle) is not mu._norm_workspace(1, handle)
    kept = dict(mu._norm_workspaces)
    for handle in (1, 0x7000):  # handles from elsewhere: torch takes the handle as the id
        current.stream_id = handle
        first, second = mu._norm_workspace(0, handle), mu._norm_workspace(0, handle)
        assert first is not second and first.count_nonzero() == 0
    assert mu._norm_workspaces == kept
    # one of the pool's streams under its raw handle is the same stream
    current.stream_id = 0x5000
    assert mu._norm_workspace(0, 0x5000) is kept[0, 0x5000]


def test_the_per_thread_stream_is_refused():
    """Handle 2, hipStreamPerThread, is another stream in every host thread,
    but one stream to the allocator that a call takes its memory from."""
    import optimizer_muon_step_amd as mu
    for call in (lambda: mu.muon_grad_norm([], stream=2), lambda: mu.muon_grad_clip([], 1.0, stream=2),
                 lambda: mu._norm_workspace(0, 2)):
        with pytest.raises(ValueError, match="hipStreamPerThread"):
            call()


def test_the_plain_adamw_step_names_the_tensor_it_refuses():
    import torch

    import optimizer_muon_step_amd as mu
    t = torch.zeros(4)
    for lists, text in ((([t],) * 4, "params[0]: expected a contiguous float32 tensor on the GPU"),
                        (([3], [t], [t], [t]), "params[0]: expected a tensor")):
        with pytest.raises(ValueError) as refusal:
            mu.muon_adamw_step(*lists, 1e-3)
        assert str(refusal.value) == text
    with pytest.raises(ValueError) as refusal:
        mu.muon_adamw_untie(t, t, t)
    assert str(refusal.value) == "param: expected a contiguous float32 tensor on the GPU"
