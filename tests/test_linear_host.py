"""CPU checks of the layers' products and of dropout: the host code under
sanitizers, refusals at the C entries and in the binding, and the oracle
against closed forms and published values."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from optimizer_muon_step_amd import _lib
from oracle import linear_oracle as lo

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
    exe = tmp_path / "linear_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-I", "/opt/rocm/include", "-I", CSRC, os.path.join(CSRC, "linear_host.cpp"),
           os.path.join(CSRC, "plan_host.cpp"), os.path.join(ROOT, "tests", "native", "linear_check.cpp"),
           "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no host C compiler")
def test_binding_structs_lie_as_the_header_says(tmp_path):
    """Size and field offsets of the ctypes structures against a C compiler's."""
    structs = {"muon_linear_t": _lib.MuonLinear, "muon_linear_dw_t": _lib.MuonLinearDw, "muon_dropout_t": _lib.MuonDropout}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "muon.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    cmd = ["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           str(src), "-o", str(tmp_path / "t")]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "t")], capture_output=True, text=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def test_entries_refuse_before_any_hip_call(lib):
    """Addresses that no GPU has: a refusal must come before they are used."""
    text = lambda: lib.muon_last_error().decode()  # noqa: E731
    good = dict(m=64, k=64, n=64, x=0x100000, w=0x200000, y=0x300000, ldx=64, ldw=64, ldy=64, x_type=1, w_type=1, y_type=1)

    def linear(entry, ws=None, nbytes=0, **kw):
        return entry(ctypes.byref(_lib.MuonLinear(**{**good, **kw})), ws, nbytes, None)

    assert lib.muon_linear(None, None, 0, None) == -1 and "NULL" in text()
    assert linear(lib.muon_linear, k=0) == -1 and "k = 0" in text()
    assert linear(lib.muon_linear, x_type=0) == -1 and "x_type" in text()
    assert linear(lib.muon_linear, act=9) == -1 and "act" in text()
    assert linear(lib.muon_linear, dropout=1.5) == -1 and "dropout" in text()
    assert linear(lib.muon_linear, y=0x100000) == -1 and "overlaps" in text()
    assert linear(lib.muon_linear, x=0x100002, k=7) == -1 and "workspace is NULL" in text()
    assert linear(lib.muon_linear, x=0x100002, k=7, ws=0x500000, nbytes=64) == -2 and "needs" in text()
    assert linear(lib.muon_linear_dx, bias=0x400000, bias_type=1) == -1 and "bias" in text()
    assert linear(lib.muon_linear_dx, act=1) == -1 and "preact" in text()
    assert lib.muon_linear_workspace_bytes(ctypes.byref(_lib.MuonLinear(**good)), 0) == 0
    assert lib.muon_linear_workspace_bytes(ctypes.byref(_lib.MuonLinear(**{**good, "w_type": 0, "n": 7})), 1) >= 2 * 64 * 8 * 2
    assert lib.muon_linear_workspace_bytes(ctypes.byref(_lib.MuonLinear(**{**good, "n": 0})), 0) == 0 and "n = 0" in text()
    dw = dict(m=64, k=64, n=64, x=0x100000, dz=0x200000, dw=0x300000, ldx=64, lddz=64, lddw=64, type=1)
    assert lib.muon_linear_dw(ctypes.byref(_lib.MuonLinearDw(**{**dw, "dw": 0x200000})), None, 0, None) == -1 and "overlaps" in text()
    assert lib.muon_linear_dw(ctypes.byref(_lib.MuonLinearDw(**{**dw, "type": 0})), None, 0, None) == -1 and "type" in text()
    assert lib.muon_linear_dw_workspace_bytes(ctypes.byref(_lib.MuonLinearDw(**{**dw, "m": 100000}))) > 0
    d = dict(m=4, n=4, x=0x100000, y=0x200000, ldx=4, ldy=4)
    assert lib.muon_dropout(ctypes.byref(_lib.MuonDropout(**{**d, "dropout": -1.0})), None) == -1 and "dropout" in text()
    assert lib.muon_dropout(ctypes.byref(_lib.MuonDropout(**{**d, "y": 0x100004})), None) == -1 and "overlaps" in text()
    # nothing to do: no device needed
    assert linear(lib.muon_linear, m=0, x=None, y=None) == 0
    assert lib.muon_linear_dw(ctypes.byref(_lib.MuonLinearDw(**{**dw, "m": 0, "accumulate": 1})), None, 0, None) == 0
    assert lib.muon_dropout(ctypes.byref(_lib.MuonDropout(**{**d, "m": 0})), None) == 0


def test_binding_refuses():
    import torch

    import optimizer_muon_step_amd as mu
    x, w, y = torch.zeros(4, 8).bfloat16(), torch.zeros(8, 16).bfloat16(), torch.zeros(4, 16).bfloat16()
    for call in (lambda: mu.muon_linear(x, w), lambda: mu.muon_linear_dx(y, w), lambda: mu.muon_linear_dw(x, y, torch.zeros(8, 16)),
                 lambda: mu.muon_dropout(x, 0.1, (1, 2))):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="expected a tensor"):
        mu.muon_linear(None, w)
    with pytest.raises(ValueError, match="not Double"):
        mu.muon_dropout(torch.zeros(3).double(), 0.1, (1, 2))
    with pytest.raises(ValueError, match="act"):
        mu.muon_linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="act"):
        mu.muon_linear(x, w, act=["gelu"])
    with pytest.raises(ValueError, match="out_dtype"):
        mu.muon_linear(x, w, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        mu.muon_dropout(x, "0.1", (1, 2))
    with pytest.raises(TypeError):
        mu.muon_linear(x, w, dropout=None)


def test_binding_fails_loudly_without_its_calls(monkeypatch):
    import sys

    import optimizer_muon_step_amd as mu
    monkeypatch.setattr(_lib, "_tensor_calls", None)
    monkeypatch.delattr(mu, "_tensor_calls", raising=False)
    monkeypatch.setitem(sys.modules, "optimizer_muon_step_amd._tensor_calls", None)
    with pytest.raises(RuntimeError, match="no fallback"):
        mu.muon_dropout(None, 0.1, (1, 2))


def test_philox_known_answers():
    """The generator's published test vectors, 10 rounds (the authors'
    Random123 distribution, kat_vectors), which fix its rounds and key steps."""
    full = 0xFFFFFFFF
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((full,) * 4, (full,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for counter, key, want in cases:
        assert tuple(int(w) for w in lo.philox(counter, key, rounds=10)) == want


def test_oracle_closed_forms():
    z = np.linspace(-9, 9, 2001)
    for kind in (None, "gelu", "relu", "relu2"):
        h = 1e-5
        away = np.abs(z) > 1e-3  # from the corners
        diff = (lo.act(z + h, kind) - lo.act(z - h, kind)) / (2 * h)
        # a central difference is off by h^2 / 6 of the third derivative (below 10) and by rounding, 2^-52 of up to 81 over 2 h
        assert np.all(np.abs(diff - lo.slope(z, kind))[away] < 2e-9 + 81 * 2.0 ** -52 / h)
    assert lo.act(np.array([0.0, 30.0, -30.0]), "gelu").tolist() == [0.0, 30.0, -0.0]
    # 0.5 z (1 + tanh(u)), the form the pages give, where it does not cancel
    z = np.linspace(-2, 6, 100)
    want = 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    assert np.allclose(lo.act(z, "gelu"), want, rtol=1e-13, atol=1e-15)


def test_oracle_mask():
    # each word of 32 bits serves two elements, low half first, in groups of 8 columns
    b = lo.bits(3, 20, seed=5 + (7 << 32), step=11, site=13)
    for r in (0, 2):
        for c in (0, 1, 7, 8, 19):
            words = [int(w) for w in lo.philox((c // 8, r, 13, 11), (5, 7))]
            assert b[r, c] == (words[c % 8 // 2] >> (16 * (c % 2))) & 0xFFFF
    assert lo.border(0.5) == 32768 and lo.border(0.0) == 0 and lo.border(0.1) == 6554
    f = lo.keep_factor(64, 256, 0.25, 1, 2, 3)
    assert set(np.unique(f)) == {0.0, 65536 / 49152} and abs((f != 0).mean() - 0.75) < 6 * math.sqrt(0.1875 / f.size)
    # one row after another of a larger matrix
    assert np.array_equal(lo.bits(5, 24, 9, 1, 2)[2:], lo.bits(3, 24, 9, 1, 2, row0=2))


def test_oracle_gradients_by_differences():
    """The backward formulas against central differences of the forward one, in fp64."""
    rng = np.random.default_rng(3)
    m, k, n = 5, 7, 6
    x, w1, b1, w2 = (rng.standard_normal(s) for s in ((m, k), (k, n), (n,), (n, k)))
    res, up = rng.standard_normal((m, k)), rng.standard_normal((m, k))
    f1, f2 = lo.keep_factor(m, n, 0.3, 1, 2, 3), lo.keep_factor(m, k, 0.3, 1, 2, 4)
    for kind in ("gelu", "relu", "relu2"):
        def loss(x, w1, b1, w2):
            h, _ = lo.linear(x, w1, b1, kind, f1)
            return float((lo.linear(h, w2, None, None, f2, res)[0] * up).sum())
        h, z = lo.linear(x, w1, b1, kind, f1)
        dz2 = lo.through(up, factor=f2)
        dz1 = lo.through(dz2 @ w2.T, kind, z, f1)
        grads = (dz1 @ w1.T, x.T @ dz1, dz1.sum(0), h.T @ dz2)
        args = (x, w1, b1, w2)
        for i, g in enumerate(grads):
            for _ in range(4):
                at = tuple(rng.integers(0, s) for s in args[i].shape)
                step = 1e-6
                hi, lo_ = [a.copy() for a in args], [a.copy() for a in args]
                hi[i][at] += step
                lo_[i][at] -= step
                diff = (loss(*hi) - loss(*lo_)) / (2 * step)
                assert abs(diff - g[at]) <= 1e-6 * max(1.0, abs(g[at])), (kind, i, at)
