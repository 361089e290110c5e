"""CPU checks of the layer products at the limits of a launch: the host code
under sanitizers, what the inputs of the long GPU tests show, and the oracle at
special values."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import linear_oracle as lo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "optimizer_muon_step_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_host_code_at_the_limits_of_a_launch(tmp_path):
    exe = tmp_path / "linear_limits_check"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=undefined", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-I", "/opt/rocm/include", "-I", CSRC, os.path.join(CSRC, "linear_host.cpp"),
           os.path.join(CSRC, "plan_host.cpp"), os.path.join(ROOT, "tests", "native", "linear_limits_check.cpp"),
           "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stdout + build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr


@pytest.mark.parametrize("k", [1608, 20000])
def test_a_lost_slice_shows(k):
    """Values of -1, 0 and 1 (a half, a quarter each): a slice of 64 that is left out, or read in the
    place of another, changes nearly nine sums in ten.  Its own sum has a variance of
    64 / 4 and is 0 for 1 in sqrt(2 pi 16) = 10; the difference of two, for 1 in 14."""
    rng = np.random.default_rng(k)
    a, b = (rng.integers(0, 4, s).astype(np.float32) for s in ((k, 100), (k, 120)))
    a, b = (np.where(v < 2, 0, 2 * v - 5) for v in (a, b))
    whole = a.T @ b
    lost, stale = slice(k // 128 * 64, k // 128 * 64 + 64), slice(64, 128)
    without = whole - a[lost].T @ b[lost]
    assert np.mean(without != whole) > 0.85
    assert np.mean(without + a[stale].T @ b[stale] != whole) > 0.85


def test_oracle_at_special_values():
    """act and act' of a NaN are NaN; relu's and relu2's slope at zeros and infinities."""
    nan, inf = float("nan"), float("inf")
    for kind in ("gelu", "relu", "relu2"):
        assert np.isnan(lo.act(np.array([nan]), kind)).all() and np.isnan(lo.slope(np.array([nan]), kind)).all()
    z = np.array([0.0, -0.0, 3.0, -3.0, inf, -inf])
    assert lo.slope(z, "relu").tolist() == [0, 0, 1, 0, 1, 0] and lo.slope(z, "relu2").tolist() == [0, 0, 6, 0, inf, 0]
    # a dropped element does not see it
    assert lo.through(np.ones(2), "relu", np.array([nan, nan]), np.array([0.0, 2.0])).tolist()[0] == 0
