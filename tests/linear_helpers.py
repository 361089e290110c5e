"""Inputs and error bounds shared by the tests of the layers' products and of
dropout.

Bounds are derived, element by element.  A product of two 16-bit values is
exact in fp32; a sum of k of them in any order errs by less than k steps of
2^-23 of the sum of their absolute values (a full step for every addition, so
whether it rounds or truncates does not matter).  What follows is counted in
roundings of 2^-24 relative to the value they happen at, and the store in half a step of
the output's type."""
from __future__ import annotations

import numpy as np

from gpu_helpers import torch_mod
from oracle import linear_oracle as lo

U = 2.0 ** -24
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# half of the smallest step, that of subnormal values
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}


def dtype(kind):
    torch = torch_mod()
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[kind]


def values(t):
    return t.detach().double().cpu().numpy()


def make(rng, shape, kind, std=1.0, offset=0, gap=0, order="rows", fill=0.0):
    """A matrix on the GPU, `offset` elements into its buffer, rows `gap` elements
    longer apart than they are; order 'columns': stored transposed.  What lies
    around it holds `fill`."""
    torch = torch_mod()
    r, c = shape if order == "rows" else shape[::-1]
    buf = torch.full((offset + max(1, r) * (c + gap) + 64,), fill, dtype=dtype(kind), device="cuda")
    view = buf[offset:].as_strided((r, c), (c + gap, 1))
    view.copy_(torch.from_numpy((rng.standard_normal((r, c)) * std).astype(np.float32)))
    return view if order == "rows" else view.T


def outside_unchanged(view, fill):
    """Everything of the buffer that holds `view` but the view itself still holds `fill`."""
    torch = torch_mod()
    n = view.untyped_storage().nbytes() // view.element_size()
    whole = torch.empty(0, dtype=view.dtype, device=view.device).set_(view.untyped_storage(), 0, (n,), (1,))
    mark = torch.zeros(n, dtype=torch.bool, device=view.device)
    mark.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    rest = whole[~mark]
    return bool(torch.isnan(rest).all()) if fill != fill else bool((rest == fill).all())


def stored(err, v, kind):
    """Bound after rounding a value that may be `err` off v to a type."""
    return err + HALF[kind] * (np.abs(v) + err) * (1 + 2 * HALF[kind]) + TINY[kind]


def act_bound(z, err, kind):
    """Error of act(z) when z may be `err` off, with the evaluation's own.
    GELU: its slope stays below 1.13; the exponent 2u comes from 6 roundings and
    exp turns its error into a relative one, and 8 roundings follow."""
    if kind == "gelu":
        e = 2 * lo.C * np.abs(z + 0.044715 * z ** 3)
        return 1.13 * err + np.abs(lo.act(z, kind)) * U * (6 * np.minimum(e, 100.0) + 8) + 2.0 ** -120
    if kind == "relu2":
        return (2 * np.abs(z) + err) * err + U * z * z
    return err


def slope_bound(z, kind):
    """Evaluation error of act'(z) on an exact z.  GELU: s + z s (1 - s) 2u', s and
    1 - s each to a relative 6 |2u| + 10 roundings at most, 4 more for the rest of the
    second term and one for the sum; beyond |z| = 10 the kernels take 0 and 1, less
    than 1e-34 off."""
    if kind == "gelu":
        e = np.minimum(2 * lo.C * np.abs(z + 0.044715 * z ** 3), 100.0)
        s, rest = lo.gate_of(z)
        second = np.abs(z) * s * rest * 2 * lo.C * (1 + 3 * 0.044715 * z * z)
        return U * ((6 * e + 11) * s + (12 * e + 25) * second) + 1e-34
    return U * np.abs(lo.slope(z, kind))


def check(got, want, bound, what, kind=None):
    """Elementwise |got - want| <= bound; says by how much it was kept."""
    got = values(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    if kind == "fp16":  # the largest value is 65504 and the next step is 32: from 65520 on rounding gives an infinity
        off[np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= 65520)] = 0
    bad = ~(off <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / bound, 0)), off.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound, e.g. at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {bound[i]:.3e}")
