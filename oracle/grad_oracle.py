"""Plain CPU oracle of the global gradient norm and clipping.

TEST INFRASTRUCTURE ONLY, like the other oracles here: only the test suite
imports it, and it shares no code with the library.

The GPT-2 lecture pages clip the global norm of the gradients at 1.0 before
every optimizer step.  Over every element of every tensor:

    norm   = scale * sqrt(sum g^2)
    c      = min(1, max_norm / (norm + 1e-6));  1 when max_norm = inf
    factor = scale * c
    g'     = fp32(g) * factor

Readings taken where the pages are silent:

  C1 epsilon      1e-6 is added to the norm before the division
  C2 precision    the sum, the root and c are held in fp64; norm and factor
                  are each rounded once, to fp32; g' is one fp32 product, and
                  one more rounding (nearest even) where it is stored in 16 bits
  C3 specials     a NaN among the gradients makes norm and factor NaN, an
                  infinity makes norm inf (and c = 0 under a finite limit)
"""

from __future__ import annotations

import math

import numpy as np

from .muon_oracle import bf16_round


def norm_factor(grads, max_norm=math.inf, scale=1.0):
    """(norm, factor) in fp64, before their rounding to fp32."""
    total = math.fsum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)
    norm = float(np.float32(scale)) * math.sqrt(total)
    if math.isnan(norm):
        return norm, norm
    limit = float(np.float32(max_norm))
    c = 1.0 if math.isinf(limit) else min(1.0, limit / (norm + 1e-6))
    return norm, float(np.float32(scale)) * c


def clipped(g, factor):
    """g' in fp32: g holds the gradient's values, factor is the fp32 one."""
    with np.errstate(invalid="ignore", over="ignore"):
        return np.asarray(g, np.float32) * np.float32(factor)


def rounded(v, kind):
    """fp32 values rounded to a type, as fp32 values."""
    if kind == "fp32":
        return np.asarray(v, np.float32)
    if kind == "fp16":
        with np.errstate(over="ignore"):
            return np.asarray(v, np.float32).astype(np.float16).astype(np.float32)
    return bf16_round(np.asarray(v, np.float32))
