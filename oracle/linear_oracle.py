"""Plain CPU oracle of the hidden layers' products and of dropout.

TEST INFRASTRUCTURE ONLY, like the other oracles here: only the test suite
imports it, and it shares no code with the library.  fp64 throughout, from the
operands' own values:

    linear   z = x w + bias;  y = residual + drop(act(z))
    dx       residual + drop(dz w^T) act'(preact)
    dw       x^T dz;  dbias the sums of dz over its rows
    dropout  residual + drop(x) act'(preact)

Readings taken where the pages are silent:

  L1 GELU         the tanh form (the pages name the approximation of GPT-2)
  L2 generator    Philox 4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random
                  numbers: as easy as 1, 2, 3", SC'11) with 7 rounds; counter
                  (column // 8, row, site, step), key (seed low, seed high)
  L3 mask         16 bits an element; kept where they are >= t = floor(2^16 p +
                  1/2), at most 65535, and then times 2^16 / (2^16 - t); p is
                  the fp32 value of the argument
  L4 NaN          act and act' of a NaN are NaN, in every activation; a dropped
                  element is 0 whatever it was
"""

from __future__ import annotations

import math

import numpy as np

C = math.sqrt(2.0 / math.pi)


def philox(counter, key, rounds=7):
    """Words of Philox 4x32: counter four and key two arrays (or ints) of 32 bits."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def border(p):
    return min(65535, math.floor(65536.0 * float(np.float32(p)) + 0.5))


def bits(rows, cols, seed, step, site, row0=0):
    """The 16 random bits of every element."""
    groups = -(-cols // 8)
    g = np.arange(groups, dtype=np.uint64)[None, :].repeat(rows, 0)
    r = (row0 + np.arange(rows, dtype=np.uint64))[:, None].repeat(groups, 1)
    words = philox((g, r, np.uint64(site), np.uint64(step)), (seed % 2 ** 32, seed >> 32))
    words = [np.broadcast_to(w, (rows, groups)) for w in words]
    out = np.empty((rows, groups, 8), np.uint32)
    for i in range(8):
        out[:, :, i] = (words[i // 2] >> np.uint64(16 * (i % 2))) & np.uint64(0xFFFF)
    return out.reshape(rows, groups * 8)[:, :cols]


def keep_factor(rows, cols, p, seed, step, site):
    """What drop() multiplies each element by: 0 or the scale."""
    t = border(p)
    return np.where(bits(rows, cols, seed, step, site) >= t, 65536.0 / (65536.0 - t), 0.0)


def gate_of(z):
    """(1 + tanh(u)) / 2 and (1 - tanh(u)) / 2 without cancellation, u = C (z + 0.044715 z^3):
    with 1 + tanh(u) itself the slope below z = -6 would be right to 2 digits only."""
    with np.errstate(over="ignore"):
        two_u = 2.0 * C * (z + 0.044715 * z ** 3)
        return 1.0 / (1.0 + np.exp(-two_u)), 1.0 / (1.0 + np.exp(two_u))


def act(z, kind):
    if kind == "gelu":
        return z * gate_of(z)[0]
    if kind == "relu":
        return np.where(z < 0, 0.0, z)
    if kind == "relu2":
        return np.where(z < 0, 0.0, z * z)
    return z


def slope(z, kind):
    if kind == "gelu":
        gate, rest = gate_of(z)
        return gate + z * gate * rest * 2.0 * C * (1.0 + 3 * 0.044715 * z * z)
    if kind == "relu":
        return np.where(z <= 0, 0.0, np.where(z > 0, 1.0, z))
    if kind == "relu2":
        return np.where(z <= 0, 0.0, 2.0 * z)
    return np.ones_like(z)


def linear(x, w, bias=None, kind=None, factor=None, residual=None):
    """(y, z) in fp64; factor: keep_factor of the output, or None."""
    z = x @ w
    if bias is not None:
        z = z + bias
    y = act(z, kind)
    if factor is not None:
        y = np.where(factor == 0, 0.0, y * factor)
    return (y if residual is None else residual + y), z


def through(v, kind=None, preact=None, factor=None, residual=None):
    """residual + drop(v) act'(preact): the epilogue of dx, and dropout."""
    if kind is not None:
        v = v * slope(preact, kind)
    if factor is not None:
        v = np.where(factor == 0, 0.0, v * factor)
    return v if residual is None else residual + v
