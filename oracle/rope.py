"""Rotary positions of block rows, and E4M3 rounding (float64).

TEST INFRASTRUCTURE ONLY: part of the CPU oracle.  Only tests may import it.

A pair (a, b) of a head at position t is the complex number a + i b times
m e^(i t f); the half layout pairs elements rot / 2 apart, the interleaved one
neighbours; elements from rot on stay.  Angles: t f reduced modulo 2 pi by
exact rational arithmetic on the float64 value of f / (2 pi), so that far
positions are as exact as near ones.
"""
import math
from fractions import Fraction

import numpy as np

from .sampling import e4m3_to_f64


def rope_frequencies(rot, base=10000.0, kind="plain", factor=1.0, trained=1, fast=32.0, slow=1.0,
                     low=1.0, high=4.0):
    """(radians per token of each pair [rot / 2], factor on cos and sin)."""
    out, m = [], 1.0
    for p in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if kind == "ntk" and rot > 2 else base
        f = b ** (-2 * p / rot)
        if kind == "linear":
            f = f / factor
        elif kind == "yarn":
            # the pair index at which a pair makes n turns over the trained length
            def where(n):
                return rot / 2 * math.log(trained / (2 * math.pi * n), base)
            lo, hi = max(math.floor(where(fast)), 0), min(math.ceil(where(slow)), rot - 1)
            x = min(max((p - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f, m = f * (x / factor + 1 - x), 1 + 0.1 * math.log(factor)
        elif kind == "banded":
            turns = trained * f / (2 * math.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                x = (turns - low) / (high - low)
                f = f * x + f / factor * (1 - x)
        out.append(f)
    return np.array(out), m


def angles(positions, freqs):
    """[n, pairs] angles in [-pi, pi] of integer positions."""
    out = np.empty((len(positions), len(freqs)))
    for p, f in enumerate(freqs):
        turn = Fraction(float(f) / (2 * math.pi))
        for r, t in enumerate(positions):
            x = turn * int(t)
            out[r, p] = 2 * math.pi * float(x - round(x))
    return out


def rope_rows(x, positions, freqs, layout="half", mscale=1.0):
    """x [R, H, D] float64 with its first 2 len(freqs) elements turned."""
    x = np.asarray(x, dtype=np.float64)
    h = len(freqs)
    y = x.copy()
    w = mscale * np.exp(1j * angles(positions, freqs))[:, None, :]
    if layout == "half":
        z = (x[..., :h] + 1j * x[..., h:2 * h]) * w
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    else:
        z = (x[..., 0:2 * h:2] + 1j * x[..., 1:2 * h:2]) * w
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = z.real, z.imag
    return y


def row_positions(cu_q, kv_len):
    """Positions of the block rows: row j of sequence i at kv_len[i] + j."""
    return [int(kv_len[i]) + j for i in range(len(cu_q) - 1)
            for j in range(int(cu_q[i + 1]) - int(cu_q[i]))]


def e4m3_nearest(y):
    """E4M3 codes (uint8) of float64 values: nearest, ties to the even code,
    saturating at +-448; NaN to 0x7F."""
    y = np.asarray(y, dtype=np.float64)
    grid = e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))        # 0 .. 448, ascending
    mag = np.minimum(np.abs(y), 448.0)
    hi = np.searchsorted(grid, np.nan_to_num(mag))              # grid[hi] >= mag
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = mag - grid[lo], grid[hi] - mag
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(y), 0x7F, code | (np.signbit(y).astype(np.int64) << 7))
    return code.astype(np.uint8)
