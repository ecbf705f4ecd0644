"""Penalties, biases and grammar masks on logits rows, and the table of tokens
they read (float64 / Python integers).

TEST INFRASTRUCTURE ONLY: part of the CPU oracle.  Only tests may import it.

Row j of a sequence follows the table's tokens, the ctx tokens and drafts 1..j
of its block.  A known token (in the prompt, or emitted) has a positive logit
divided and any other multiplied by the repetition penalty; every emitted token
loses frequency x times + presence; biases add; barred tokens become -inf.
Draft row j takes what target row j takes ("Accelerating Large Language Model
Decoding with Speculative Sampling", section "Modified rejection sampling":
such changes are made to both distributions before the scheme).
"""
import math

import numpy as np

from .sampling import DEV_BAD_PARAM, DEV_BAD_TOKEN, to_f64


def count_tokens(counts, tokens, start, num_accepted=None, slots=None, prompt=False, reset=False):
    """(counts', seen', status): counts [S, V] int32 (sign bit: prompt)."""
    c = [[int(x) & 0xFFFFFFFF for x in row] for row in np.asarray(counts)]
    V, B, status = len(c[0]), len(start) - 1, 0
    rows = list(range(B)) if slots is None else [int(s) for s in slots]
    good = [0 <= s < len(c) for s in rows]
    if any(not g and s != -1 for g, s in zip(good, rows)):
        status |= DEV_BAD_PARAM
    if reset:
        for s, g in zip(rows, good):
            if g:
                c[s] = [0] * V
    for i in range(B):
        n = int(start[i + 1]) - int(start[i])
        if num_accepted is not None:
            n = min(n, int(num_accepted[i]) + 1)
        for t in tokens[int(start[i]):int(start[i]) + max(n, 0)]:
            if not good[i]:
                continue
            if not 0 <= int(t) < V:
                status |= DEV_BAD_TOKEN
            elif prompt:
                c[rows[i]][int(t)] |= 1 << 31
            else:
                c[rows[i]][int(t)] += 1
    out = np.array(c, dtype=np.uint32).view(np.int32)
    return out, seen_bits(out), status


def seen_bits(counts):
    """[S, ceil(V / 32)] int32: bit t % 32 of word t / 32 where counts is not 0."""
    S, V = counts.shape
    pad = np.zeros((S, (V + 31) // 32 * 32), dtype=bool)
    pad[:, :V] = counts != 0
    return np.packbits(pad, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def allowed_tokens(words, V):
    """Truth per token of one mask row of 32-bit words."""
    w = np.ascontiguousarray(words).astype("<i4").view(np.uint8)
    return np.unpackbits(w, bitorder="little")[:V].astype(bool)


def adjust_row(x, prompt, times, repetition, presence, frequency, bias, allowed):
    """One row in float64: x, prompt (truth), times (integers), bias [V]."""
    y = np.array(x, dtype=np.float64)
    known = prompt | (times > 0)
    with np.errstate(invalid="ignore", over="ignore"):
        up = known & (y > 0)
        y[up] = y[up] / repetition
        rest = known & ~up
        y[rest] = y[rest] * repetition
        hit = times > 0
        y[hit] = y[hit] - (frequency * times[hit] + presence)
        y = np.where(bias != 0, y + bias, y)
    if allowed is not None:
        y[~allowed] = -math.inf
    return y


def adjust_logits(target, cu_q, draft=None, draft_tokens=None, counts=None, slots=None, ctx=None,
                  repetition=1.0, presence=0.0, frequency=0.0, bias=None, mask=None,
                  mask_rows=None):
    """(target', draft', status) in float64.  repetition / presence / frequency:
    a number or one per sequence; bias: per sequence a list of (token, value);
    mask [M, W] words; ctx [n, B]; a failing sequence's rows are NaN."""
    t64 = to_f64(np.asarray(target))
    d64 = None if draft is None else to_f64(np.asarray(draft))
    V, B, status = t64.shape[1], len(cu_q) - 1, 0

    def of(v, i):
        return float(v[i]) if np.ndim(v) else float(np.float32(v))

    for i in range(B):
        r0, r1 = int(cu_q[i]), int(cu_q[i + 1])
        rep, pres, freq = of(repetition, i), of(presence, i), of(frequency, i)
        slot = -1 if counts is None else i if slots is None else int(slots[i])
        rows = [r if mask_rows is None else int(mask_rows[r]) for r in range(r0, r1)]
        fails = not (2.0 ** -64 <= rep <= 2.0 ** 64 and all(map(math.isfinite, (pres, freq)))) or slot < -1 or \
            (counts is not None and slot >= len(counts)) or \
            (mask is not None and any(not -1 <= m < len(mask) for m in rows))
        word = np.zeros(V, dtype=np.int64)
        if not fails and slot >= 0:
            word = np.asarray(counts[slot]).view(np.uint32).astype(np.int64)
        prompt, times = word >= 1 << 31, word & 0x7FFFFFFF
        for t in ([] if ctx is None else [int(c[i]) for c in ctx]):
            if 0 <= t < V:
                times[t] += 1
        add = np.zeros(V)
        for t, v in ([] if bias is None or fails else bias[i]):
            if 0 <= t < V:
                add[t] = v              # of a token named twice the last entry holds
            else:
                status |= DEV_BAD_TOKEN
        if fails:
            status |= DEV_BAD_PARAM
        for j, r in enumerate(range(r0, r1)):
            if j and draft_tokens is not None:
                t = int(draft_tokens[r - i - 1])
                if 0 <= t < V:
                    times[t] += 1
            allowed = None
            if not fails and mask is not None and rows[j] >= 0:
                allowed = allowed_tokens(mask[rows[j]], V)
            for x, row in ((t64, r), (d64, r - i)):
                if x is None or (x is d64 and r == r1 - 1):
                    continue
                x[row] = math.nan if fails else adjust_row(x[row], prompt, times, rep, pres, freq,
                                                           add, allowed)
    return t64, d64, status
