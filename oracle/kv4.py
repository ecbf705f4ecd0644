"""Per-head norms and the paged 4-bit KV cache (float64).

TEST INFRASTRUCTURE ONLY: part of the CPU oracle.  Only tests may import it.

E2M1 values are 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign; 16 of them share an E4M3
scale, a tensor a factor: x = code * scale * factor, scale = nearest E4M3 of
max|x| / (6 factor), code = nearest E2M1 of x / (scale factor).  A slab is 16
tokens of one KV head: K codes [16, D/2], K scales [16, D/16], V's the same; a
page is [Hkv, page / 16] slabs; token t of a sequence is in page table[t // page].
"""
import numpy as np

from .rope import e4m3_nearest
from .sampling import e4m3_to_f64, to_f64

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_nearest(y):
    """Codes 0..15 of float64 values: nearest, ties to the even code, saturating at +-6 (NaN: 7)."""
    y = np.asarray(y, dtype=np.float64)
    d = np.abs(np.where(np.isnan(y), 6.0, np.minimum(np.abs(y), 6.0))[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (code | (np.signbit(y) & ~np.isnan(y)) * 8).astype(np.uint8)


def e2m1_to_f64(codes):
    return np.concatenate([E2M1, -E2M1])[np.asarray(codes)]


def kv4_quantize(x, factor):
    """(codes [.., D], scale codes [.., D / 16]) of float64 x [.., D]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    scales = e4m3_nearest(np.abs(b).max(-1) / (6.0 * factor))       # (max of a NaN is NaN)
    unit = e4m3_to_f64(scales)[..., None] * factor
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(unit == 0, 0, e2m1_nearest(b / unit))
    return codes.reshape(x.shape).astype(np.uint8), scales


def kv4_values(codes, scales, factor):
    """float64 values of codes [.., D] and scale codes [.., D / 16]."""
    v = e2m1_to_f64(codes)
    unit = e4m3_to_f64(scales) * factor
    return (v.reshape(*v.shape[:-1], v.shape[-1] // 16, 16) * unit[..., None]).reshape(v.shape)


def kv4_store(pages, table, page, i, pos, h, which, codes, scales):
    """Writes one token's row (which 0: K, 1: V) into uint8 pages [P, Hkv, page / 16, 18 D]."""
    D = codes.shape[-1]
    slab = pages[table[i, pos // page], h, pos % page // 16]
    t, at = pos % 16, which * 9 * D
    slab[at + t * D // 2:at + (t + 1) * D // 2] = codes[0::2] | codes[1::2] << 4
    at += 8 * D
    slab[at + t * D // 16:at + (t + 1) * D // 16] = scales


def kv4_load(pages, table, page, i, n, h, which):
    """(codes [n, D], scale codes [n, D / 16]) of the first n tokens of sequence i, KV head h."""
    D = pages.shape[-1] // 18
    ids = table[i, :-(-n // page)]
    slabs = pages[ids, h].reshape(-1, 18 * D)[:, which * 9 * D:(which + 1) * 9 * D]
    both = slabs[:, :8 * D].reshape(-1, D // 2)[:n]
    codes = np.stack([both & 15, both >> 4], -1).reshape(n, D)
    return codes, slabs[:, 8 * D:].reshape(-1, D // 16)[:n]


def head_norm(x, weight, eps, offset=0.0):
    """RMS norm over the last axis, float64."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)


def kv4_attention(q, pages, table, page, cu_q, kv_len, scale=None, k_scale=1.0, v_scale=1.0):
    """Outputs [R, Hq, D] float64 and, for tolerances, the same with |V| and each row's largest
    sum of |q k| times the scale [R, Hq] and sum of |v| over the sum of weights [R, Hq, D]."""
    R, Hq, D = q.shape
    Hkv = pages.shape[1]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if not scale else float(np.float32(scale))
    qf = to_f64(q)
    out, mag, small = np.zeros((R, Hq, D)), np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    reach = np.zeros((R, Hq))
    for i in range(len(cu_q) - 1):
        r0, n = int(cu_q[i]), int(cu_q[i + 1]) - int(cu_q[i])
        if n == 0:
            continue
        keys = int(kv_len[i]) + n
        for h in range(Hkv):
            K = kv4_values(*kv4_load(pages, table, page, i, keys, h, 0), k_scale)
            V = kv4_values(*kv4_load(pages, table, page, i, keys, h, 1), v_scale)
            for j in range(n):
                m = int(kv_len[i]) + j + 1
                for a in range(h * g, (h + 1) * g):
                    s = scale * (K[:m] @ qf[r0 + j, a])
                    e = np.exp(s - s.max())
                    out[r0 + j, a] = e @ V[:m] / e.sum()
                    mag[r0 + j, a] = e @ np.abs(V[:m]) / e.sum()
                    small[r0 + j, a] = np.abs(V[:m]).sum(0) / e.sum()
                    reach[r0 + j, a] = scale * (np.abs(K[:m]) @ np.abs(qf[r0 + j, a])).max()
    return out, mag, small, reach
