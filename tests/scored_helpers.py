"""Plain fp64 references of the scored attention, rotary and eviction calls, and
the tolerances that follow from the arithmetic the library states.

Attention.  With weights p_i (1 + e_i), |e_i| <= E, in place of p_i, a normalised
output moves by at most 2 E sum p_i |v_i| <= 2 E max|v|.  E collects
  - the logit: fp32 accumulation of D products (each addition off by at most 2^-23
    of the sum of magnitudes, rounding or truncating), the cap (tanh to 4 units in
    the last place, times the cap) and the bias (two roundings of slope * distance);
  - ex2.approx (2 units, 2^-22) and, for 16-bit caches, the weight's split into two
    16-bit parts (bf16: 2^-17; f16: 2^-21, and 2^-25 absolute per key where a weight
    is subnormal, with the largest weight at least 1);
  - sums over n keys in fp32 (at most 2^-24 per addition, a few dozen deep).
A 16-bit output adds half a step of its type relative to its value.
"""
from __future__ import annotations

import numpy as np

from paged_helpers import widen
from paged_kv_cache_127_gb300 import synth

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def gather(cache, table, n, B, dtype):
    """[n, Hkv, D] float64 of a sequence's first n tokens."""
    if n == 0:
        return np.zeros((0, cache.shape[1], cache.shape[3]))
    blocks = np.asarray(table[: -(-n // B)])
    rows = cache[blocks].transpose(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:n]
    return widen(np.ascontiguousarray(rows), dtype)


def ranges(pos, length, rows, window=0, key_begin=None, key_end=None):
    """begin, end of each query row as include/pa.h states them."""
    pos = np.asarray(pos, np.int64)
    begin = np.zeros_like(pos) if key_begin is None else np.maximum(0, np.asarray(key_begin, np.int64)[rows])
    if window > 0:
        begin = np.maximum(begin, pos - window + 1)
    end = pos + 1 if key_end is None else np.asarray(key_end, np.int64)[rows]
    return begin, np.minimum(length, end)


def scored_rows(q, K, V, pos, begin, end, scale, cap=0.0, slopes=None):
    """q [n, Hq, D], K/V [L, Hkv, D] float64 -> (out [n, Hq, D], weights [n, Hq, L], logit error bound)."""
    n, Hq, D = q.shape
    L, Hkv = K.shape[0], K.shape[1]
    G = Hq // Hkv
    out, w = np.zeros((n, Hq, D)), np.zeros((n, Hq, L))
    worst = 0.0
    j = np.arange(L)
    for t in range(n):
        b, e = int(begin[t]), int(end[t])
        if b >= e:
            continue
        dist = np.abs(pos[t] - j[b:e])
        for h in range(Hq):
            k, v = K[b:e, h // G], V[b:e, h // G]
            z = scale * (k @ q[t, h])
            d = D * 2.0 ** -23 * abs(scale) * float((np.abs(k) @ np.abs(q[t, h])).max())
            if cap > 0:
                z = cap * np.tanh(z / cap)
                d += cap * 2.0 ** -21
            if slopes is not None:
                z = z - slopes[h] * dist
                d += 2.0 ** -22 * float(np.abs(slopes[h] * dist).max())
            d += 2.0 ** -22 * float(np.abs(z).max())  # log2 units: two roundings of the logit
            p = np.exp(z - z.max())
            p /= p.sum()
            out[t, h] = p @ v
            w[t, h, b:e] = p
            worst = max(worst, d)
    return out, w, worst


def weight_error(dtype, logit_error, n):
    """E above, for rows of at most n keys."""
    split = {"f32": 0.0, "bf16": 2.0 ** -17, "f16": 2.0 ** -21 + n * 2.0 ** -25}[dtype]
    return logit_error + 2.0 ** -22 + split + 64 * 2.0 ** -24


def assert_rows_close(got, ref, dtype, out_dtype, E, vmax):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.isfinite(got).all(), "non-finite output"
    tol = 2.5 * E * vmax + HALF_STEP[out_dtype] * np.abs(ref) + 2.0 ** -24 * (out_dtype == "f16")
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside; worst {np.abs(got - ref).max():.3e}, tol {tol.min():.3e}"


def rotate(x, pos, freqs, R, interleaved, mscale):
    """Rotated rows [T, H, D] in float64 (angles in extended precision) and the
    magnitude |a| + |b| of each pair, for the tolerance."""
    y, mag = x.copy(), np.zeros_like(x)
    angle = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freqs, np.longdouble)[None, :]
    c, s = np.cos(angle).astype(np.float64)[:, None] * mscale, np.sin(angle).astype(np.float64)[:, None] * mscale
    i = np.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(mscale)
    return y, mag


def kept_tokens(sums, length, keep, recent):
    """Old positions of the tokens one KV head keeps, in order (length > keep)."""
    recent = min(recent, keep)
    n = length - recent
    w = np.where(np.isnan(sums[:n]), -np.inf, sums[:n].astype(np.float64)) + 0.0
    nan = np.isnan(sums[:n])
    # larger sums first, NaN last of all, equal ones by rising position
    order = sorted(range(n), key=lambda j: (nan[j], -w[j] if not nan[j] else 0.0, j))
    return np.array(sorted(order[: keep - recent]) + list(range(n, length)), dtype=np.int64)


def values(rng, shape, std, dtype):
    return synth.normal(rng, shape, std, dtype)
