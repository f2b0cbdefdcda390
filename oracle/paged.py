"""A paged e4m3 KV cache in the oracle: append with rotation, and attention.

TEST INFRASTRUCTURE ONLY: only the test suite may import this module.  It
shares no code with the CUDA path.

The cache is a dict of NumPy arrays: k, v uint8 codes [n_pages, Hkv, page, hd]
and k_exp, v_exp uint8 [n_pages, Hkv]; a value is e4m3(code) 2^(exp - 127).
Sequences are lists of (first token row, new rows, cached rows, page ids).
"""
import math

import numpy as np

from . import fp8

SCALE_MIN, SCALE_MAX = -40, 100


def rotate(x, rope, positions, interleaved):
    """x [n, heads, hd] float32 rotated by rope [positions, half, 2] float32; fp32 operations."""
    y = x.astype(np.float32).copy()
    half = rope.shape[1]
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c = rope[positions, None, :, 0]
    s = rope[positions, None, :, 1]
    a, b = x[..., first].astype(np.float32), x[..., second].astype(np.float32)
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def exponent(amax):
    """The smallest integer e with amax <= 448 * 2^e, within the scale's range."""
    if amax == 0:
        return SCALE_MIN
    e = math.frexp(float(amax))[1] - 9
    while float(amax) > 448.0 * 2.0 ** e:
        e += 1
    while float(amax) <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(max(e, SCALE_MIN), SCALE_MAX)


def _codes(x):
    """e4m3 codes of float64 values; infinities saturate, NaN stays NaN."""
    c = fp8.encode(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0))
    return np.where(np.isnan(x), np.uint8(0x7F), c)


def append(cache, seqs, k, v, rope=None, interleaved=False):
    """Store the new rows k, v [T, Hkv, hd] float32 of every sequence; changes cache in place."""
    page = cache["k"].shape[2]
    for t0, n, c0, pages in seqs:
        if n == 0:
            continue
        pos = np.arange(c0, c0 + n)
        rows = {"k": k[t0:t0 + n], "v": v[t0:t0 + n].astype(np.float32)}
        if rope is not None:
            rows["k"] = rotate(rows["k"], rope, pos, interleaved)
        for name in "kv":
            for j in range(c0 // page, (c0 + n - 1) // page + 1):
                lo, hi = max(c0, j * page), min(c0 + n, (j + 1) * page)
                part = rows[name][lo - c0:hi - c0].astype(np.float64)
                for g in range(part.shape[1]):
                    x = part[:, g]
                    fine = np.abs(x[np.isfinite(x)])
                    e = exponent(fine.max() if fine.size else 0.0)
                    at = cache[name][pages[j], g]
                    kept = lo - j * page
                    if kept:
                        old = int(cache[name + "_exp"][pages[j], g]) - 127
                        if e > old:
                            at[:kept] = _codes(fp8_values(at[:kept]) * 2.0 ** (old - e))
                        e = max(e, old)
                    at[kept:kept + hi - lo] = _codes(x * 2.0 ** -e)
                    cache[name + "_exp"][pages[j], g] = e + 127


def fp8_values(codes):
    return np.where((codes & 0x7F) == 0x7F, np.nan, fp8.decode(codes))


def keys_of(cache, name, pages, g, n):
    """The first n cached values [n, hd] of kv head g, float64."""
    x = fp8_values(cache[name][pages, g]) * (
        2.0 ** (cache[name + "_exp"][pages, g].astype(np.int64) - 127))[:, None, None]
    return x.reshape(-1, x.shape[-1])[:n]


def attend(cache, seqs, q, causal, scale):
    """q [T, Hq, hd] float64 -> out [T, Hq, hd], lse [T, Hq] (rows of no sequence stay 0)."""
    T, Hq, hd = q.shape
    Hkv = cache["k"].shape[1]
    out, lse = np.zeros((T, Hq, hd)), np.zeros((T, Hq))
    for t0, n, c0, pages in seqs:
        for h in range(Hq if n else 0):
            k = keys_of(cache, "k", pages, h * Hkv // Hq, c0 + n)
            v = keys_of(cache, "v", pages, h * Hkv // Hq, c0 + n)
            s = q[t0:t0 + n, h] @ k.T * scale
            if causal:
                s[np.arange(c0 + n)[None, :] > c0 + np.arange(n)[:, None]] = -np.inf
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            out[t0:t0 + n, h] = (p / l) @ v
            lse[t0:t0 + n, h] = (m + np.log(l))[:, 0]
    return out, lse
