"""64-bit references of the dense-table operators (4-bit matrices, token
lookups and their gradient), in NumPy.

TEST INFRASTRUCTURE ONLY, as the rest of this package. Written from the
formulas: values are the definition's in float64; what an operator rounds on
the way (scales, codes, a result's type) is rounded here by ``round_to``.
Pinned by hand-worked examples, exact rational arithmetic and round trips
(``tests/test_oracle_tables.py``).
"""
from __future__ import annotations

import numpy as np


def round_to(v, dtype):
    """float64 or float32 values rounded (to nearest, ties to even) to
    'f32', 'f16' or 'bf16', returned as float32 values."""
    v = np.asarray(v)
    with np.errstate(over="ignore", invalid="ignore"):
        if dtype == "f32":
            return v.astype(np.float32)
        if dtype == "f16":
            return v.astype(np.float16).astype(np.float32)
        if dtype != "bf16":
            raise ValueError(dtype)
        f = np.ascontiguousarray(v, dtype=np.float32)  # callers pass values that fp32 holds
        bits = f.view(np.uint32).astype(np.uint64)
        bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
        out = bits.astype(np.uint32).view(np.float32).reshape(f.shape).copy()
        out[np.isnan(f)] = np.nan
        return out


def half_ulp(v, dtype):
    """Bound on the error of rounding values near ``v`` to dtype."""
    bits, least = {"f32": (24, 2.0 ** -150), "f16": (11, 2.0 ** -25),
                   "bf16": (8, 2.0 ** -134)}[dtype]
    return np.abs(v) * 2.0 ** -bits + least


def unpack(codes, cols):
    """[rows, cols] integers 0..15: column k in the low (even) or high (odd)
    half of byte k // 2."""
    codes = np.asarray(codes, dtype=np.uint8)
    out = np.empty((codes.shape[0], cols), np.int64)
    for k in range(cols):
        byte = codes[:, k // 2]
        out[:, k] = (byte >> 4) if k % 2 else (byte & 15)
    return out


def pack(q):
    """The inverse of unpack; the unused half of an odd row's last byte is 0."""
    q = np.asarray(q, dtype=np.uint8)
    rows, cols = q.shape
    out = np.zeros((rows, (cols + 1) // 2), np.uint8)
    out |= q[:, 0::2]
    out[:, :cols // 2] |= q[:, 1::2] << 4
    return out


def q4_values(codes, scales, zeros, group, cols):
    """A[r][k] = scale[r][k//group] * (code[r][k] - zero[r][k//group])."""
    at = np.arange(cols) // group
    z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[:, at]
    return np.asarray(scales, np.float64)[:, at] * (unpack(codes, cols) - z)


def q4_run(values, x, c=None):
    """(y, sum of magnitudes) of y_j = A x_j + c_j."""
    x = np.atleast_2d(np.asarray(x, np.float64))
    y = x @ values.T
    mag = np.abs(x) @ np.abs(values).T
    if c is not None:
        c = np.atleast_2d(np.asarray(c, np.float64))
        y, mag = y + c, mag + np.abs(c)
    return y, mag


def q4_quantize(w, group, scale_type, with_zeros):
    """(codes, scales as float32 values, zeros or None) of a float32 matrix;
    the factors 1/15 and 1/7, the quotients and their rounding are in float32, as the
    operator says."""
    w = np.asarray(w, np.float32)
    rows, cols = w.shape
    groups = -(-cols // group)
    q = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, groups), np.float32)
    zeros = np.full((rows, groups), 8, np.uint8)
    f32 = np.float32
    with np.errstate(all="ignore"):
        for r in range(rows):
            for g in range(groups):
                part = w[r, g * group:(g + 1) * group]
                low, high = min(part.min(), f32(0)), max(part.max(), f32(0))
                raw = (f32(f32(high - low) * f32(1 / 15)) if with_zeros
                       else f32(max(high, -low) * f32(1 / 7)))
                if not np.all(np.isfinite(part)):
                    raw = f32(np.nan)
                s = round_to(np.array([raw]), scale_type)[0]
                scales[r, g] = s
                usable = s > 0 and np.isfinite(s)
                z = 8
                if with_zeros:
                    z = int(np.clip(np.rint(f32(-low / s)), 0, 15)) if usable else 0
                zeros[r, g] = z
                n = len(part)
                q[r, g * group:g * group + n] = (
                    np.clip(np.rint(part / s) + z, 0, 15).astype(np.uint8) if usable else z)
    return pack(q), scales, zeros if with_zeros else None


def embed(table, tokens, scale, out_type):
    """Rows of the table times scale (the product rounded to float32, then to
    out_type); zeros for tokens outside it. Float32 values."""
    table = np.asarray(table, np.float32)
    out = np.zeros((len(tokens), table.shape[1]), np.float32)
    for t, v in enumerate(tokens):
        if 0 <= v < table.shape[0]:
            out[t] = table[v] * np.float32(scale)
    return round_to(out, out_type)


def embed_grad(g, tokens, vocab, scale, base=None):
    """(gradient, sum of magnitudes, terms per row) in float64."""
    g = np.asarray(g, np.float64)
    grad = np.zeros((vocab, g.shape[1]))
    mag = np.zeros_like(grad)
    count = np.zeros(vocab, np.int64)
    for t, v in enumerate(tokens):
        if 0 <= v < vocab:
            grad[v] += scale * g[t]
            mag[v] += abs(scale) * np.abs(g[t])
            count[v] += 1
    if base is not None:
        grad += base
        mag += np.abs(base)
    return grad, mag, count
