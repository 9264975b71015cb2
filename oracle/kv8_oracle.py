"""Plain float64 restatement of the 8-bit paged cache and of the head norm with
rotation.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages hold the history in the model's type and take queries and keys as
rotated; both operators are this library's, and their definitions are those of
its C header. The scale of a block, its reciprocal and the product with it are
float32 numbers there, so they are rounded here too: a code is decided by them
at the border between two codes.

Parity status: pinned (special cases and brute force in the tests' CPU part).
"""

from __future__ import annotations

import numpy as np

__all__ = ["kv8_round", "kv8_value", "kv8_write_block", "KV8_TOP", "norm_rotate"]

KV8_TOP = {"int8": 127.0, "e4m3": 448.0}
_LEAST = 2.0 ** -107


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def kv8_round(y, fmt: str):
    """(number of the format, its byte) nearest to each y, ties to even, saturating."""
    y = np.asarray(y, np.float64)
    if fmt == "int8":
        n = np.clip(np.rint(y), -127, 127)
        n = np.where(np.isnan(n), 0.0, n)
        return n, n.astype(np.int64).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y), 464.0)                       # above 448 all round to 448
    _, ex = np.frexp(a)
    gap = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    r = np.minimum(np.rint(a / gap) * gap, 448.0)
    frac, ex = np.frexp(r)
    ex = ex - 1                                            # r = 2 frac * 2^ex
    sub = r < 2.0 ** -6
    byte = np.where(sub, r * 512.0, (ex + 7) * 8 + (2.0 * frac - 1.0) * 8)
    byte = byte.astype(np.int64) + np.where(np.signbit(y), 128, 0)
    return np.where(np.signbit(y), -r, r), byte.astype(np.uint8)


def kv8_value(byte, fmt: str):
    """The numbers that bytes stand for."""
    b = np.asarray(byte, np.uint8)
    if fmt == "int8":
        return b.view(np.int8).astype(np.float64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    size = np.where(e > 0, np.ldexp(1.0 + m / 8.0, e.astype(np.int64) - 7), m * 2.0 ** -9)
    size = np.where((b & 127) == 127, np.nan, size)
    return np.where(b >= 128, -size, size)


def kv8_write_block(codes, scale, first: int, x, fmt: str):
    """Write the tokens x [n][d] into slots first.. of one block's half (K or V
    of one head): codes uint8 [16][d] in place; returns the new scale (float)."""
    x = np.asarray(x, np.float64)
    n = x.shape[0]
    held = float(scale) if first > 0 else 0.0
    top = np.abs(x).max()
    with np.errstate(invalid="ignore"):
        if not np.isfinite(x).all() or np.isnan(held):
            new = np.nan
        else:
            new = max(float(_f32(top / KV8_TOP[fmt])), held)
            if new < _LEAST:
                new = 0.0
        inv = float(_f32(1.0 / new)) if new > 0 else 0.0
        if first > 0 and new > held:
            ratio = float(_f32(held * inv))
            codes[:first] = kv8_round(_f32(kv8_value(codes[:first], fmt) * ratio), fmt)[1]
        codes[first:first + n] = kv8_round(_f32(x * inv), fmt)[1]
    return new


def norm_rotate(x, weight, eps, positions, inv_freq, neighbours=False):
    """x [n][heads][d]; weight [d] or None; positions [n]; inv_freq [rot / 2]."""
    x = np.asarray(x, np.float64)
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y = y.copy()
    if inv_freq is None:
        return y
    f = np.asarray(inv_freq, np.float64)
    half = f.shape[0]
    angle = np.asarray(positions, np.float64)[:, None, None] * f
    c, s = np.cos(angle), np.sin(angle)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y
