"""Plain 64-bit implementations of the MXFP4 and mixture-of-experts operators,
and the error bounds their tests use."""
from __future__ import annotations

import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([GRID, -GRID])


def encode(x):
    """Float rows [R][K] -> (codes [R][K/2], scales [R][K/32]) by the stated rule."""
    R, K = x.shape
    v = x.astype(np.float64).reshape(R, K // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(np.isfinite(v), v, 0.0)
    top = np.abs(v).max(-1)
    e = np.full(top.shape, -127, np.int64)
    nz = top > 0
    e[nz] = np.clip(np.frexp(top[nz])[1] - 1 - 2, -127, 127)
    y = np.ldexp(np.abs(v), -e[..., None])
    c = ((y > 0.25).astype(np.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    c = c + 8 * np.signbit(v).astype(np.uint8)
    c = np.where(bad[..., None], 0, c).reshape(R, K).astype(np.uint8)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def decode(q, s):
    """Codes and scales -> float64 values (NaN where the scale byte is 255)."""
    c = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    with np.errstate(invalid="ignore"):
        return VALUES[c] * np.repeat(scale, 32, axis=1)


def act(x, kind):
    if kind == "relu":
        return np.where(x > 0, x, 0.0)
    if kind == "silu":
        return x / (1.0 + np.exp(-x))
    if kind == "gelu":
        return 0.5 * x * (1.0 + np.vectorize(math.erf)(x / math.sqrt(2.0)))
    return x


def plan(ids, E):
    """Stable layout of expert ids [T][topk]: offsets, rows, slots."""
    T, topk = ids.shape
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    slots = np.empty(T * topk, np.int64)
    slots[order] = np.arange(T * topk)
    slots[key == E] = -1
    return offsets.astype(np.int32), (order // max(topk, 1)).astype(np.int32), slots.reshape(T, topk).astype(np.int32)


def check_product(C, ref, sumabs, K, out="f32", what=""):
    """C against the float64 result `ref` before no rounding at all. The
    products of the operands are exact in fp32; at most K + 16 additions each
    round by at most one unit (2^-23) of a partial sum, which never exceeds
    sumabs = sum |a w| (+ |bias| + |residual|); the activations here have slope
    at most 1.13 and the device functions add at most 8 units of the result;
    an fp16 output adds half its own unit. Taken over the whole matrix the
    roundings are independent: 4 sqrt(K) 2^-24 of the norm of sumabs."""
    C = C.astype(np.float64)
    assert C.shape == ref.shape
    assert np.isfinite(C).all(), f"{what}: {np.count_nonzero(~np.isfinite(C))} non-finite outputs"
    err = np.abs(C - ref)
    half = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 if out == "f16" else 0.0
    bound = 1.13 * (K + 16) * 2.0 ** -23 * sumabs + 8 * 2.0 ** -23 * np.abs(ref) + half + 1e-37
    assert (err <= bound).all(), f"{what}: {np.count_nonzero(err > bound)}/{err.size} beyond the bound, " \
                                 f"first at {np.argwhere(err > bound)[0].tolist()}, max {err.max():.3e}"
    if err.size:
        norm = np.linalg.norm(np.maximum(err - half, 0.0))
        most = 4 * math.sqrt(K + 16) * 2.0 ** -24 * np.linalg.norm(sumabs)
        assert norm <= most, f"{what}: error norm {norm:.3e} above {most:.3e}"
