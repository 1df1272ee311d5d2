"""Plain float64 reference of the microscaled (MX) operators: quantisation to
e2m1 and e4m3 codes with one power-of-two scale per 32 elements, the residual's
addition with the root-mean-square norm, and the experts' products.

Formats as the OCP Microscaling Formats specification (v1.0) defines them.
Numpy only; nothing here is shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
FP4, FP8 = 0, 1
EMAX = {FP4: 2, FP8: 8}


def element_values(fmt: int) -> np.ndarray:
    """Every non-negative value of the element type; the position is the code."""
    if fmt == FP4:
        return np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    c = np.arange(127)  # 0x7f is NaN
    field, part = c >> 3, (c & 7) / 8.0
    return np.where(field > 0, (1 + part) * 2.0 ** (field - 7.0), part * 2.0 ** -6)


def scale_bytes(x: np.ndarray, fmt: int) -> np.ndarray:
    """[rows, n] -> uint8 [rows, n/32]."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    amax = np.abs(b).max(axis=2) if b.size else np.zeros(b.shape[:2])
    ok = np.isfinite(b).all(axis=2)
    _, e = np.frexp(np.where(ok & (amax > 0), amax, 1.0))
    s = np.where(amax > 0, e - 1 - EMAX[fmt] + 127, 0)
    return np.where(ok, np.clip(s, 0, 254), 255).astype(np.uint8)


def round_codes(a: np.ndarray, fmt: int) -> np.ndarray:
    """Signed element values (already divided by the scale) to codes: nearest, ties to the even code, saturating."""
    table = element_values(fmt)
    mag = np.minimum(np.abs(a), table[-1])
    hi = np.searchsorted(table, mag).clip(max=len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - mag, mag - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + np.where(np.signbit(a), len(table) + (fmt == FP8), 0)).astype(np.uint8)


def quantize(x: np.ndarray, fmt: int):
    """[rows, n] -> (codes, one per byte uint8 [rows, n], scale bytes uint8 [rows, n/32])."""
    s = scale_bytes(x, fmt)
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    bad = (s == 255)[:, :, None]
    scale = 2.0 ** (np.where(s == 255, 127, s).astype(np.float64) - 127)[:, :, None]
    codes = round_codes(np.where(bad, 0.0, b) / scale, fmt)
    return np.where(bad, 0, codes).astype(np.uint8).reshape(x.shape), s


def values(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    """The float64 values of codes (one per byte) and scale bytes."""
    table = element_values(fmt)
    if fmt == FP8:
        table = np.append(table, np.nan)
    v = np.concatenate([table, -table])[codes]
    scale = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(scale, BLOCK, axis=-1)


def pack(codes: np.ndarray, fmt: int) -> np.ndarray:
    """One code per byte -> the stored bytes."""
    return codes if fmt == FP8 else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(stored: np.ndarray, fmt: int) -> np.ndarray:
    return stored if fmt == FP8 else np.stack([stored & 15, stored >> 4], axis=-1).reshape(*stored.shape[:-1], -1)


def add_rmsnorm(x, residual, gamma, eps):
    """(s, n) in float64."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + residual
    n = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps) * gamma
    return s, n


def expert_up(xv, perm, offsets, w1v, k):
    """The product u [N, F] before its GELU, and (for error bounds) sum |x w| and the largest |x w| of every 8 summed."""
    return expert_down(xv[perm[:int(offsets[-1])] // k], offsets, w1v)


def expert_down(hv, offsets, w2v):
    N = int(offsets[-1])
    d = w2v.shape[1]
    y, total, peak = np.zeros((N, d)), np.zeros((N, d)), np.zeros((N, d))
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            y[a:b], total[a:b], peak[a:b] = product(hv[a:b], w2v[e])
    return y, total, peak


def product(x, w):
    """x w^T, the sum of |x w| and the sum over groups of 8 along K of the group's largest |x w|."""
    ax, aw = np.abs(x), np.abs(w)
    g = np.zeros((x.shape[0], w.shape[0]))
    for at in range(0, x.shape[1], 8):
        top = ax[:, None, at] * aw[None, :, at]
        for i in range(at + 1, at + 8):
            np.maximum(top, ax[:, None, i] * aw[None, :, i], out=top)
        g += top
    return x @ w.T, ax @ aw.T, g
