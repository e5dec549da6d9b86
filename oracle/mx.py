"""fp64 oracle of the microscaled (MX) formats, their product, and the RMS norm.

Definitions: OCP Microscaling Formats specification, v1.0 (E8M0 scale per 32 values, E2M1 and E4M3
elements, conversion with a power-of-two scale from the block's largest magnitude, round to
nearest even, saturating); the root-mean-square norm as y = h / sqrt(mean(h^2) + eps) * w.
Elements are kept one code to a byte here; ``pack_fp4`` gives the two-to-a-byte form.
"""
from __future__ import annotations

import numpy as np

from .reference import silu

EMAX = {4: 2, 8: 8}


def mx_elements(fmt: int) -> np.ndarray:
    """Values of codes 0 .. 7 (E2M1) or 0 .. 126 (E4M3), ascending, from sign-less exponent and
    mantissa fields: (1 + m / 2^M) * 2^(e - bias), or m / 2^M * 2^(1 - bias) for e = 0."""
    M, bias, n = (1, 1, 8) if fmt == 4 else (3, 7, 127)
    c = np.arange(n)
    e, m = c >> M, (c & ((1 << M) - 1)) / (1 << M)
    return np.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * 2.0 ** (e - bias))


def nearest_code(a: np.ndarray, fmt: int) -> np.ndarray:
    """Code of the element nearest to each a >= 0, the even code on a tie, the last one beyond it."""
    v = mx_elements(fmt)
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)  # v[hi - 1] < a <= v[hi] inside the range
    lo = hi - 1
    up, down = v[hi] - a, a - v[lo]
    pick_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo).astype(np.uint8)


def quantize_mx(x: np.ndarray, fmt: int):
    """x [T, K] (exact in fp64) -> (codes uint8 [T, K], scale bytes uint8 [T, K / 32])."""
    x = np.asarray(x, dtype=np.float64)
    T, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    b = x.reshape(T, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    safe = np.where(bad[:, :, None], 0.0, b)
    m = np.abs(safe).max(axis=2)
    # floor(log2 m): frexp gives m = f * 2^e with f in [0.5, 1)
    E = np.where(m > 0, np.frexp(m)[1] - 1 - EMAX[fmt], -127)
    E = np.maximum(E, -127)
    mag = nearest_code(np.ldexp(np.abs(safe), -E[:, :, None]), fmt)
    codes = mag | (np.signbit(safe).astype(np.uint8) << (3 if fmt == 4 else 7))
    codes = np.where(bad[:, :, None], 0, codes).astype(np.uint8).reshape(T, K)
    return codes, np.where(bad, 255, E + 127).astype(np.uint8)


def mx_value(codes: np.ndarray, bytes_: np.ndarray, fmt: int) -> np.ndarray:
    """fp64 values of codes [T, K] with scale bytes [T, K / 32] (NaN where the byte is 255)."""
    v = mx_elements(fmt)
    half = 8 if fmt == 4 else 128
    mag = np.append(v, np.nan) if fmt == 8 else v  # E4M3 code 127 is NaN
    val = mag[codes % half] * np.where(codes >= half, -1.0, 1.0)
    scale = np.where(bytes_ == 255, np.nan, np.ldexp(1.0, bytes_.astype(np.int64) - 127))
    return val * np.repeat(scale, 32, axis=1)


def pack_fp4(codes: np.ndarray) -> np.ndarray:
    """One code to a byte -> two to a byte, the even column in the low nibble."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack_fp4(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def linear_mx(x: np.ndarray, w_codes: np.ndarray, w_bytes: np.ndarray, fmt: int) -> np.ndarray:
    """X . W^T in fp64: x quantised to fmt, W of E2M1 codes [N, K]."""
    return mx_value(*quantize_mx(x, fmt), fmt) @ mx_value(w_codes, w_bytes, 4).T


def swiglu_mx(x, gate, up, fmt: int) -> np.ndarray:
    return silu(linear_mx(x, *gate, fmt)) * linear_mx(x, *up, fmt)


def rmsnorm(x, weight, eps: float, residual=None):
    """(y, h) in fp64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64), h
