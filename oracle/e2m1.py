"""Oracle of the 4-bit KV cache format: E2M1 codes with one E4M3 scale per 16 values (numpy).

From the format's definition alone: y = float(x) * float(1/gs), s = E4M3(float(max|y| / 6)),
code = E2M1(float(y / s)), each rounding to nearest even with saturation, by distance in double.
"""
from __future__ import annotations

import numpy as np

from . import e4m3_to_double, inv_scale

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_E4M3 = e4m3_to_double(np.arange(127, dtype=np.uint8))          # non-negative finite values, by code


def _nearest(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest grid value to each x >= 0; half way goes to the even index, past the end to the last."""
    hi = np.clip(np.searchsorted(grid, x), 1, grid.size - 1)
    lo = hi - 1
    d_lo, d_hi = x - grid[lo], grid[hi] - x
    take_hi = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def to_float(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def quantize(bits: np.ndarray, gs: float):
    """(codes [..., D] 0..15, scale codes [..., D/16]) of bf16 rows; a zero's code is 0."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        y = to_float(bits) * inv_scale(gs)
        y = y.reshape(*y.shape[:-1], -1, 16)
        amax = np.abs(y).max(-1)                               # keeps a NaN
        t = (amax / np.float32(6)).astype(np.float32).astype(np.float64)
        s_code = np.where(np.isnan(t), 127, _nearest(np.where(np.isnan(t), 0, t), _E4M3)).astype(np.uint8)
        s = np.where(s_code == 127, np.nan, _E4M3[np.minimum(s_code, 126)])[..., None]
        live = s > 0
        t = (y / np.where(live, s, 1).astype(np.float32)).astype(np.float32).astype(np.float64)
        t = np.where(live, t, 0.0)
        code = _nearest(np.abs(t), MAGNITUDES) + np.where(t < 0, 8, 0)
    return code.reshape(*bits.shape).astype(np.uint8), s_code


def pack(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Pages [..., Bs * 9 D / 16] of rows codes [..., Bs, D], scales [..., Bs, D/16]."""
    rows = codes[..., 0::2] | (codes[..., 1::2] << 4)
    flat = lambda a: a.reshape(*a.shape[:-2], -1)
    return np.concatenate([flat(rows), flat(np.swapaxes(scales, -1, -2))], -1)


def unpack(pages: np.ndarray, block_size: int, head_dim: int):
    """(codes [..., Bs, D], scales [..., Bs, D/16]) of pages."""
    n = block_size * head_dim // 2
    raw = pages[..., :n].reshape(*pages.shape[:-1], block_size, head_dim // 2)
    codes = np.empty((*raw.shape[:-1], head_dim), dtype=np.uint8)
    codes[..., 0::2], codes[..., 1::2] = raw & 15, raw >> 4
    scales = np.swapaxes(pages[..., n:].reshape(*pages.shape[:-1], head_dim // 16, block_size), -1, -2)
    return codes, np.ascontiguousarray(scales)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """code * scale in double (times the cache's own scale: the value read back)."""
    mag = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return mag * np.repeat(e4m3_to_double(scales), 16, axis=-1)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """Bits of doubles that are bf16 values (as code * scale is)."""
    f = x.astype(np.float32)
    bits = f.view(np.uint32)
    assert np.all((bits & 0xFFFF) == 0) and np.all(f.astype(np.float64) == x)
    return (bits >> 16).astype(np.uint16)


def pool_bits(pages: np.ndarray, block_size: int, head_dim: int) -> np.ndarray:
    """A 4-bit pool [N, Hkv, page] as a bf16 pool [N, Hkv, Bs, D] of code * scale."""
    return bf16_bits(values(*unpack(pages, block_size, head_dim)))


def append(pages: np.ndarray, rows_bits: np.ndarray, gs: float, slots, block_size: int) -> np.ndarray:
    """A copy of the pool with each token's rows [T, Hkv, D] quantized into its slot."""
    D = rows_bits.shape[-1]
    codes, scales = unpack(pages.copy(), block_size, D)
    codes, scales = codes.copy(), scales.copy()
    c, s = quantize(rows_bits, gs)
    for t, slot in enumerate(np.asarray(slots)):
        if 0 <= slot < pages.shape[0] * block_size:
            codes[slot // block_size, :, slot % block_size] = c[t]
            scales[slot // block_size, :, slot % block_size] = s[t]
    return pack(codes, scales)


def rope_rows(bits: np.ndarray, positions, theta: float) -> np.ndarray:
    """K rows turned in double, rounded to float, then to nearest-even bf16 (bits)."""
    x = to_float(bits).astype(np.float64)
    half = x.shape[-1] // 2
    a = (np.asarray(positions, dtype=np.float64)[:, None] *
         np.float64(np.float32(theta)) ** (-2.0 * np.arange(half) / (2 * half)))[:, None, :]
    x1, x2 = x[..., :half], x[..., half:]
    y = np.concatenate([x1 * np.cos(a) - x2 * np.sin(a), x1 * np.sin(a) + x2 * np.cos(a)], -1).astype(np.float32)
    u = y.view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
