"""Microscaled 4-bit quantisation and product in plain numpy float64.

The OCP Microscaling Formats specification v1.0 (MXFP4): blocks of 32 values,
E2M1 elements, E8M0 scales, the scale floor(log2(max)) - 2. Shares no code with
the GPU path; `pack` spells out the byte layout of include/rlk_mx4.h.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def decode_bf16(bits: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):  # signalling NaN patterns
        return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize(bits: np.ndarray):
    """(codes uint8 [n, d], scale bytes uint8 [n, d / 32]) of BF16 bit patterns, one code a byte."""
    n, d = bits.shape
    x = decode_bf16(bits).reshape(n, d // BLOCK, BLOCK)
    sign = (np.asarray(bits, dtype=np.uint16) >> 15).astype(np.uint8).reshape(x.shape)
    bad = ~np.isfinite(x).all(-1)
    mag = np.where(bad[..., None], 0.0, np.abs(x))
    top = mag.max(-1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2, -127)
    e = np.clip(e, -127, 127)
    y = np.ldexp(mag, -e[..., None])
    # nearest grid value, ties to the even code: compare with the middles
    middle = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(y.shape, np.uint8)
    for k, m in enumerate(middle):  # from code k to k + 1
        code += ((y > m) | ((y == m) & (k % 2 == 1))).astype(np.uint8)
    code |= sign << 3
    code[bad] = 0
    byte = (e + 127).astype(np.uint8)
    byte[bad] = 255
    return code.reshape(n, d), byte


def values(code: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """float64 values that codes and scale bytes stand for (NaN for byte 255)."""
    n, d = code.shape
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = np.ldexp(v.reshape(n, -1, BLOCK), (byte.astype(np.int64) - 127)[..., None])
    v = np.where((byte == 255)[..., None], np.nan, v)
    return v.reshape(n, d)


def pack(code: np.ndarray, byte: np.ndarray):
    """The packed (codes, scales) byte arrays."""
    n, d = code.shape
    rt, s4 = -(-n // 32), -(-d // 256)
    codes = np.zeros((rt, 4 * s4, 2, 32, 16), np.uint8)
    scales = np.zeros((rt, s4, 2, 32, 4), np.uint8)
    for b in range(d // BLOCK):
        s, h = b // 2, b % 2
        block = code[:, b * BLOCK:(b + 1) * BLOCK]
        two = block[:, 0::2] | (block[:, 1::2] << 4)
        for row in range(n):
            codes[row // 32, s, h, row % 32] = two[row]
            scales[row // 32, s // 4, h, row % 32, s % 4] = byte[row, b]
    return codes.reshape(-1), scales.reshape(-1)


def linear(hidden_bits, weight_code, weight_byte):
    """(exact-in-float64 logits before the BF16 rounding, sum of |products|) [n, vocab_real]."""
    h = values(*quantize(hidden_bits))
    w = values(weight_code, weight_byte)
    return h @ w.T, np.abs(h) @ np.abs(w).T
