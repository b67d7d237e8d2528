"""The 4-bit microscaled formats in numpy, in 64 bits, from their definitions (include/fp8blk.h)."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def round_e2m1(v):
    """Codes (0 .. 15) of v: the nearest value, ties to the even code, beyond 6 saturating."""
    a = np.minimum(np.abs(v), 6.0)
    low = np.searchsorted(GRID, a, side="right") - 1
    high = np.minimum(low + 1, 7)
    down, up = a - GRID[low], GRID[high] - a
    code = np.where((up < down) | ((up == down) & (low % 2 == 1)), high, low)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def e4m3_values():
    code = np.arange(128)
    e, m = code >> 3, code & 7
    v = np.where(e == 0, m * 2.0**-9, (8 + m) * 2.0 ** (e - 10.0))
    return v[:127]                                   # the last code is NaN


def round_e4m3(v):
    """Codes of v >= 0: the nearest value, ties to the even code, beyond 448 saturating."""
    grid = e4m3_values()
    v = np.minimum(v, 448.0)
    low = np.searchsorted(grid, v, side="right") - 1
    high = np.minimum(low + 1, 126)
    down, up = v - grid[low], grid[high] - v
    return np.where((up < down) | ((up == down) & (low % 2 == 1)), high, low).astype(np.uint8)


def quantize(x, fmt, g=1.0):
    """x [r, c] (float64 values) -> codes [r, c] (0 .. 15), scale bytes [r, c/block]."""
    r, c = x.shape
    b = BLOCK[fmt]
    blocks = x.reshape(r, c // b, b)
    amax = np.abs(blocks).max(axis=2)
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2, -127)
        byte = (np.clip(e, -127, 127) + 127).astype(np.uint8)
        codes = round_e2m1(blocks / 2.0 ** (byte.astype(np.float64) - 127)[..., None])
    else:
        sixth = (amax / 6.0).astype(np.float32).astype(np.float64)
        byte = round_e4m3((sixth / np.float64(np.float32(g))).astype(np.float32).astype(np.float64))
        d = (e4m3_values()[byte] * np.float64(np.float32(g))).astype(np.float32).astype(np.float64)[..., None]
        q = (blocks / np.where(d > 0, d, 1.0)).astype(np.float32).astype(np.float64)
        codes = np.where(d > 0, round_e2m1(q), 0).astype(np.uint8)
    return codes.reshape(r, c), byte


def values(codes, byte, fmt):
    """Values (64 bits) of codes and scale bytes, without the tensor's scale."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = 2.0 ** (byte.astype(np.float64) - 127) if fmt == "mxfp4" else e4m3_values()[byte]
    return v * np.repeat(s, BLOCK[fmt], axis=1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)


def tile(byte):
    """Scale bytes [r, blocks] in atoms [ceil(r/128), ceil(blocks/4), 512], zeros where nothing is."""
    r, n = byte.shape
    out = np.zeros((-(-r // 128), -(-n // 4), 512), np.uint8)
    rows, blocks = np.meshgrid(np.arange(r), np.arange(n), indexing="ij")
    out[rows // 128, blocks // 4, (rows % 32) * 16 + (rows % 128 // 32) * 4 + blocks % 4] = byte
    return out


def pad_rows(x, multiple=32):
    want = -(-x.shape[0] // multiple) * multiple
    return np.concatenate([x, np.zeros((want - x.shape[0], x.shape[1]), x.dtype)])
