"""64-bit reference of the 4-bit formats (CPU, float64), written from the
definitions in include/moe.h: quantisation, the scale tiles, the values."""
import numpy as np
import torch

BLOCK = {"mx": 32, "nv": 16}
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_round(v):
    """Nearest e4m3 value (ties to even) of v >= 0, at most 448, and its byte."""
    v = np.asarray(v, dtype=np.float64)
    e = np.clip(np.floor(np.log2(np.maximum(v, 2.0 ** -9))), -6, 8)
    e = np.where(v >= 2.0 ** (e + 1), e + 1, e)          # log2 rounded down across a power
    e = np.where((v < 2.0 ** e) & (e > -6), e - 1, e)
    step = 2.0 ** (e - 3)
    r = np.minimum(np.rint(v / step) * step, 448.0)
    er = np.where(r >= 2.0 ** -6, np.floor(np.log2(np.maximum(r, 2.0 ** -6)) + 1e-12), -7)
    byte = np.where(er < -6, np.rint(r * 512), (er + 7) * 8 + np.rint((r / 2.0 ** er - 1) * 8))
    return r, byte.astype(np.uint8)


def quantize(x, fmt, scale_exp=0):
    """x [n, K] float64 (bf16 values) -> codes uint8 [n, K] (sign in bit 3),
    scale bytes [n, K/block], values float64 [n, K]."""
    x = np.asarray(x, dtype=np.float64)
    n, K = x.shape
    b = x.reshape(n, K // BLOCK[fmt], BLOCK[fmt])
    amax = np.abs(b).max(axis=2)
    if fmt == "mx":
        _, e = np.frexp(amax)
        e = np.where(amax > 0, np.maximum(e - 1 - 2, -127), -127)
        byte = (e + 127).astype(np.uint8)
        scale = 2.0 ** e.astype(np.float64)
    else:
        r, byte = e4m3_round(amax / 6.0 * 2.0 ** -scale_exp)
        scale = r * 2.0 ** scale_exp
    v = np.divide(b, scale[:, :, None], out=np.zeros_like(b), where=scale[:, :, None] > 0)
    a = np.abs(v)
    hi = np.searchsorted(GRID, a, side="left").clip(max=7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - GRID[lo], GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 6.0, 7, code)
    val = np.copysign(GRID[code], b) * scale[:, :, None]
    code = (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)
    return code.reshape(n, K), byte, val.reshape(n, K)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def row_blocks(n, offsets):
    """(128-row block, row in it) of every row; -1 where no group holds it."""
    r = np.arange(n)
    if offsets is None:
        return r // 128, r % 128
    off = np.asarray(offsets, dtype=np.int64)
    blk = np.full(n, -1)
    loc = np.zeros(n, dtype=np.int64)
    for g in range(len(off) - 1):
        rows = np.arange(off[g], off[g + 1])
        blk[rows] = off[g] // 128 + g + (rows - off[g]) // 128
        loc[rows] = (rows - off[g]) % 128
    return blk, loc


def scale_positions(n, nb, offsets=None):
    """Byte positions [n, nb] of the scales; -1 where no group holds the row."""
    blk, loc = row_blocks(n, offsets)
    b = np.arange(nb)
    pos = ((blk[:, None] * (nb // 4) + b // 4) * 512 + ((loc % 32) * 16 + loc // 32 * 4)[:, None] +
           b % 4)
    return np.where(blk[:, None] >= 0, pos, -1)


def place(byte, offsets, size, fill=0):
    n, nb = byte.shape
    out = np.full(size, fill, dtype=np.uint8)
    pos = scale_positions(n, nb, offsets)
    out[pos[pos >= 0]] = byte[pos >= 0]
    return out


def values(code, byte, fmt, scale_exp=0):
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    if fmt == "mx":
        s = 2.0 ** (byte.astype(np.float64) - 127)
    else:
        e, m = (byte >> 3) & 15, (byte & 7).astype(np.float64)
        s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
        s = s * 2.0 ** scale_exp
    return v * np.repeat(s, BLOCK[fmt], axis=1)


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
