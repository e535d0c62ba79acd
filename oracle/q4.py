"""The rotating append and the 4-bit cache by definition (numpy).

A pool is uint8 [NB, Hkv, bs, RB]; 16-bit numbers travel as float64 values or
as uint16 bit patterns.  `wide` is float64 for the definitions, float32 where
the library's own roundings (every product and sum by itself) are wanted.
Shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

GROUP = 64


def row_bytes(D: int) -> int:
    return D // 2 + D // GROUP * 4


# ---------------------------------------------------------------- 16-bit types
def widen(bits, dtype: str):
    bits = np.asarray(bits, np.uint16)
    if dtype == "f16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def narrow(x, dtype: str):
    """Bit patterns of x rounded once to the type (to nearest, ties to even)."""
    x = np.asarray(x)
    if dtype == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint16)
    x64 = x.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        y = x64.astype(np.float32)
        lost = x64 - y.astype(np.float64)  # y's own rounding, so that a tie is a tie of x
    b = y.view(np.uint32).astype(np.int64)
    low, up = b & 0xffff, b >> 16
    away = np.where(np.signbit(y), -lost, lost)  # > 0: x is farther from zero than y
    tie = low == 0x8000
    up = up + ((low > 0x8000) | (tie & ((away > 0) | ((away == 0) & (up % 2 == 1)))))
    up = np.where(np.isnan(x64), 0x7fc0, up)
    return up.astype(np.uint16)


# ---------------------------------------------------------------- rotation
def rotate(x, cos, sin, interleaved: bool):
    """Rows x [..., D] of one token by cos and sin [R / 2], in x's own type."""
    y = np.array(x)
    R = 2 * len(cos)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[..., a] = x[..., a] * cos[i] - x[..., b] * sin[i]
        y[..., b] = x[..., b] * cos[i] + x[..., a] * sin[i]
    return y


# ---------------------------------------------------------------- codes
def quantise(x, dtype: str, wide=np.float64):
    """(step bits, centre bits [..., D / 64], codes [..., D]) of rows [..., D]."""
    g = np.asarray(x, wide).reshape(x.shape[:-1] + (-1, GROUP))
    hi, lo = g.max(-1), g.min(-1)
    if wide is np.float32:
        part = np.float32(1) / np.float32(15)
        step, centre = narrow((hi - lo) * part, dtype), narrow((np.float32(8) * hi + np.float32(7) * lo) * part, dtype)
    else:
        step, centre = narrow((hi - lo) / 15, dtype), narrow((8 * hi + 7 * lo) / 15, dtype)
    s, a = widen(step, dtype).astype(wide)[..., None], widen(centre, dtype).astype(wide)[..., None]
    t = (g - a) / np.where(s > 0, s, 1)
    code = np.where(s > 0, np.clip(np.rint(t), -8, 7), 0).astype(np.int64) + 8
    return step, centre, code.reshape(x.shape)


def _byte(D: int, off: int, d: int) -> int:
    """Byte of element d of the token at offset `off` of a block, within the (block, head)'s run."""
    unit, r, chunk = off // 8, off % 8, d // 32
    place = chunk ^ ((r // 2) % 4 if D == 128 else (r // 4) % 2)
    return unit * 8 * row_bytes(D) + r * (D // 2) + place * 16 + d % 32 // 2


def _pair(D: int, off: int, g: int) -> int:
    return off // 8 * 8 * row_bytes(D) + 4 * D + off % 8 * (D // 16) + 4 * g


def pack(step, centre, code):
    """The pool uint8 [NB, Hkv, bs, RB] of steps and centres (bits [NB, bs, Hkv, D / 64]) and codes [NB, bs, Hkv, D]."""
    NB, bs, Hkv, D = code.shape
    RB = row_bytes(D)
    run = np.zeros((NB, Hkv, bs * RB), np.uint8)
    for off in range(bs):
        for d in range(0, D, 2):
            run[:, :, _byte(D, off, d)] = code[:, off, :, d] | code[:, off, :, d + 1] << 4
        for g in range(D // GROUP):
            at = _pair(D, off, g)
            pair = np.stack([step[:, off, :, g], centre[:, off, :, g]], -1).astype("<u2")
            run[:, :, at:at + 4] = np.ascontiguousarray(pair).view(np.uint8)
    return run.reshape(NB, Hkv, bs, RB)


def parts(pool, D: int):
    """(step, centre bits [NB, bs, Hkv, D / 64], codes [NB, bs, Hkv, D]) of a whole pool."""
    NB, Hkv, bs, RB = pool.shape
    run = pool.reshape(NB, Hkv, bs * RB)
    code = np.zeros((NB, bs, Hkv, D), np.int64)
    pair = np.zeros((NB, bs, Hkv, D // GROUP, 2), np.uint16)
    for off in range(bs):
        for d in range(D):
            code[:, off, :, d] = run[:, :, _byte(D, off, d)] >> (4 * (d % 2)) & 15
        for g in range(D // GROUP):
            at = _pair(D, off, g)
            pair[:, off, :, g] = np.ascontiguousarray(run[:, :, at:at + 4]).view("<u2")
    return pair[..., 0], pair[..., 1], code


def values(pool, D: int, dtype: str):
    """What a pool stands for: float64 [NB, bs, Hkv, D]."""
    step, centre, code = parts(pool, D)
    s, a = widen(step, dtype), widen(centre, dtype)
    with np.errstate(invalid="ignore", over="ignore"):
        v = a[..., None] + s[..., None] * (code.reshape(code.shape[:-1] + (-1, GROUP)) - 8)
    return v.reshape(code.shape)


def slots(tables, seq, pos, bs: int):
    """Slot of every token: -1 for padding (pos < 0)."""
    return np.array([-1 if p < 0 else int(tables[s][p // bs]) * bs + p % bs for s, p in zip(seq, pos)], np.int64)
