"""Plain models of the paged-cache operators in numpy and 64 bits: the rotation, the 4-bit
rows, the pages, and where a token lies.  Shared by the CPU and the GPU tests."""
from __future__ import annotations

import numpy as np

from long_context_attention_fwd_b200 import inputs as I


def bf16(x) -> np.ndarray:
    """fp64 values of x rounded to bf16 (nearest, ties to even; by way of fp32)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    r = np.where(np.isnan(np.asarray(x, dtype=np.float32)), np.uint16(0x7FC0), r)
    return I.bf16_bits_to_f64(r)


def bits16(x) -> np.ndarray:
    """uint16 bit patterns of fp64 values that bf16 holds exactly."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def places(cache_len, cu, T):
    """[(t, b, position)] of the packed tokens (cu None: one per sequence)."""
    cu = list(range(len(cache_len) + 1)) if cu is None else cu
    out = []
    for b in range(len(cache_len)):
        n = cu[b + 1] - cu[b]
        out += [(cu[b] + i, b, int(cache_len[b]) - n + i) for i in range(n)]
    return [x for x in out if x[0] < T]


def rotate(x, cos, sin, interleaved):
    """x [..., D] (fp64) with its first 2 * len(cos) elements rotated, and the magnitudes
    |a cos| + |b sin| that rounding errors scale with."""
    r = cos.shape[-1]
    y, mag = x.copy(), np.zeros_like(x)
    ia = 2 * np.arange(r) if interleaved else np.arange(r)
    ib = ia + 1 if interleaved else ia + r
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia] = np.abs(a * cos) + np.abs(b * sin)
    mag[..., ib] = np.abs(b * cos) + np.abs(a * sin)
    return y, mag


def quantise(x):
    """(codes [..., D] uint8, step [..., D/64], minimum [..., D/64]) of bf16 values x."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        step = bf16(np.float32(np.float32(hi - lo) / np.float32(15)))
        bad = ~np.isfinite(step)
        q = (g - lo[..., None]) / np.where(step > 0, step, 1)[..., None]
        code = np.where((step > 0)[..., None] & ~bad[..., None], np.clip(np.rint(q), 0, 15), 0)
    step, lo = np.where(bad, np.nan, step), np.where(bad, np.nan, lo + 0.0)
    return code.reshape(x.shape).astype(np.uint8), step, lo


def value(code, step, lo):
    """fp64 values step * code + lo."""
    g = code.reshape(*code.shape[:-1], code.shape[-1] // 64, 64).astype(np.float64)
    return (g * step[..., None] + lo[..., None]).reshape(code.shape)


def row_bytes(code, step, lo):
    """(code bytes [..., D/2], scale bytes [..., D/16]) of a token's row."""
    D = code.shape[-1]
    ng = D // 64
    words = np.zeros((*code.shape[:-1], D // 8), dtype=np.uint32)
    for g in range(ng):
        for i in range(8):
            for j in range(8):
                words[..., ng * i + g] |= code[..., 64 * g + 8 * i + j].astype(np.uint32) << np.uint32(4 * j)
    nan = np.uint16(0x7FC0)
    s = np.where(np.isnan(step), nan, bits16(np.nan_to_num(step)))
    m = np.where(np.isnan(lo), nan, bits16(np.nan_to_num(lo)))
    sc = s.astype(np.uint32) | (m.astype(np.uint32) << 16)
    return words.view(np.uint8), np.ascontiguousarray(sc).view(np.uint8)


def unit_parts(D):
    """Byte ranges of a unit: K codes, V codes, K scales, V scales, and a row's bytes."""
    c, s = D // 2, D // 16
    return {"kc": (0, c), "vc": (16 * c, c), "ks": (32 * c, s), "vs": (32 * c + 16 * s, s)}


def store4(pages, pg, slot, D, which, rows):
    """Writes (code, scale) bytes [Hkv, ...] of one token into pages [P, Hkv, units, 18 D]."""
    parts = unit_parts(D)
    for part, r in zip((which + "c", which + "s"), rows):
        at, n = parts[part]
        at += (slot % 16) * n
        pages[pg, :, slot // 16, at:at + n] = r


def load4(pages, table_row, ps, L, D):
    """(codes, steps, minima) of K and of V of the first L tokens of a sequence, from the bytes:
    a dict which -> (code [L, Hkv, D], step [L, Hkv, D/64], lo)."""
    pos = np.arange(L)
    pg, slot = np.asarray(table_row)[pos // ps], pos % ps
    unit = pages[pg, :, slot // 16]                                # [L, Hkv, 18 D]
    ng, parts, out = D // 64, unit_parts(D), {}
    for which in "kv":
        at, n = parts[which + "c"]
        idx = (at + (slot % 16)[:, None] * n + np.arange(n))[:, None]
        words = np.ascontiguousarray(np.take_along_axis(unit, np.broadcast_to(idx, (L, unit.shape[1], n)), 2)).view(np.uint32)
        code = np.empty((L, unit.shape[1], D), dtype=np.uint8)
        for g in range(ng):
            for i in range(8):
                for j in range(8):
                    code[..., 64 * g + 8 * i + j] = (words[..., ng * i + g] >> np.uint32(4 * j)) & 15
        at, n = parts[which + "s"]
        idx = (at + (slot % 16)[:, None] * n + np.arange(n))[:, None]
        sc = np.ascontiguousarray(np.take_along_axis(unit, np.broadcast_to(idx, (L, unit.shape[1], n)), 2)).view(np.uint16)
        sc = I.bf16_bits_to_f64(sc).reshape(L, unit.shape[1], ng, 2)
        out[which] = (code, sc[..., 0], sc[..., 1])
    return out


def table_for(rng, lens, ps, width=None, spare=3, unused=-(1 << 30)):
    """A block table [B, width] of distinct random pages for the lengths, `unused` past them,
    and the pool's size."""
    used = [-(-L // ps) for L in lens]
    width = max(1, max(used)) if width is None else width
    P = sum(used) + spare
    order = rng.permutation(P)
    t = np.full((len(lens), width), unused, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        t[b, :n] = order[at:at + n]
        at += n
    return t, P
