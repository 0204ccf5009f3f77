"""Oracle: the 4-bit K/V cache (include/gqa_int4.h) and the rotating append (include/gqa_rope.h).

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.  Codes are integers
decided by floating point, so the writer works in IEEE fp32 as the format says; reading back and
attention are in fp64.  Places inside a tile are computed one element at a time from the header's
formulas (no permutations), so that they share nothing with the kernels' or any other packing.
"""
from __future__ import annotations

import functools

import numpy as np

from .paged_attention import attend_one_query, kv_head_of

__all__ = [
    "int4_quantize_rows",
    "int4_dequantize_rows",
    "int4_write_token",
    "int4_read_token",
    "int4_pool_from_rows",
    "int4_rows_from_pool",
    "rotate_rows_f32",
    "f32_to_bf16_bits",
    "paged_multi_query_attention_int4",
]

GROUP, TILE = 64, 16


def f32_to_bf16_bits(x) -> np.ndarray:
    """Round fp32 values to bf16 (nearest, ties to even); NaN -> 0x7fff, as the format stores it."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def _bits_f32(bits) -> np.ndarray:
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def int4_quantize_rows(x):
    """x [..., D] fp32 -> codes [..., D] uint8, (step, low) bf16 bits [..., D / 64, 2]."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # numpy's min and max keep a NaN
        low = f32_to_bf16_bits(lo)
        step = f32_to_bf16_bits((hi - lo).astype(np.float32) / np.float32(15))
        bad = ~(np.isfinite(_bits_f32(low)) & np.isfinite(_bits_f32(step)))
        low, step = np.where(bad, np.uint16(0x7FFF), low), np.where(bad, np.uint16(0x7FFF), step)
        s, m = _bits_f32(step)[..., None], _bits_f32(low)[..., None]
        q = ((g - m).astype(np.float32) / s).astype(np.float32)
        code = np.where(s > 0, np.clip(np.rint(q), 0, 15), 0)
    code = np.where(np.isnan(code), 0, code).astype(np.uint8)
    return code.reshape(x.shape), np.stack([step, low], -1)


def int4_dequantize_rows(codes, params) -> np.ndarray:
    """Cached values in fp64."""
    c = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float64)
    p = _bits_f32(params).astype(np.float64)
    return (c * p[..., :1] + p[..., 1:]).reshape(codes.shape)


@functools.lru_cache(maxsize=None)
def _places(d: int):
    """(byte, shift) of each code [K/V][tau][channel], and byte of each (step, low) [K/V][tau][group]."""
    groups = d // GROUP
    at = np.zeros((2, TILE, d, 2), dtype=np.int64)
    par = np.zeros((2, TILE, groups), dtype=np.int64)
    for tau in range(TILE):
        for ch in range(d):
            r, rest = divmod(ch, 64)
            q, rest2 = divmod(rest, 16)
            b, n = divmod(rest2, 8)
            word = tau * d // 2 + q * d // 8 + r * 8 + b * 4
            at[0, tau, ch] = word + n // 2, 4 * (n % 2)
            u, rest = divmod(ch, 64)
            g, n = divmod(rest, 8)
            per = 8 // groups
            row = tau // 8 * 8 + tau % 2 * 4 + tau % 8 // 2
            word = 8 * d + g // per * 512 + row * 32 + g % per * 4 * groups + u * 4
            at[1, tau, ch] = word + n // 2, 4 * (n % 2)
        for kv in range(2):
            for r in range(groups):
                par[kv, tau, r] = 16 * d + tau * 8 * groups + kv * 4 * groups + 4 * r
    return at, par


def int4_write_token(tile: np.ndarray, tau: int, kv: int, codes: np.ndarray, params: np.ndarray) -> None:
    """Put one token's codes [D] and (step, low) bits [groups, 2] of K (0) or V (1) into a tile [18 D]."""
    at, par = _places(codes.shape[-1])
    for ch, c in enumerate(codes):
        byte, shift = at[kv, tau, ch]
        tile[byte] = (int(tile[byte]) & ~(15 << shift) | int(c) << shift) & 0xFF
    for r in range(params.shape[0]):
        tile[par[kv, tau, r]:par[kv, tau, r] + 4] = np.ascontiguousarray(params[r]).view(np.uint8)


def int4_read_token(tile: np.ndarray, tau: int, kv: int):
    at, par = _places(tile.shape[-1] // 18)
    codes = (tile[at[kv, tau, :, 0]] >> at[kv, tau, :, 1].astype(np.uint8)) & 15
    params = np.stack([np.ascontiguousarray(tile[b:b + 4]).view(np.uint16) for b in par[kv, tau]])
    return codes, params


def int4_pool_from_rows(k, v) -> np.ndarray:
    """K, V pools [P, Hk, ps, D] in fp32 -> the 4-bit pool's bytes [P, Hk, ps / 16, 18 D]."""
    P, Hk, ps, d = k.shape
    at, par = _places(d)
    pool = np.zeros((P, Hk, ps // TILE, 18 * d), dtype=np.uint8)
    for kv, x in enumerate((k, v)):
        codes, params = int4_quantize_rows(x)
        codes = codes.reshape(P, Hk, ps // TILE, TILE, d)
        params = np.ascontiguousarray(params).view(np.uint8).reshape(P, Hk, ps // TILE, TILE, d // GROUP, 4)
        for tau in range(TILE):
            for nib in range(2):  # the two nibbles of a byte, so that no place repeats in one update
                ch = np.flatnonzero(at[kv, tau, :, 1] == 4 * nib)
                pool[..., at[kv, tau, ch, 0]] |= codes[..., tau, ch] << np.uint8(4 * nib)
            for r in range(d // GROUP):
                b = par[kv, tau, r]
                pool[..., b:b + 4] = params[..., tau, r, :]
    return pool


def int4_rows_from_pool(pool):
    """Cached values (fp64) of a 4-bit pool: K, V [P, Hk, ps, D]."""
    P, Hk, tiles, b = pool.shape
    d = b // 18
    at, par = _places(d)
    out = []
    for kv in range(2):
        codes = (pool[..., at[kv, :, :, 0]] >> at[kv, :, :, 1].astype(np.uint8)) & 15  # [P, Hk, tiles, 16, d]
        where = par[kv][..., None] + np.arange(4)
        params = np.ascontiguousarray(pool[..., where]).view(np.uint16)  # [P, Hk, tiles, 16, groups, 2]
        with np.errstate(invalid="ignore"):
            out.append(int4_dequantize_rows(codes, params).reshape(P, Hk, tiles * TILE, d))
    return tuple(out)


def rotate_rows_f32(x, cos_sin, positions, interleaved: bool) -> np.ndarray:
    """x [T, heads, D] fp32 rotated by positions [T], one IEEE fp32 operation at a time."""
    x = np.asarray(x, dtype=np.float32)
    r = cos_sin.shape[1]
    y = x.copy()
    for t, p in enumerate(positions):
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
            c, s = np.float32(cos_sin[p, i]), np.float32(cos_sin[p, r // 2 + i])
            x1, x2 = x[t, :, a], x[t, :, b]
            y[t, :, a] = x1 * c - x2 * s
            y[t, :, b] = x2 * c + x1 * s
    return y


def paged_multi_query_attention_int4(q, pool, block_table, seq_lens, scale) -> np.ndarray:
    """q [B, Q, H, D] fp64 -> [B, Q, H, D] fp64 over the pool's cached values."""
    k, v = int4_rows_from_pool(pool)
    q = np.asarray(q, dtype=np.float64)
    B, Q, H, d = q.shape
    Hk, ps = k.shape[1], k.shape[2]
    out = np.zeros_like(q)
    for b in range(B):
        L = int(seq_lens[b])
        pages = block_table[b, :(L + ps - 1) // ps]
        for h in range(H):
            kvh = kv_head_of(h, H, Hk)
            kk = k[pages, kvh].reshape(-1, d)[:L]
            vv = v[pages, kvh].reshape(-1, d)[:L]
            for i in range(Q):
                n = L - Q + 1 + i
                if n > 0:
                    out[b, i, h] = attend_one_query(q[b, i, h], kk[:n], vv[:n], scale)
    return out
