"""Inputs and error bounds shared by the tests of the 4-bit cache (CPU side only)."""
import numpy as np
import torch

import oracle


def make_pool(rng, pages, kv_heads, page, d, spread=1.0):
    """K, V rows and the 4-bit pool that holds them."""
    k = (rng.standard_normal((pages, kv_heads, page, d)) * spread + rng.standard_normal((1, kv_heads, 1, d))).astype(np.float32)
    v = (rng.standard_normal((pages, kv_heads, page, d)) * spread).astype(np.float32)
    return oracle.int4_pool_from_rows(k, v)


def make_table(rng, lens, page, spare=2):
    """Shuffled block table (-1 past a sequence's pages) and the number of pages."""
    blocks = [-(-max(n, 0) // page) for n in lens]
    pages = sum(blocks) + spare
    order = rng.permutation(pages).astype(np.int32)
    bt = np.full((len(lens), max(1, max(blocks, default=1))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt, pages


def poison(pool, bt, lens, page):
    """Sets every byte that no token of the batch owns: codes to 15, steps and minima to NaN."""
    d = pool.shape[-1] // 18
    owned = np.zeros(pool.shape[:1] + (page,), dtype=bool)
    for b, n in enumerate(lens):
        for t in range(n):
            owned[bt[b, t // page], t % page] = True
    codes = np.full(d, 15, np.uint8)
    nan = np.full((d // 64, 2), 0x7FFF, np.uint16)
    for p, t in zip(*np.nonzero(~owned)):
        for h in range(pool.shape[1]):
            for kv in range(2):
                oracle.int4_write_token(pool[p, h, t // 16], t % 16, kv, codes, nan)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def attention_bound(q, pool, bt, lens, scale):
    """Largest error that the attention over the 4-bit pool may have, per output [B, Q, H, D].

    With c s and m a cached value's code part and minimum, w the softmax weights:
      * the output's rounding to bf16: 2^-8 |out|;
      * a score is a sum of D products of c and q, then of its group's minimum times a sum of q, in
        fp32, whose terms are at most |q| (c s + |m|): off by scale * sum |q| (c s + |m|) *
        (D + 16) * 2^-23 =: e (2^-23, not 2^-24: the tensor core may truncate); it moves a weight by
        e^(2 e) relative to the sum, 2^-20 more for the exponential and its argument's own rounding
        (|score| log2(e) * 2^-23, in e already: |score| is at most sum |q| (c s + |m|) scale);
      * p s is rounded to fp16: 2^-11; a product that is subnormal in fp16 is off by 2^-25 of the
        largest of its row at most, 2^-11 of the whole for up to 2^14 tokens;
      * sums over n tokens in fp32: (n / 16 + 64) * 2^-23.
    The weights multiply (c s + |m|): A = sum_t w_t (c_t s_t + |m_t|) bounds what they act on.
    """
    at = [oracle.int4_cache._places(pool.shape[-1] // 18)]
    k, v = oracle.int4_rows_from_pool(pool)
    parts = []
    for kv, x in enumerate((k, v)):
        par = at[0][1][kv][..., None] + np.arange(4)
        low = np.ascontiguousarray(pool[..., par]).view(np.uint16)[..., 1]
        low = (low.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        low = np.repeat(low, 64, axis=-1).reshape(x.shape)
        parts.append(np.abs(x - low) + np.abs(low))
    kabs, vabs = parts
    q = np.asarray(q, dtype=np.float64)
    B, Q, H, d = q.shape
    Hk, ps = k.shape[1], k.shape[2]
    out = np.zeros_like(q)
    for b in range(B):
        L = int(lens[b])
        pages = bt[b, :(L + ps - 1) // ps]
        for h in range(H):
            kvh = h // (H // Hk)
            kk, ka = (x[pages, kvh].reshape(-1, d)[:L] for x in (k, kabs))
            vv, va = (x[pages, kvh].reshape(-1, d)[:L] for x in (v, vabs))
            for i in range(Q):
                n = L - Q + 1 + i
                if n <= 0:
                    continue
                s = scale * (kk[:n] @ q[b, i, h])
                e = abs(scale) * (ka[:n] @ np.abs(q[b, i, h])).max() * (d + 16) * 2.0 ** -23
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, i, h] = (2.0 ** -8 * np.abs(w @ vv[:n]) +
                                (w @ va[:n]) * (2.0 ** -10 + np.expm1(2 * e) + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23))
    return out + 1e-30
