"""GPU: the rotating appends are bit-exact against the oracle, into all three caches.

The rotation is defined one fp32 operation at a time and each result is rounded once, so q, the
bf16 rows, the e4m3 codes and the 4-bit codes, steps and minima all have to be equal bit by bit,
and no other byte of the pools may change."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
import oracle
from int4_cases import bf16, make_pool, make_table

pytestmark = pytest.mark.gpu


def table(n, r, rng):
    """Angles of any size, as far positions have them."""
    a = rng.random((n, r // 2)) * 2 * np.pi
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Case:
    def __init__(self, cache, new, H, Hk, D, r, inter, ps, seed=0, fused=False, prior=40, rows=None):
        """new: new tokens per sequence, each sequence starting at its own position."""
        rng = np.random.default_rng(seed + D + r)
        first = [int(rng.integers(0, prior)) for _ in new]
        lens = [f + n for f, n in zip(first, new)]
        self.bt, pages = make_table(rng, lens, ps)
        self.cache, self.H, self.Hk, self.D, self.inter, self.ps = cache, H, Hk, D, inter, ps
        self.ids = np.repeat(np.arange(len(new)), new).astype(np.int32)
        self.pos = np.concatenate([np.arange(f, f + n) for f, n in zip(first, new)] or [np.zeros(0)]).astype(np.int32)
        order = rng.permutation(len(self.ids))  # tokens in any order
        self.ids, self.pos = self.ids[order], self.pos[order]
        T = len(self.ids)
        self.cs = table(max(lens) + 3, r, rng)
        qkv = bf16(rng.standard_normal((T, H + 2 * Hk, D)) * 3)
        self.q, self.k, self.v = qkv.split([H, Hk, Hk], 1)
        self.fused = fused
        if cache == "int4":
            self.pools = [torch.from_numpy(make_pool(rng, pages, Hk, ps, D))]
        elif cache == "e4m3":
            self.pools = [torch.from_numpy(rng.integers(0, 256, (pages, Hk, ps, D)).astype(np.uint8)) for _ in range(2)]
        else:
            self.pools = [bf16(rng.standard_normal((pages, Hk, ps, D))) for _ in range(2)]
        self.scales = [torch.from_numpy((rng.random(Hk) * 0.02 + 0.01).astype(np.float32)) for _ in range(2)]
        self.qkv = qkv

    def call(self, dev, ids=True, q_out=None, pos=None, stream=None, seq=None):
        qkv = self.qkv.to(dev)
        q, k, v = qkv.split([self.H, self.Hk, self.Hk], 1)
        if not self.fused:
            q, k, v = (x.contiguous() for x in (q, k, v))
        self.dev_pools = [x.to(dev) for x in self.pools]
        extra = [x.to(dev) for x in self.scales] if self.cache == "e4m3" else []
        fn = {"bf16": gq.rope_kv_append, "e4m3": gq.rope_kv_append_fp8, "int4": gq.rope_kv_append_int4}[self.cache]
        seq = torch.from_numpy(self.ids if seq is None else seq).to(dev) if ids else None
        return fn(q, k, v, torch.from_numpy(self.cs).to(dev), *self.dev_pools, *extra, torch.from_numpy(self.bt).to(dev),
                  torch.from_numpy(self.pos if pos is None else pos).to(dev), seq, self.inter, q_out=q_out, stream=stream)

    def want(self, keep=None):
        """q_out bits and the pools after the rows in keep (default: all)."""
        T = len(self.ids)
        keep = range(T) if keep is None else keep
        f = lambda x: x.float().numpy()
        q, k, v = f(self.q), f(self.k), f(self.v)
        q_rot = oracle.rotate_rows_f32(q, self.cs, self.pos, self.inter)
        k_rot = oracle.rotate_rows_f32(k, self.cs, self.pos, self.inter)
        pools = [(x.view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()).copy() for x in self.pools]
        for t in keep:
            page, slot = self.bt[self.ids[t], self.pos[t] // self.ps], self.pos[t] % self.ps
            for i, row in enumerate((k_rot[t], v[t])):
                if self.cache == "bf16":
                    pools[i][page, :, slot] = oracle.f32_to_bf16_bits(row)
                elif self.cache == "e4m3":
                    quot = (row / self.scales[i].numpy()[:, None]).astype(np.float32)
                    pools[i][page, :, slot] = oracle.f64_to_e4m3_bits(quot)
                else:
                    codes, params = oracle.int4_quantize_rows(row)
                    for h in range(self.Hk):
                        oracle.int4_write_token(pools[0][page, h, slot // 16], slot % 16, i, codes[h], params[h])
        return oracle.f32_to_bf16_bits(q_rot), pools

    def check(self, q_out, keep=None):
        gq.check_device_error()
        q_bits, pools = self.want(keep)
        got = q_out.cpu().view(torch.int16).numpy().view(np.uint16)
        rows = slice(None) if keep is None else list(keep)
        assert np.array_equal(got[rows], q_bits[rows])
        for x, y in zip(self.dev_pools, pools):
            x = x.cpu()
            x = x.view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()
            assert np.array_equal(x, y)


CASES = [
    # new, H, Hk, D, r, interleaved, ps, fused
    ([1], 8, 2, 128, 128, False, 16, False),
    ([1, 1, 1, 1, 1], 12, 3, 64, 64, False, 16, True),
    ([1] * 9, 32, 8, 128, 128, False, 32, True),
    ([7, 1, 30, 16], 4, 1, 128, 64, False, 16, False),   # partial rotation
    ([7, 1, 30, 16], 6, 2, 64, 16, True, 48, True),      # the smallest rotation, odd pages
    ([40, 33], 8, 8, 64, 32, False, 64, False),
    ([3, 50], 16, 4, 128, 96, True, 256, True),          # 96 of 128 channels
    ([100, 70, 131], 7, 7, 128, 112, False, 16, False),  # MHA, 112 channels, more than one row chunk
    ([600, 700, 1], 32, 8, 64, 64, True, 16, True),      # enough rows for several per thread
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{sum(c[0])}_H{c[1]}_Hk{c[2]}_D{c[3]}_r{c[4]}{'i' if c[5] else ''}_ps{c[6]}")
def test_bit_exact(cuda_device, cache, case):
    new, H, Hk, D, r, inter, ps, fused = case
    c = Case(cache, new, H, Hk, D, r, inter, ps, fused=fused, seed=len(new))
    c.check(c.call(cuda_device))


@pytest.mark.parametrize("cache,ps", [("bf16", 5), ("e4m3", 7), ("bf16", 1)])
def test_odd_page_sizes(cuda_device, cache, ps):
    c = Case(cache, [3, 9, 1], 4, 2, 64, 64, False, ps)
    c.check(c.call(cuda_device))


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
def test_q_in_place_and_without_ids(cuda_device, cache):
    c = Case(cache, [1] * 6, 8, 2, 128, 128, False, 16)
    order = np.argsort(c.ids)
    c.ids, c.pos = c.ids[order], c.pos[order]
    q = c.q.contiguous().to(cuda_device)
    fn = {"bf16": gq.rope_kv_append, "e4m3": gq.rope_kv_append_fp8, "int4": gq.rope_kv_append_int4}[cache]
    c.dev_pools = [x.to(cuda_device) for x in c.pools]
    extra = [x.to(cuda_device) for x in c.scales] if cache == "e4m3" else []
    out = fn(q, c.k.contiguous().to(cuda_device), c.v.contiguous().to(cuda_device), torch.from_numpy(c.cs).to(cuda_device),
             *c.dev_pools, *extra, torch.from_numpy(c.bt).to(cuda_device), torch.from_numpy(c.pos).to(cuda_device), q_out=q)
    assert out is q
    c.check(out)


@pytest.mark.parametrize("cache", ["bf16", "int4"])
def test_padding_rows_are_left_alone(cuda_device, cache):
    c = Case(cache, [2, 3, 1], 8, 2, 64, 64, False, 16)
    seq = c.ids.copy()
    seq[[1, 4]] = -1
    q_out = torch.full((6, 8, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    pos = c.pos.copy()
    pos[1] = -123  # a padding row's position is not looked at
    keep = [0, 2, 3, 5]
    out = c.call(cuda_device, q_out=q_out, seq=seq, pos=pos)
    c.check(out, keep=keep)
    assert torch.all(out[[1, 4]] == 7.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
def test_out_of_range_rows_are_skipped_and_reported(cuda_device, cache):
    c = Case(cache, [2, 2, 2, 2], 4, 2, 64, 64, False, 16)
    seq, pos = c.ids.copy(), c.pos.copy()
    seq[0] = 4                       # no such sequence
    pos[1] = c.bt.shape[1] * 16      # past the table
    pos[2] = c.cs.shape[0]           # no such angle
    pos[3] = -1
    q_out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    out = c.call(cuda_device, q_out=q_out, seq=seq, pos=pos)
    with pytest.raises(gq.GQAError) as e:
        gq.check_device_error()
    assert e.value.status == -4
    c.check(out, keep=[4, 5, 6, 7])
    assert torch.all(out[:4] == 7.0)


def test_bad_page_is_skipped_and_reported(cuda_device):
    c = Case("int4", [1, 1, 1], 4, 2, 64, 64, False, 16)
    keep = [t for t in range(3) if c.ids[t] != 1]
    good = c.bt.copy()
    c.bt = c.bt.copy()
    c.bt[1] = 10 ** 6
    out = c.call(cuda_device)
    with pytest.raises(gq.GQAError):
        gq.check_device_error()
    c.bt = good
    c.check(out, keep=keep)


def test_special_values_into_the_4_bit_cache(cuda_device):
    """Constant groups, NaN, infinities, overflowing ranges, ties, tiny and huge steps: as the oracle codes them."""
    d = 128
    x = np.random.default_rng(9).standard_normal((12, 1, d)).astype(np.float32)
    x[0] = 2.5
    x[1, 0, 3] = np.inf
    x[2, 0, 70] = np.nan
    x[3, 0, :64] = np.linspace(-3e38, 3e38, 64)
    x[4] = (np.arange(d) % 31) / 2
    x[5] = np.linspace(0, 2.0 ** -120, d)
    x[6] = np.linspace(0, 2.0 ** 100, d)
    x[7] = 1000 + np.linspace(0, 4, d)
    x[8] = 0.0
    x[9, 0, 64:] = -np.inf
    x[10] = np.linspace(-2.0 ** -126, 2.0 ** -130, d)
    kb = bf16(x)
    bt = np.arange(12, dtype=np.int32)[:, None]
    pos = np.arange(12, dtype=np.int32)
    pool = torch.full((12, 1, 1, 18 * d), 0xAB, dtype=torch.uint8, device=cuda_device)
    gq.kv_append_int4(kb.to(cuda_device), kb.flip(0).contiguous().to(cuda_device), pool, torch.from_numpy(bt).to(cuda_device),
                      torch.from_numpy(pos).to(cuda_device))
    gq.check_device_error()
    want = np.full((12, 1, 1, 18 * d), 0xAB, np.uint8)
    f = kb.float().numpy()
    for t in range(12):
        for kv, row in enumerate((f[t, 0], f[11 - t, 0])):
            oracle.int4_write_token(want[t, 0, 0], t, kv, *oracle.int4_quantize_rows(row))
    assert np.array_equal(pool.cpu().numpy(), want)
    # the whole-pool writer codes the same rows the same way
    k16 = kb.view(12, 1, 1, d).expand(12, 1, 16, d).contiguous().to(cuda_device)
    got = gq.quantize_pages_int4(k16, k16).cpu().numpy()
    assert np.array_equal(got, oracle.int4_pool_from_rows(k16.float().cpu().numpy(), k16.float().cpu().numpy()))


def test_replays_in_a_graph_and_on_another_stream(cuda_device):
    c = Case("int4", [1] * 5, 8, 2, 128, 128, False, 16)
    c.check(c.call(cuda_device))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.call(cuda_device, stream=s)
    s.synchronize()
    c.check(out)


def test_no_tokens(cuda_device):
    c = Case("bf16", [1], 4, 2, 64, 64, False, 16)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=cuda_device)
    i = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    pools = [x.to(cuda_device) for x in c.pools]
    out = gq.rope_kv_append(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), torch.from_numpy(c.cs).to(cuda_device), *pools,
                            torch.from_numpy(c.bt).to(cuda_device), i, i)
    assert out.shape == (0, 4, 64)
    assert all(torch.equal(a.cpu().view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, c.pools))
