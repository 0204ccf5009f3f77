"""GPU: the rotating appends where a thread takes several rows (more than the GPU holds with one row a thread):
bit-exact against the oracle in every form that the small calls are tested in."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
import oracle
from int4_cases import bf16
from test_rope_append_gpu import Case

pytestmark = pytest.mark.gpu


def write_rows(pool, page, slot, kv, rows):
    """oracle.int4_write_token for rows [T, Hk, D] at once."""
    at, par = oracle.int4_cache._places(rows.shape[-1])
    assert np.array_equal(at[..., 0::2, 0], at[..., 1::2, 0]) and (at[..., 0::2, 1] == 0).all() and (at[..., 1::2, 1] == 4).all()
    codes, params = oracle.int4_quantize_rows(rows)
    tau = slot % 16
    where = np.s_[page[:, None, None], np.arange(rows.shape[1])[:, None], (slot // 16)[:, None, None]]
    pool[(*where, at[kv, tau, 0::2, 0][:, None])] = codes[..., 0::2] | codes[..., 1::2] << np.uint8(4)
    bytes4 = (par[kv, tau][..., None] + np.arange(4)).reshape(len(tau), 1, -1)
    pool[(*where, bytes4)] = np.ascontiguousarray(params).view(np.uint8).reshape(*rows.shape[:2], -1)


class Many(Case):
    """A Case whose expectation is made for all rows at once."""

    def __init__(self, cache, tokens, *args, **kw):
        first = tokens // 3
        super().__init__(cache, [first, 1, tokens - first - 1], *args, **kw)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert tokens * (self.H + 2 * self.Hk) > 1024 * sms // (self.D // 8), "one row a thread"

    def want(self, keep=None):
        keep = np.arange(len(self.ids)) if keep is None else np.asarray(keep)
        q, k, v = (x.float().numpy() for x in (self.q, self.k, self.v))
        q_rot = oracle.rotate_rows_f32(q, self.cs, self.pos, self.inter)
        k_rot = oracle.rotate_rows_f32(k, self.cs, self.pos, self.inter)
        pools = [(x.view(torch.int16).numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.numpy()).copy() for x in self.pools]
        page, slot = self.bt[self.ids[keep], self.pos[keep] // self.ps], self.pos[keep] % self.ps
        for i, rows in enumerate((k_rot[keep], v[keep])):
            if self.cache == "bf16":
                pools[i][page, :, slot] = oracle.f32_to_bf16_bits(rows)
            elif self.cache == "e4m3":
                pools[i][page, :, slot] = oracle.f64_to_e4m3_bits((rows / self.scales[i].numpy()[:, None]).astype(np.float32))
            else:
                write_rows(pools[0], page, slot, i, rows)
        return oracle.f32_to_bf16_bits(q_rot), pools


CASES = [
    # tokens, H, Hk, D, r, interleaved, ps, fused
    (250, 32, 8, 128, 128, False, 16, True),
    (251, 32, 8, 128, 128, True, 16, False),
    (1300, 32, 8, 128, 128, False, 16, True),   # two batches of q rows a thread
    (901, 4, 4, 128, 128, False, 16, False),    # few q heads, more k and v rows
    (701, 16, 8, 128, 128, True, 16, True),
    (3300, 1, 1, 128, 64, False, 32, False),
    (457, 7, 7, 128, 112, False, 16, False),    # 14 lanes turn, 2 do not; 7 rows are no multiple of anything
    (400, 33, 3, 128, 32, True, 16, False),     # one row past a batch
    (1201, 13, 2, 64, 64, False, 48, True),
    (640, 32, 1, 64, 32, False, 16, True),      # more rows side by side than k and v have
    (1201, 8, 8, 64, 16, True, 64, False),
    (2000, 5, 3, 64, 48, False, 16, True),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}_H{c[1]}_Hk{c[2]}_D{c[3]}_r{c[4]}{'i' if c[5] else ''}_ps{c[6]}")
def test_bit_exact(cuda_device, cache, case):
    *sizes, fused = case
    c = Many(cache, *sizes, fused=fused)
    c.check(c.call(cuda_device))


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("D,inter", [(128, False), (64, True)])
def test_q_in_place(cuda_device, cache, D, inter):
    c = Many(cache, 700, 24, 4, D, D, inter, 16)
    q = c.q.contiguous().to(cuda_device)
    c.dev_pools = [x.to(cuda_device) for x in c.pools]
    fn = {"bf16": gq.rope_kv_append, "e4m3": gq.rope_kv_append_fp8, "int4": gq.rope_kv_append_int4}[cache]
    extra = [x.to(cuda_device) for x in c.scales] if cache == "e4m3" else []
    k, v = (x.contiguous().to(cuda_device) for x in (c.k, c.v))
    cs, bt, pos, ids = (torch.from_numpy(x).to(cuda_device) for x in (c.cs, c.bt, c.pos, c.ids))
    assert fn(q, k, v, cs, *c.dev_pools, *extra, bt, pos, ids, inter, q_out=q) is q
    c.check(q)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("H,Hk,D,inter", [(32, 8, 128, False), (4, 4, 64, True)])
def test_padding_and_rows_out_of_range(cuda_device, cache, H, Hk, D, inter):
    c = Many(cache, 1700, H, Hk, D, D, inter, 16)
    rng = np.random.default_rng(5)
    odd = rng.permutation(1700)[:60].reshape(6, 10)
    seq, pos = c.ids.copy(), c.pos.copy()
    seq[odd[0]], pos[odd[0][:5]] = -1, -123      # padding, whatever its position
    q_out = torch.full((1700, H, D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    keep = np.setdiff1d(np.arange(1700), odd[0])
    out = c.call(cuda_device, q_out=q_out, seq=seq, pos=pos)
    c.check(out, keep=keep)
    assert torch.all(out[torch.from_numpy(odd[0])] == 7.0)
    seq[odd[1]] = c.bt.shape[0]                  # no such sequence
    pos[odd[2]] = c.bt.shape[1] * 16             # past the table
    pos[odd[3]] = c.cs.shape[0]                  # no such angle
    pos[odd[4]] = -1
    bad = np.sort(odd[:5].reshape(-1))
    out = c.call(cuda_device, q_out=torch.full_like(q_out, 7.0), seq=seq, pos=pos)
    with pytest.raises(gq.GQAError) as e:
        gq.check_device_error()
    assert e.value.status == -4
    c.check(out, keep=np.setdiff1d(np.arange(1700), bad))
    assert torch.all(out[torch.from_numpy(bad)] == 7.0)


@pytest.mark.parametrize("B,Hk,D", [(593, 8, 128), (700, 8, 128), (1111, 3, 128), (2400, 8, 64), (20000, 1, 64), (320, 32, 128)])
def test_append_without_rotation(cuda_device, B, Hk, D):
    """gqa_kv_append_int4: no q rows at all."""
    rng = np.random.default_rng(B)
    k, v = (bf16(rng.standard_normal((B, Hk, D)) * 3) for _ in range(2))
    pages, blocks = B // 8 + 3, 3
    bt = rng.integers(0, pages, (B, blocks)).astype(np.int32)
    # a place of its own for every sequence
    place = rng.permutation(pages * 16)[:B]
    pos = rng.integers(0, blocks, B) * 16 + place % 16
    bt[np.arange(B), pos // 16] = place // 16
    before = rng.integers(0, 256, (pages, Hk, 1, 18 * D)).astype(np.uint8)
    pool = torch.from_numpy(before).to(cuda_device)
    gq.kv_append_int4(*(x.to(cuda_device) for x in (k, v)), pool, *(torch.from_numpy(x.astype(np.int32)).to(cuda_device) for x in (bt, pos)))
    gq.check_device_error()
    want = before.copy()
    for i, x in enumerate((k, v)):
        write_rows(want, place // 16, place % 16, i, x.float().numpy())
    assert np.array_equal(pool.cpu().numpy(), want)


def test_special_rows(cuda_device):
    """Constant groups, NaN, infinities and ranges far from 1 beside ordinary rows of the same warp."""
    B, Hk, D = 800, 8, 128
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, B, Hk, D)).astype(np.float32) * 10.0 ** rng.integers(-30, 30, (2, B, Hk, 1))
    x[0, ::7, 1] = 2.5
    x[1, ::5, 3, 9] = np.nan
    x[0, ::11, 2, 70:] = -np.inf
    x[1, ::3, 0] = np.linspace(-3e38, 3e38, D)
    x[0, ::13] = 0.0
    x = bf16(x)
    pool = torch.zeros(B // 16, Hk, 1, 18 * D, dtype=torch.uint8, device=cuda_device)
    table = torch.arange(B, dtype=torch.int32, device=cuda_device)[:, None] // 16
    # position in its one page
    gq.kv_append_int4(x[0].to(cuda_device), x[1].to(cuda_device), pool, table.contiguous(),
                      torch.arange(B, dtype=torch.int32, device=cuda_device) % 16)
    gq.check_device_error()
    want = np.zeros(pool.shape, np.uint8)
    t = np.arange(B)
    for i in range(2):
        write_rows(want, t // 16, t % 16, i, x[i].float().numpy())
    assert np.array_equal(pool.cpu().numpy(), want)


def microseconds(call, n=20):
    """Device time of a call in a replayed graph (median of nine)."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    times = []
    for i in range(12):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / n)
    return sorted(times[3:])[4]


@pytest.mark.parametrize("Hk", [8, 32])
def test_one_more_sequence_is_no_cliff(cuda_device, Hk):
    """The first batch whose rows no longer fit one a thread takes about the time of the last that does (1.4 times;
    7 to 13 where each thread took all rows of a token)."""
    D = 128
    fits = 1024 * torch.cuda.get_device_properties(0).multi_processor_count // (D // 8) // (2 * Hk)
    took = []
    for B in (fits, fits + 1):
        x = torch.randn(2, B, Hk, D, device=cuda_device).bfloat16()
        pool = torch.zeros(B // 16 + 1, Hk, 1, 18 * D, dtype=torch.uint8, device=cuda_device)
        row = torch.arange(B, dtype=torch.int32, device=cuda_device)
        table, pos = (row // 16)[:, None].contiguous(), row % 16
        took.append(microseconds(lambda: gq.kv_append_int4(x[0], x[1], pool, table, pos)))
    gq.check_device_error()
    assert took[1] < 2.5 * took[0], took
