"""GPU: conversion to and from the 4-bit pool is bit-exact, and attention over it is within the bound that
int4_cases.attention_bound derives, against the oracle in fp64 over the same cached values."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
import oracle
from int4_cases import attention_bound, bf16, make_pool, make_table, poison
from parity import gpu_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _defaults():
    gq.set_num_workers(0)
    yield
    gq.set_num_workers(0)
    gq.set_wait_limit_ns(10 ** 9, False)


def check(out, q, pool, bt, lens, scale, what=""):
    q4 = q.float().double().numpy()
    if q4.ndim == 3:
        q4 = q4[:, None]
    want = oracle.paged_multi_query_attention_int4(q4, pool, bt, lens, scale)
    got = gpu_f64(out).reshape(want.shape)
    assert np.all(np.isfinite(got)), what
    bound = attention_bound(q4, pool, bt, lens, scale)
    far = np.abs(got - want) / bound
    assert far.max() <= 1, f"{what}: {far.max():.2f} of the bound at {np.unravel_index(far.argmax(), far.shape)}"
    return far.max()


def device(dev, *xs):
    return [torch.from_numpy(x).to(dev) if isinstance(x, np.ndarray) else x.to(dev) for x in xs]


def run(dev, lens, H, Hk, D, ps, Q=None, seed=0, scale=None, poisoned=True, q_spread=1.0, spread=1.0, workers=0, **kw):
    rng = np.random.default_rng(seed + sum(lens) + H + D)
    bt, pages = make_table(rng, lens, ps)
    pool = make_pool(rng, pages, Hk, ps, D, spread)
    if poisoned:
        poison(pool, bt, lens, ps)
    q = bf16(rng.standard_normal((len(lens),) + ((Q,) if Q else ()) + (H, D)) * q_spread)
    sl = np.asarray(lens, dtype=np.int32)
    fn = gq.paged_multi_query_attn_int4 if Q else gq.paged_decode_attn_int4
    dq, dpool, dbt, dsl = device(dev, q, pool, bt, sl)
    gq.set_num_workers(workers)
    out = fn(dq, dpool, dbt, dsl, scale=scale, **kw)
    gq.check_device_error()
    clean = pool.copy()
    scale = D ** -0.5 if scale is None else scale
    check(out, q, clean, bt, lens, scale, f"{lens} H{H} Hk{Hk} D{D} ps{ps} Q{Q} workers{workers}")
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.count_nonzero(out[b]) == 0
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [16, 48, 256])
def test_conversion_is_bit_exact(cuda_device, D, ps):
    rng = np.random.default_rng(D + ps)
    k, v = (bf16(rng.standard_normal((3, 2, ps, D)) * s + 1) for s in (1.0, 20.0))
    pool = gq.quantize_pages_int4(*device(cuda_device, k, v))
    want = oracle.int4_pool_from_rows(k.float().numpy(), v.float().numpy())
    assert np.array_equal(pool.cpu().numpy(), want)
    kk, vv = gq.dequantize_pages_int4(pool)
    for got, x in zip((kk, vv), oracle.int4_rows_from_pool(want)):
        # code * step + low is exact in 64 bits; the kernel's single fma rounds it to fp32, then to bf16
        bits = oracle.f32_to_bf16_bits(x.astype(np.float32))
        assert np.array_equal(got.cpu().view(torch.int16).numpy().view(np.uint16), bits)


def test_conversion_of_nothing_and_into_given_pools(cuda_device):
    z = torch.zeros(0, 2, 16, 64, dtype=torch.bfloat16, device=cuda_device)
    assert gq.quantize_pages_int4(z, z).shape == (0, 2, 1, 18 * 64)
    k = torch.randn(2, 1, 32, 64, device=cuda_device).bfloat16()
    pool = torch.empty(2, 1, 2, 18 * 64, dtype=torch.uint8, device=cuda_device)
    assert gq.quantize_pages_int4(k, k, pool) is pool
    a, b = torch.empty_like(k), torch.empty_like(k)
    assert gq.dequantize_pages_int4(pool, a, b)[0] is a
    assert torch.equal(a, b) and (a.float() - k.float()).abs().max() < 0.4


# sequences, H, Hk, D, ps
SHAPES = [
    ([17, 40], 4, 1, 64, 16),
    ([1, 15, 16, 17, 31, 33, 100], 8, 2, 128, 16),
    ([300, 1, 77], 32, 8, 128, 16),
    ([129, 64, 65], 16, 2, 128, 32),
    ([5, 0, 33, 0], 8, 8, 128, 16),                # MHA, empty sequences
    ([0, 0, 3], 8, 2, 64, 16),
    ([0], 8, 2, 64, 16),
    ([700, 47, 96], 16, 4, 128, 48),               # a page that is no power of two
    ([1300, 81], 8, 1, 64, 80),
    ([700, 90], 8, 1, 128, 256),
    ([250, 7], 12, 1, 128, 64),                    # more than 8 rows
    ([90, 200], 16, 1, 64, 128),
    ([70, 300], 96, 1, 128, 64),                   # MQA
    ([500, 17], 17, 1, 64, 16),                    # one row past a tile
    ([300, 1, 65], 50, 2, 128, 32),                # 25 rows a kv head
    ([150], 200, 1, 64, 16),
    ([200, 33], 128, 1, 128, 128),
    ([3000], 4, 1, 128, 16),                       # one sequence over many CTAs
    ([40] * 70 + [900], 4, 2, 64, 16),             # many short ones around a long one
    ([1] * 300, 2, 1, 64, 16),                     # more sequences than threads in a block
    ([3, 0] * 200, 2, 2, 128, 16),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"B{len(c[0])}_L{sum(c[0])}_H{c[1]}_Hk{c[2]}_D{c[3]}_ps{c[4]}")
def test_decode(cuda_device, case):
    lens, H, Hk, D, ps = case
    run(cuda_device, lens, H, Hk, D, ps, poisoned=len(lens) < 100)


@pytest.mark.parametrize("heads", [(16, 4, 128), (8, 1, 64), (24, 2, 128), (96, 1, 64)], ids=str)
@pytest.mark.parametrize("workers", [1, 2, 3, 37, 1000])
def test_forced_splits(cuda_device, workers, heads):
    H, Hk, D = heads
    run(cuda_device, [700, 33, 1, 2000, 129, 0, 16], H, Hk, D, 16, workers=workers, poisoned=False)


MULTI = [
    ([33, 100], 4, 1, 64, 16, 2),
    ([5, 60, 2, 0], 8, 2, 128, 16, 4),     # windows that are empty for the first tokens
    ([130, 47], 32, 8, 128, 48, 3),
    ([300], 16, 4, 128, 64, 8),
    ([64, 16, 17], 8, 8, 64, 16, 16),
    ([200, 31], 8, 2, 64, 32, 32),         # 128 rows
    ([90], 6, 2, 128, 16, 7),              # 21 rows
    ([1, 2, 3], 4, 4, 64, 16, 5),
]


@pytest.mark.parametrize("workers", [0, 3])
@pytest.mark.parametrize("case", MULTI, ids=lambda c: f"L{'_'.join(map(str, c[0]))}_H{c[1]}_Hk{c[2]}_D{c[3]}_ps{c[4]}_Q{c[5]}")
def test_multi_query(cuda_device, case, workers):
    lens, H, Hk, D, ps, Q = case
    run(cuda_device, lens, H, Hk, D, ps, Q=Q, workers=workers)


def test_multi_of_one_token_is_the_decode(cuda_device):
    a = run(cuda_device, [100, 37], 8, 2, 128, 16)
    b = run(cuda_device, [100, 37], 8, 2, 128, 16, Q=1)
    assert torch.equal(a, b[:, 0])


def test_not_a_number_past_a_window_does_not_reach_it(cuda_device):
    """The last of three tokens holds NaN in K and V: only the query that sees it is NaN."""
    rng = np.random.default_rng(1)
    bt, pages = make_table(rng, [40], 16)
    pool = make_pool(rng, pages, 1, 16, 64)
    clean = pool.copy()
    for kv in range(2):
        oracle.int4_write_token(pool[bt[0, 2], 0, 0], 39 % 16, kv, np.zeros(64, np.uint8), np.full((1, 2), 0x7FFF, np.uint16))
    q = bf16(rng.standard_normal((1, 3, 4, 64)))
    out = gq.paged_multi_query_attn_int4(*device(cuda_device, q, pool, bt, np.array([40], np.int32)))
    assert torch.isnan(out[0, 2]).all()
    check(out[:, :2], q[:, :2], clean, bt, [39], 0.125)


def test_not_a_number_in_q_stays_in_its_row(cuda_device):
    rng = np.random.default_rng(2)
    bt, pages = make_table(rng, [50], 16)
    pool = make_pool(rng, pages, 2, 16, 128)
    q = bf16(rng.standard_normal((1, 8, 128)))
    bad = q.clone()
    bad[0, 1, 5] = float("nan")
    bad[0, 6, 100] = float("inf")
    a, b = (gq.paged_decode_attn_int4(*device(cuda_device, x, pool, bt, np.array([50], np.int32))) for x in (q, bad))
    for h in range(8):
        assert torch.isnan(b[0, h]).all() if h in (1, 6) else torch.equal(a[0, h], b[0, h])


@pytest.mark.parametrize("q_spread,spread,scale", [
    (1e-3, 1.0, None), (1e4, 1e-3, None), (1.0, 300.0, 1e-4), (1e-20, 1.0, 1e18), (1e20, 1e-18, None),
    (1.0, 1e-30, None), (1.0, 1e30, 1e-31), (1.0, 1.0, 0.0), (1.0, 1.0, -0.3), (8.0, 4.0, 1.0),
])
def test_ranges(cuda_device, q_spread, spread, scale):
    run(cuda_device, [90, 300, 20], 8, 2, 128, 16, q_spread=q_spread, spread=spread, scale=scale, workers=2, seed=3)


def test_steps_of_very_different_size(cuda_device):
    """Values of a token 1e6 times another's, groups of one token too: the dominating tokens keep their precision."""
    rng = np.random.default_rng(7)
    lens = [400, 35]
    bt, pages = make_table(rng, lens, 16)
    k = rng.standard_normal((pages, 2, 16, 128)).astype(np.float32)
    v = (rng.standard_normal((pages, 2, 16, 128)) * 10.0 ** rng.uniform(-6, 3, (pages, 2, 16, 1))).astype(np.float32)
    v[..., 64:] *= 1e-5
    v[:, :, 3] = 0.0
    pool = oracle.int4_pool_from_rows(k, v)
    q = bf16(rng.standard_normal((2, 8, 128)) * 4)
    out = gq.paged_decode_attn_int4(*device(cuda_device, q, pool, bt, np.array(lens, np.int32)), scale=0.5)
    check(out, q, pool, bt, lens, 0.5)


def test_rising_scores_move_the_reference(cuda_device):
    """Scores that rise by hundreds along the sequence, and a fall after them."""
    rng = np.random.default_rng(8)
    lens = [600]
    bt, pages = make_table(rng, lens, 16)
    k = rng.standard_normal((pages, 1, 16, 64)).astype(np.float32) * 0.1
    for t in range(600):
        k[bt[0, t // 16], 0, t % 16] += 0.02 * (t if t < 500 else 1000 - 2 * t)
    v = rng.standard_normal((pages, 1, 16, 64)).astype(np.float32)
    pool = oracle.int4_pool_from_rows(k, v)
    q = bf16(np.stack([np.full(64, 1.0), np.full(64, -1.0), np.full(64, 0.01), np.zeros(64)])[None])
    for workers in (0, 1):
        gq.set_num_workers(workers)
        out = gq.paged_decode_attn_int4(*device(cuda_device, q, pool, bt, np.array(lens, np.int32)), scale=0.5)
        check(out, q, pool, bt, lens, 0.5)


def test_bad_lengths_and_pages_are_skipped_and_reported(cuda_device):
    rng = np.random.default_rng(11)
    lens = [40, 60, 20, 33]
    bt, pages = make_table(rng, lens, 16)
    pool = make_pool(rng, pages, 2, 16, 64)
    q = bf16(rng.standard_normal((4, 8, 64)))
    def fine(out, rows):  # (how a sequence is split depends on the others' lengths: equal within the bound)
        check(out[rows], q[rows], pool, bt[rows], [lens[b] for b in rows], 0.125)

    sl = np.array([40, -5, bt.shape[1] * 16 + 1, 33], np.int32)
    out = gq.paged_decode_attn_int4(*device(cuda_device, q, pool, bt, sl))
    with pytest.raises(gq.GQAError) as e:
        gq.check_device_error()
    assert e.value.status == -4
    fine(out, [0, 3])
    assert torch.count_nonzero(out[1:3]) == 0
    bt2 = bt.copy()
    bt2[1, 1], bt2[3, 0] = pages, -7
    out = gq.paged_decode_attn_int4(*device(cuda_device, q, pool, bt2, np.array(lens, np.int32)))
    with pytest.raises(gq.GQAError):
        gq.check_device_error()
    fine(out, [0, 2])
    assert torch.isfinite(out).all()
    gq.check_device_error()


def test_a_wait_that_runs_out_is_reported_and_leaves_the_workspace_usable(cuda_device):
    rng = np.random.default_rng(12)
    lens = [400, 60]
    bt, pages = make_table(rng, lens, 16)
    pool = make_pool(rng, pages, 2, 16, 64)
    q = bf16(rng.standard_normal((2, 8, 64)))
    args = device(cuda_device, q, pool, bt, np.array(lens, np.int32))
    ws = gq.int4_workspace()
    good = gq.paged_decode_attn_int4(*args, workspace=ws)
    gq.set_wait_limit_ns(100_000, True)
    out = gq.paged_decode_attn_int4(*args, workspace=ws)
    with pytest.raises(gq.GQAError) as e:
        gq.check_device_error()
    assert e.value.status == -5
    assert torch.isfinite(out).all()
    gq.set_wait_limit_ns(10 ** 9, False)
    assert torch.equal(gq.paged_decode_attn_int4(*args, workspace=ws), good)
    gq.check_device_error()


def test_one_workspace_serves_every_shape(cuda_device):
    ws = gq.int4_workspace()
    for lens, H, Hk, D in (([900, 40], 8, 2, 128), ([3000], 96, 1, 128), ([70] * 40, 8, 1, 64), ([900, 40], 8, 2, 128)):
        run(cuda_device, lens, H, Hk, D, 16, poisoned=False, workspace=ws)
    assert torch.count_nonzero(ws[:16384]) == 0


def test_two_streams_at_once(cuda_device):
    """Calls that overlap, each with a workspace of its own, or with none given."""
    rng = np.random.default_rng(13)
    lens = [2500, 1200]
    bt, pages = make_table(rng, lens, 16)
    pool = make_pool(rng, pages, 2, 16, 128)
    qs = [bf16(rng.standard_normal((2, 8, 128))) for _ in range(2)]
    dpool, dbt, dsl = device(cuda_device, pool, bt, np.array(lens, np.int32))
    want = [gq.paged_decode_attn_int4(q.to(cuda_device), dpool, dbt, dsl) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    dq = [q.to(cuda_device) for q in qs]
    spaces = [gq.int4_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for own in (True, False):
        outs = [[], []]
        for _ in range(30):
            for i, s in enumerate(streams):
                outs[i].append(gq.paged_decode_attn_int4(dq[i], dpool, dbt, dsl, workspace=spaces[i] if own else None, stream=s))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(o, want[i]) for o in outs[i])
    gq.check_device_error()


# ----------------------------------------------------------------------------- the operators together
class Serving:
    """A cache that is filled from a bf16 pool, then grows a step at a time, on the host in the oracle."""

    def __init__(self, dev, lens, H, Hk, D, ps, r, seed=21):
        rng = np.random.default_rng(seed)
        self.dev, self.H, self.Hk, self.D, self.ps = dev, H, Hk, D, ps
        self.bt, pages = make_table(rng, [n + 40 for n in lens], ps)
        self.lens = np.array(lens, np.int32)
        k, v = (bf16(rng.standard_normal((pages, Hk, ps, D))) for _ in range(2))
        self.pool = oracle.int4_pool_from_rows(k.float().numpy(), v.float().numpy())
        self.dpool = gq.quantize_pages_int4(*device(dev, k, v))
        a = np.arange(400)[:, None] * 100.0 ** -(np.arange(r // 2) / r)
        self.cs = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
        self.rng = rng

    def new(self, n):
        B = len(self.lens)
        return [bf16(self.rng.standard_normal((B * n, h, self.D))) for h in (self.H, self.Hk, self.Hk)]

    def expect(self, q, k, v, n, inter, rotate=True):
        """Appends n tokens a sequence in the oracle; the rotated q."""
        B = len(self.lens)
        pos = (self.lens[:, None] + np.arange(n)).reshape(-1)
        f = [x.float().numpy() for x in (q, k, v)]
        if rotate:
            f[:2] = [oracle.rotate_rows_f32(x, self.cs, pos, inter) for x in f[:2]]
        for t in range(B * n):
            b, p = t // n, pos[t]
            for kv in range(2):
                codes, params = oracle.int4_quantize_rows(f[1 + kv][t])
                for h in range(self.Hk):
                    oracle.int4_write_token(self.pool[self.bt[b, p // self.ps], h, p % self.ps // 16], p % 16, kv, codes[h], params[h])
        self.lens = self.lens + n
        q_bits = oracle.f32_to_bf16_bits(f[0])
        return torch.from_numpy(q_bits.view(np.int16)).view(torch.bfloat16), pos.astype(np.int32)


@pytest.mark.parametrize("inter", [False, True])
def test_fill_append_and_attend(cuda_device, inter):
    s = Serving(cuda_device, [30, 1, 77], 16, 4, 128, 16, 64)
    dbt, dcs = device(cuda_device, s.bt, s.cs)
    ws = gq.int4_workspace()
    for n in (5, 1, 1, 3):  # a prompt's rest, single steps, a draft
        q, k, v = s.new(n)
        ids = np.repeat(np.arange(3), n).astype(np.int32)
        q_rot, pos = s.expect(q, k, v, n, inter)
        args = device(cuda_device, q, k, v)
        out_q = gq.rope_kv_append_int4(*args, dcs, s.dpool, dbt, *device(cuda_device, pos, ids), interleaved=inter)
        assert torch.equal(out_q.cpu(), q_rot)
        assert np.array_equal(s.dpool.cpu().numpy(), s.pool)
        dsl = torch.from_numpy(s.lens).to(cuda_device)
        out = gq.paged_multi_query_attn_int4(out_q.view(3, n, 16, 128), s.dpool, dbt, dsl, workspace=ws)
        gq.check_device_error()
        check(out, q_rot.view(3, n, 16, 128), s.pool, s.bt, s.lens, 128 ** -0.5)


@pytest.mark.parametrize("rotate", [True, False])
def test_decode_step_and_its_graph(cuda_device, rotate):
    """The step is its two halves; captured once, it replays with new contents of its buffers; two graphs
    captured with a workspace each may be replayed at once."""
    s = Serving(cuda_device, [30, 200, 16], 8, 2, 64, 32, 64)
    B = 3
    dbt, dcs = device(cuda_device, s.bt, s.cs)
    bufs = [torch.zeros(B, h, 64, dtype=torch.bfloat16, device=cuda_device) for h in (8, 2, 2)]
    pos, sl = (torch.zeros(B, dtype=torch.int32, device=cuda_device) for _ in range(2))
    out, q_rot = torch.empty_like(bufs[0]), torch.empty_like(bufs[0]) if rotate else None
    ws = gq.int4_workspace()

    def call():
        gq.decode_step_int4(*bufs, s.dpool, dbt, pos, sl, cos_sin=dcs if rotate else None, q_rot=q_rot, out=out, workspace=ws)

    def fill():
        q, k, v = s.new(1)
        q_want, p = s.expect(q, k, v, 1, False, rotate)
        for b, x in zip(bufs, (q, k, v)):
            b.copy_(x)
        pos.copy_(torch.from_numpy(p))
        sl.copy_(torch.from_numpy(s.lens))
        return q_want

    def verify(q_want):
        gq.check_device_error()
        assert np.array_equal(s.dpool.cpu().numpy(), s.pool)
        check(out, q_want, s.pool, s.bt, s.lens, 0.125)

    q_want = fill()
    call()
    verify(q_want)
    graph = torch.cuda.CUDAGraph()
    q_want = fill()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        verify(q_want)
        q_want = fill()


def test_two_graphs_replayed_at_once(cuda_device):
    """Graphs captured without a workspace each hold one of their own."""
    rng = np.random.default_rng(31)
    lens = [1500, 700]
    bt, pages = make_table(rng, lens, 16)
    dpool, dbt, dsl = device(cuda_device, make_pool(rng, pages, 2, 16, 128), bt, np.array(lens, np.int32))
    qs = [bf16(rng.standard_normal((2, 8, 128))).to(cuda_device) for _ in range(2)]
    want = [gq.paged_decode_attn_int4(q, dpool, dbt, dsl) for q in qs]
    graphs, outs = [], []
    for q in qs:
        g, o = torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.graph(g):
            for _ in range(10):
                gq.paged_decode_attn_int4(q, dpool, dbt, dsl, out=o)
        graphs.append(g)
        outs.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    gq.check_device_error()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_given_outputs_go_the_native_way_and_give_the_same(cuda_device):
    """Calls whose outputs are given are marshalled natively: the same results, the same refusals."""
    assert gq._fast is not None
    rng = np.random.default_rng(41)
    lens = [60, 33]
    bt, pages = make_table(rng, lens, 16)
    k, v = (bf16(rng.standard_normal((pages, 2, 16, 64))).to(cuda_device) for _ in range(2))
    dbt, dsl = device(cuda_device, bt, np.array(lens, np.int32))
    pool = gq.quantize_pages_int4(k, v)
    given = torch.empty_like(pool)
    assert gq.quantize_pages_int4(k, v, given) is given and torch.equal(given, pool)
    a, b = torch.empty_like(k), torch.empty_like(k)
    gq.dequantize_pages_int4(pool, a, b)
    assert all(torch.equal(x, y) for x, y in zip((a, b), gq.dequantize_pages_int4(pool)))
    ws = gq.int4_workspace()
    for shape, fn in (((2, 8, 64), gq.paged_decode_attn_int4), ((2, 3, 8, 64), gq.paged_multi_query_attn_int4)):
        q = bf16(rng.standard_normal(shape)).to(cuda_device)
        out = torch.empty_like(q)
        for scale in (None, 0.3):
            assert fn(q, pool, dbt, dsl, out, scale, ws) is out
            assert torch.equal(out, fn(q, pool, dbt, dsl, scale=scale))
        for bad in (dict(out=out.float()), dict(out=out[..., :32]), dict(workspace=ws[:100].clone()), dict(scale=float("nan")),
                    dict(workspace=ws.float()), dict(out=out.cpu()), dict(scale="x")):
            with pytest.raises((ValueError, TypeError, gq.GQAError)):
                fn(q, pool, dbt, dsl, **{**dict(out=out, scale=0.3, workspace=ws), **bad})
        for bad in (dict(kv_pages=pool[..., :-1]), dict(block_table=dbt[:1]), dict(seq_lens=dsl.long()), dict(q=q[0])):
            with pytest.raises((ValueError, TypeError, gq.GQAError)):
                fn(**{**dict(q=q, kv_pages=pool, block_table=dbt, seq_lens=dsl, out=out, workspace=ws), **bad})
    with pytest.raises(ValueError):
        gq.quantize_pages_int4(k, v, given[:1])
    with pytest.raises((ValueError, TypeError)):
        gq.dequantize_pages_int4(pool, a, b.float())
    x = torch.zeros(2, 12, 64, dtype=torch.bfloat16, device=cuda_device)
    qkv = dict(q=x[:, :8], k_new=x[:, 8:10], v_new=x[:, 10:], cos_sin=torch.ones(100, 64, device=cuda_device),
               kv_pages=pool, block_table=dbt, positions=dsl - 1, q_out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device=cuda_device))
    assert gq.rope_kv_append_int4(**qkv) is qkv["q_out"]
    for bad in (dict(q=x[:, :8, ::2]), dict(k_new=x[:, 8:11]), dict(q_out=x[:, :8]), dict(positions=dsl.long()), dict(cos_sin=torch.ones(100, 80, device=cuda_device)),
                dict(seq_ids=dsl[:1]), dict(block_table=dbt[:1]), dict(q=x.transpose(0, 1))):
        with pytest.raises((ValueError, TypeError, gq.GQAError)):
            gq.rope_kv_append_int4(**{**qkv, **bad})
    torch.cuda.synchronize()
    gq.check_device_error()


def test_the_longest_sequence(cuda_device):
    """2^31 - 256 tokens, all in one page: equal weights on each copy of it, so the output is that of one.

    The sums take the same tokens again and again, rounded at each step.  A warp has n tokens: the work of
    8 query rows is cut evenly over 16 warps per SM.  Its weights' sums go to eight lanes
    a row (n / 8 steps of 2^-24 relative), its outputs' step by step over 16 tokens (n / 16 of 2^-23): n
    2^-26 of the largest output, which is of one sign here, for the weights' sum, the minima's and the
    outputs', and what the attention over one page may be off beside that.
    """
    rng = np.random.default_rng(51)
    ps, d, h = 256, 64, 8
    blocks = (2 ** 31 - 1) // ps
    k = (rng.standard_normal((1, 1, ps, d))).astype(np.float32)
    v = (2 + 0.25 * rng.standard_normal((1, 1, ps, d))).astype(np.float32)
    pool = oracle.int4_pool_from_rows(k, v)
    q = bf16(rng.standard_normal((1, h, d)))
    one = np.zeros((1, 1), np.int32)
    q4 = q.float().double().numpy()[:, None]
    want = oracle.paged_multi_query_attention_int4(q4, pool, one, [ps], d ** -0.5)
    bound = attention_bound(q4, pool, one, [ps], d ** -0.5)
    lens = torch.tensor([blocks * ps], dtype=torch.int32, device=cuda_device)
    table = torch.zeros((1, blocks), dtype=torch.int32, device=cuda_device)
    out = gq.paged_decode_attn_int4(q.to(cuda_device), torch.from_numpy(pool).to(cuda_device), table, lens)
    gq.check_device_error()
    n = blocks * ps / 16 / torch.cuda.get_device_properties(cuda_device).multi_processor_count
    assert np.all(np.abs(gpu_f64(out).reshape(want.shape) - want) <= bound + 3 * n * 2.0 ** -26 * np.abs(want).max())


def test_tensors_without_plain_memory_are_refused(cuda_device):
    """Nested and sparse tensors throw when they are asked for sizes or strides: an exception, no more."""
    pool = torch.zeros(2, 1, 1, 18 * 64, dtype=torch.uint8, device=cuda_device)
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=cuda_device)
    table = torch.zeros(2, 1, dtype=torch.int32, device=cuda_device)
    lens = torch.ones(2, dtype=torch.int32, device=cuda_device)
    ws = gq.int4_workspace()
    for odd in (torch.nested.nested_tensor([x[0], x[1, :3]]), x.to_sparse()):
        for kw in (dict(q=odd), dict(out=odd)):
            with pytest.raises(Exception):
                gq.paged_decode_attn_int4(**{**dict(q=x, kv_pages=pool, block_table=table, seq_lens=lens,
                                                    out=torch.empty_like(x), workspace=ws), **kw})
        with pytest.raises(Exception):
            gq.rope_kv_append_int4(odd, x[:, :1], x[:, :1], torch.ones(4, 64, device=cuda_device), pool, table, lens,
                                   q_out=torch.empty_like(x))
        pages = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=cuda_device)
        with pytest.raises(Exception):
            gq.quantize_pages_int4(pages.to_sparse(), pages, pool)
    torch.cuda.synchronize()
    gq.check_device_error()


@pytest.mark.parametrize("rotate", [True, False])
def test_a_step_with_given_outputs_goes_the_native_way_and_gives_the_same(cuda_device, rotate):
    rng = np.random.default_rng(61)
    lens = [60, 33]
    bt, pages = make_table(rng, lens, 16)
    pools = [torch.from_numpy(make_pool(rng, pages, 2, 16, 64)).to(cuda_device)]
    pools.append(pools[0].clone())
    dbt, dsl = device(cuda_device, bt, np.array(lens, np.int32))
    q, k, v = (bf16(rng.standard_normal((2, h, 64))).to(cuda_device) for h in (8, 2, 2))
    cs = torch.from_numpy(rng.standard_normal((100, 32)).astype(np.float32)).to(cuda_device) if rotate else None
    ws = gq.int4_workspace()
    args = dict(q=q, k_new=k, v_new=v, block_table=dbt, positions=dsl - 1, seq_lens=dsl, cos_sin=cs, interleaved=rotate)
    want = gq.decode_step_int4(kv_pages=pools[0], **args)
    given = dict(out=torch.empty_like(q), q_rot=torch.empty_like(q) if rotate else None, workspace=ws)
    called = []
    native = gq._fast.step

    class Counted:
        def __getattr__(self, name):
            return getattr(fast, name)

        def step(self, *a):
            called.append(native(*a))
            return called[-1]

    fast, gq._fast = gq._fast, Counted()
    try:
        assert gq.decode_step_int4(kv_pages=pools[1], **args, **given) is given["out"]
        assert called == [0]
        for bad in (dict(q=q[0]), dict(k_new=k[:, :1]), dict(v_new=v.float()), dict(positions=dsl.long()), dict(seq_lens=dsl[:1]),
                    dict(block_table=dbt[:1]), dict(out=q[:, :4]), dict(workspace=ws[:100].clone()), dict(scale=float("inf")),
                    dict(q_rot=q[:1]), dict(cos_sin=torch.ones(3, 24, device=cuda_device), q_rot=given["out"])):
            with pytest.raises((ValueError, TypeError, gq.GQAError)):
                gq.decode_step_int4(**{**args, "kv_pages": pools[1], **given, **bad})
    finally:
        gq._fast = fast
    assert torch.equal(given["out"], want) and torch.equal(*pools)
    gq.check_device_error()
