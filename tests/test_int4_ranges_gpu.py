"""GPU: attention over the 4-bit cache at the ends of what q, K and V may be, and with steps of V that differ
between the groups of a row, within a bound that a wrong output cannot meet.

The bound is int4_cases.attention_bound without its absolute term, plus what the power of two that a group's
weights carry leaves: it is at most 2^115, so a weight below fp16's normal numbers is off by 2^-25 2^-115 =
2^-140 absolutely, times a code of at most 15 and n tokens: n 2^-136 (the weights' sum is 1 or more).  An output
that is subnormal in bf16 is rounded by 2^-134.
"""
import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
import oracle
from int4_cases import attention_bound, bf16, make_table
from parity import gpu_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _defaults():
    gq.set_num_workers(0)
    yield
    gq.set_num_workers(0)


def attend(dev, q, k, v, bt, lens, scale, workers=0):
    """The attention over K, V rows [pages, Hk, ps, D] coded in 4 bits, within the bound."""
    pool = oracle.int4_pool_from_rows(k, v)
    q4 = q.float().double().numpy()
    multi = q4.ndim == 4
    if not multi:
        q4 = q4[:, None]
    want = oracle.paged_multi_query_attention_int4(q4, pool, bt, lens, scale)
    bound = attention_bound(q4, pool, bt, lens, scale) - 1e-30 + max(lens) * 2.0 ** -136 + 2.0 ** -134
    d = want.shape[-1]
    for at in range(0, d, 64):  # a bound that zeros or a wrong group could meet says nothing
        part = np.s_[..., at:at + 64]
        assert np.isfinite(bound[part]).all() and bound[part].max() < 0.1 * np.abs(want[part]).max()
    gq.set_num_workers(workers)
    fn = gq.paged_multi_query_attn_int4 if multi else gq.paged_decode_attn_int4
    out = fn(q.to(dev), *(torch.from_numpy(x).to(dev) for x in (pool, bt, np.array(lens, np.int32))), scale=scale)
    gq.check_device_error()
    got = gpu_f64(out).reshape(want.shape)
    assert np.all(np.isfinite(got))
    far = np.abs(got - want) / bound
    assert far.max() <= 1, f"{far.max():.3g} of the bound at {np.unravel_index(far.argmax(), far.shape)}"


# sizes of q, K and V, and the scale that makes ordinary scores of them (None: found below)
RANGES = [
    (1.0, 1.0, 1.0), (1e-3, 1.0, 1.0), (1e4, 1e-3, 1.0), (1e20, 1e-18, 1.0), (1e-20, 1.0, 1.0), (1.0, 1e-30, 1e-30), (1.0, 1e30, 1e28),
    (1e35, 1.0, 1.0), (1e35, 1e-20, 1.0), (5e37, 1.0, 1.0), (5e37, 1e-12, 1.0),   # q near the largest
    (1e-30, 1.0, 1.0), (1e-36, 1.0, 1.0), (1e-36, 1e-3, 1.0), (2e-38, 1.0, 1.0), (2e-38, 0.02, 1.0),  # and near the smallest normal number, with the largest scales
    (1.0, 1e-29, 1.0), (1.0, 1e-10, 1e-33), (1.0, 1.0, 1e-34),                    # |scale q| is below 2^100 in all
]


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 1, 64)], ids=str)
@pytest.mark.parametrize("size", RANGES, ids=str)
def test_sizes_of_q_k_and_v(cuda_device, size, heads):
    H, Hk, D = heads
    rng = np.random.default_rng(3 + D)
    lens, ps = [90, 300, 20], 16
    bt, pages = make_table(rng, lens, ps)
    a, b, c = size
    k = ((rng.standard_normal((pages, Hk, ps, D)) + rng.standard_normal((1, Hk, 1, D))) * b).astype(np.float32)
    v = (rng.standard_normal((pages, Hk, ps, D)) * c).astype(np.float32)
    q = bf16(rng.standard_normal((len(lens), H, D)) * a)
    scale = float(np.float32(1.0 / (a * b * D ** 0.5)))
    if not 1e-38 < scale < 3.3e38:  # as near as a scale comes
        scale = float(np.float32(min(max(scale, 1e-38), 3.3e38)))
    assert scale * float(q.abs().max()) < 2.0 ** 100
    for s, workers in ((scale, 2), (-0.7 * scale, 0)):
        attend(cuda_device, q, k, v, bt, lens, s, workers)


@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_values_of_v(cuda_device, D):
    """|v| times the number of tokens up to 2^115."""
    rng = np.random.default_rng(D)
    lens, ps = [20, 7, 1], 16
    bt, pages = make_table(rng, lens, ps)
    k = rng.standard_normal((pages, 2, ps, D)).astype(np.float32)
    v = rng.uniform(-1.0, 1.0, (pages, 2, ps, D)).astype(np.float32) * np.float32(2.0 ** 115 / 20)
    for Q in (1, 4):
        q = bf16(rng.standard_normal((3, 8, D) if Q == 1 else (3, Q, 8, D)))
        attend(cuda_device, q, k, v, bt, lens, D ** -0.5)


@pytest.mark.parametrize("rise,size", [(4.0, 1e-36), (8.0, 1e-35)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_of_zeros_behind_tiny_values(cuda_device, D, rise, size):
    """Tiny values of V, then a token whose V is zero and whose score is above all others (by less than what moves the
    reference): a zero step meets the largest power of two."""
    rng = np.random.default_rng(D)
    lens, ps = [70, 200], 16
    bt, pages = make_table(rng, lens, ps)
    k = (rng.standard_normal((pages, 1, ps, D)) * 0.01).astype(np.float32)
    v = (rng.standard_normal((pages, 1, ps, D)) * size).astype(np.float32)
    for b, t in ((0, 50), (1, 100), (1, 180)):
        k[bt[b, t // ps], 0, t % ps] = rise / D
        v[bt[b, t // ps], 0, t % ps] = 0.0
    q = bf16(np.ones((2, 4, D)))
    for workers in (0, 1):
        attend(cuda_device, q, k, v, bt, lens, 1.0, workers)


@pytest.mark.parametrize("heads", [(4, 1), (16, 1)], ids=str)
@pytest.mark.parametrize("above", [0.0, 3.0, 8.0])
@pytest.mark.parametrize("ratio", [1e-3, 1e-5, 1e-7, 1e-8, 1e-20])
def test_steps_of_the_groups_of_a_row(cuda_device, ratio, above, heads):
    """One group of V smaller than the other by `ratio`; flat scores, or one token e^above above the others."""
    rng = np.random.default_rng(int(above) + heads[0])
    lens, ps, D = [1000, 37], 16, 128
    bt, pages = make_table(rng, lens, ps)
    for small in (0, 1):
        k = (rng.standard_normal((pages, 1, ps, D)) * 0.01).astype(np.float32)
        v = (rng.standard_normal((pages, 1, ps, D)) + 0.5).astype(np.float32)
        v[..., 64 * small:64 * small + 64] *= np.float32(ratio)
        for b, t in ((0, 5 if small else 900), (1, 20)):
            k[bt[b, t // ps], 0, t % ps] = above / D
        q = bf16(np.ones((2, heads[0], D)) + 0.01 * rng.standard_normal((2, heads[0], D)))
        for workers in (0, 1):
            attend(cuda_device, q, k, v, bt, lens, 1.0, workers)


@pytest.mark.parametrize("D", [64, 128])
def test_the_largest_values_of_v_under_rising_scores(cuda_device, D):
    """The same sums where most weights are as far above the reference as they may be: e^8.3 = 2^11.97."""
    rng = np.random.default_rng(D)
    lens, ps = [32, 160], 16
    bt, pages = make_table(rng, lens, ps)
    k = (rng.standard_normal((pages, 1, ps, D)) * 0.001).astype(np.float32)
    for b, n in enumerate(lens):
        for t in range(16, n):
            k[bt[b, t // ps], 0, t % ps] = 8.3 / D
    v = rng.uniform(-1.0, 1.0, (pages, 1, ps, D)).astype(np.float32)
    v[..., ::3] = np.abs(v[..., ::3]) * 0.25 + 0.75
    q = bf16(np.ones((2, 4, D)))
    for workers in (0, 1):
        attend(cuda_device, q, k, v * np.float32(2.0 ** 115 / 160), bt, lens, 1.0, workers)
