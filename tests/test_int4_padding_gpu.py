"""GPU: sequences without a token change nothing of how a batch's others are cut over the GPU: the same bits come
out, whatever slots a captured graph leaves empty."""
import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
from int4_cases import bf16, make_pool, make_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,Hk,D", [([30000], 4, 1, 128), ([9000, 20000, 500], 16, 1, 64), ([5000, 4000], 8, 2, 128)], ids=str)
@pytest.mark.parametrize("slots", [16, 700])
def test_empty_slots_of_a_batch(cuda_device, lens, H, Hk, D, slots):
    rng = np.random.default_rng(len(lens) + D)
    bt, pages = make_table(rng, lens, 256)
    pool = torch.from_numpy(make_pool(rng, pages, Hk, 256, D)).to(cuda_device)
    # a table as wide as a serving loop's: the grid does not depend on the batch
    wide = np.full((slots, 512), -1, np.int32)
    q = torch.zeros(slots, H, D, dtype=torch.bfloat16)
    full = np.zeros(slots, np.int32)
    at = np.sort(rng.choice(slots, len(lens), replace=False))
    wide[at, :bt.shape[1]] = bt
    q[at] = bf16(rng.standard_normal((len(lens), H, D)))
    full[at] = lens
    dq, dt, dl = q.to(cuda_device), torch.from_numpy(wide).to(cuda_device), torch.from_numpy(full).to(cuda_device)
    rows = torch.from_numpy(at).to(cuda_device)
    alone = gq.paged_decode_attn_int4(dq[rows], pool, dt[rows], dl[rows])
    padded = gq.paged_decode_attn_int4(dq, pool, dt, dl)
    gq.check_device_error()
    assert torch.equal(padded[rows], alone)
    padded[rows] = 0
    assert torch.count_nonzero(padded) == 0
