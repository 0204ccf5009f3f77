"""CPU: the 4-bit cache's oracle -- places, rounding, special values -- and the host checks of its
entry points and of the rotating appends."""
import ctypes

import numpy as np
import pytest
import torch

import gqa_decode_attention_04_b200 as gq
import oracle
from int4_cases import make_pool, make_table


@pytest.mark.parametrize("d", [64, 128])
def test_every_byte_of_a_tile_belongs_to_one_token(d):
    at, par = oracle.int4_cache._places(d)
    nibbles = {(int(b), int(s)) for b, s in at.reshape(-1, 2)}
    assert len(nibbles) == 2 * 16 * d
    assert {b for b, _ in nibbles} == set(range(16 * d))
    assert sorted(int(b) + i for b in par.reshape(-1) for i in range(4)) == list(range(16 * d, 18 * d))
    owner = {}
    for kv in range(2):
        for tau in range(16):
            for b in {int(x) for x in at[kv, tau, :, 0]}:
                assert owner.setdefault(b, (kv, tau)) == (kv, tau)


@pytest.mark.parametrize("d", [64, 128])
def test_pool_and_token_writers_agree_and_read_back(d):
    rng = np.random.default_rng(d)
    k, v = (rng.standard_normal((2, 3, 32, d)).astype(np.float32) for _ in range(2))
    pool = oracle.int4_pool_from_rows(k, v)
    for p, h, t in ((0, 0, 0), (1, 2, 31), (0, 1, 17)):
        tile = np.zeros(18 * d, np.uint8)
        for kv, x in enumerate((k, v)):
            codes, params = oracle.int4_quantize_rows(x[p, h, t])
            oracle.int4_write_token(tile, t % 16, kv, codes, params)
            c2, p2 = oracle.int4_read_token(pool[p, h, t // 16], t % 16, kv)
            assert np.array_equal(c2, codes) and np.array_equal(p2, params)
    kk, vv = oracle.int4_rows_from_pool(pool)
    for x, y in ((k, kk), (v, vv)):
        g = x.reshape(-1, 64).astype(np.float64)
        step = (g.max(-1) - g.min(-1)) / 15
        # half a step, and the roundings of the step (15 times) and the minimum to bf16
        bound = step * 0.5 + 15 * step * 2.0 ** -8 + np.abs(g.min(-1)) * 2.0 ** -8
        assert np.all(np.abs(y.reshape(-1, 64) - g) <= bound[:, None] * (1 + 1e-6))


def test_quantize_special_groups():
    x = np.zeros((7, 64), np.float32)
    x[0] = 3.0                                   # constant: step 0, the minimum alone
    x[1, 5] = np.inf
    x[2, 63] = np.nan
    x[3] = np.linspace(-3.3e38, 3.3e38, 64)      # the range overflows
    x[4] = np.arange(64) % 16                    # codes are the values
    x[5] = (np.arange(64) % 31) / 2              # ties: to the even code
    x[6] = np.linspace(0, 2.0 ** -133, 64)       # a step that rounds to 0 or a subnormal
    codes, params = oracle.int4_quantize_rows(x)
    y = oracle.int4_dequantize_rows(codes, params)
    assert np.all(y[0] == 3.0) and np.all(codes[0] == 0) and params[0, 0, 0] == 0
    for i in (1, 2, 3):
        assert np.all(np.isnan(y[i])) and np.all(codes[i] == 0) and np.all(params[i] == 0x7FFF)
    assert np.array_equal(codes[4], np.arange(64) % 16) and np.array_equal(y[4], x[4])
    assert np.array_equal(codes[5], np.rint(x[5]).astype(np.uint8))
    assert np.all(np.abs(y[6] - x[6]) <= 2.0 ** -133)


def test_bf16_rounding_is_torch_s():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(5000), rng.standard_normal(5000) * 1e30, [0, -0.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8]]).astype(np.float32)
    want = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(oracle.f32_to_bf16_bits(x), want)


def test_rotation_keeps_lengths_and_is_complex_multiplication():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    a = rng.random((10, 16)) * 6
    cs = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    pos = [0, 9, 4]
    for inter in (False, True):
        y = oracle.rotate_rows_f32(x, cs, pos, inter)
        first = slice(0, 32, 2) if inter else slice(0, 16)
        second = slice(1, 32, 2) if inter else slice(16, 32)
        for t, p in enumerate(pos):
            z = (x[t, :, first] + 1j * x[t, :, second]) * np.exp(1j * a[p])
            assert np.allclose(y[t, :, first], z.real, atol=1e-5) and np.allclose(y[t, :, second], z.imag, atol=1e-5)
        assert np.array_equal(y[..., 32:], x[..., 32:])


def test_attention_oracle_against_torch():
    rng = np.random.default_rng(5)
    lens = [33, 1, 20]
    bt, pages = make_table(rng, lens, 16)
    pool = make_pool(rng, pages, 2, 16, 64)
    q = rng.standard_normal((3, 1, 8, 64))
    got = oracle.paged_multi_query_attention_int4(q, pool, bt, lens, 0.125)
    k, v = (torch.from_numpy(x) for x in oracle.int4_rows_from_pool(pool))
    for b, n in enumerate(lens):
        kk, vv = (x[bt[b, :-(-n // 16)]].transpose(0, 1).reshape(2, -1, 64)[:, :n].repeat_interleave(4, 0) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b, 0])[:, None], kk, vv, scale=0.125)[:, 0]
        assert np.allclose(got[b, 0], want.numpy(), atol=1e-12)


# ----------------------------------------------------------------------------- host checks
@pytest.fixture(scope="module")
def lib():
    return gq.load_library()


P = ctypes.c_void_p
OK = 1 << 20


def _decode(lib, B=2, Q=None, H=4, Hk=1, D=64, ps=16, scale=0.125, MB=4, pages=8, ptr=OK, ws=OK, ws_bytes=16 << 20, out=OK):
    p = P(ptr)
    q = [] if Q is None else [Q]
    fn = lib.gqa_paged_decode_attn_int4 if Q is None else lib.gqa_paged_multi_query_attn_int4
    return fn(p, p, p, p, P(out), B, *q, H, Hk, D, ps, ctypes.c_float(scale), MB, pages, P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(B=65537), -2), (dict(H=6, Hk=4), -1), (dict(H=0), -1), (dict(Hk=0), -1),
    (dict(D=96), -2), (dict(D=0), -1), (dict(ps=8), -2), (dict(ps=272), -2), (dict(ps=0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(MB=0), -1), (dict(pages=0), -1),
    (dict(pages=1 << 28), -2), (dict(MB=1 << 28), -2), (dict(ptr=0), -1), (dict(ptr=OK + 8), -1), (dict(out=OK + 8), -1),
    (dict(ws=0), -1), (dict(ws=OK + 128), -1), (dict(ws_bytes=(16 << 20) - 1), -1),
    (dict(Q=0), -1), (dict(Q=33), -2), (dict(Q=3, H=96, Hk=2), -2),
    (dict(B=0), 0), (dict(B=0, Q=32), 0), (dict(B=0, ptr=0, ws=0), 0),
    (dict(B=0, H=1 << 20, Hk=1 << 20), -2),
])
def test_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status
    if status:
        assert lib.gqa_last_error_string()


def _rope(lib, T=2, B=2, H=4, Hk=2, D=64, r=64, inter=0, maxpos=100, qs=None, ks=None, vs=None, ps=16, MB=4, pages=8, ptr=OK,
          q=None, q_out=None, seq=None, kind=""):
    p = P(ptr)
    qs, ks, vs = qs if qs is not None else H * D, ks if ks is not None else Hk * D, vs if vs is not None else Hk * D
    pools = {"": [p, p], "_fp8": [p, p, p, p], "_int4": [p]}[kind]
    fn = getattr(lib, "gqa_rope_kv_append" + kind)
    return fn(P(q if q is not None else ptr), p, p, p, P(q_out if q_out is not None else OK * 2), *pools, p, p, P(seq) if seq else None,
              T, B, H, Hk, D, r, inter, maxpos, qs, ks, vs, ps, MB, pages, None)


@pytest.mark.parametrize("kind", ["", "_fp8", "_int4"])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(B=-1), -1), (dict(H=0), -1), (dict(Hk=0), -1), (dict(D=96), -2), (dict(r=0), -1), (dict(r=8), -1),
    (dict(r=24), -1), (dict(r=80), -1), (dict(r=-16), -1), (dict(maxpos=0), -1), (dict(ps=0), -1), (dict(MB=0), -1), (dict(pages=0), -1),
    (dict(qs=252), -1), (dict(ks=120), -1), (dict(vs=132), -1), (dict(qs=260), -1), (dict(ptr=0), -1), (dict(ptr=OK + 8), -1),
    (dict(q_out=OK * 2 + 8), -1), (dict(T=3, B=2), -1), (dict(q=OK, q_out=OK, qs=512), -1),
    (dict(pages=1 << 28), -2), (dict(MB=1 << 28), -2), (dict(T=0), 0), (dict(T=0, ptr=0), 0),
])
def test_rope_refusals(lib, kind, kw, status):
    assert _rope(lib, kind=kind, **kw) == status
    if status:
        assert lib.gqa_last_error_string()


def test_int4_append_needs_tiles(lib):
    assert _rope(lib, kind="_int4", ps=8) == -2
    assert _rope(lib, kind="_int4", ps=512) == -2
    p = P(OK)
    assert lib.gqa_kv_append_int4(p, p, p, p, p, 2, 1, 64, 8, 4, 8, None) == -2
    assert lib.gqa_kv_append_int4(p, p, p, p, p, 2, 1, 72, 16, 4, 8, None) == -2
    assert lib.gqa_kv_append_int4(p, None, p, p, p, 2, 1, 64, 16, 4, 8, None) == -1
    assert lib.gqa_kv_append_int4(p, p, p, p, p, 0, 1, 64, 16, 4, 8, None) == 0


@pytest.mark.parametrize("fn", ["gqa_kv_quantize_int4", "gqa_kv_dequantize_int4"])
def test_conversion_refusals(lib, fn):
    f, p = getattr(lib, fn), P(OK)
    assert f(p, p, p, -1, 1, 16, 64, None) == -1
    assert f(p, p, p, 1, 0, 16, 64, None) == -1
    assert f(p, p, p, 1, 1, 24, 64, None) == -2
    assert f(p, p, p, 1, 1, 16, 80, None) == -2
    assert f(p, None, p, 1, 1, 16, 64, None) == -1
    assert f(p, P(OK + 4), p, 1, 1, 16, 64, None) == -1
    assert f(p, p, p, 1 << 28, 1, 16, 64, None) == -2
    assert f(None, None, None, 0, 1, 16, 64, None) == 0


def test_step_checks_both_halves_before_it_launches(lib):
    p = P(OK)

    def step(r=64, maxpos=100, cs=p, ws=p, H=4):
        return lib.gqa_decode_step_int4(p, p, p, cs, p, p, p, p, p, p, 2, H, 1, 64, r, 0, maxpos, 16, ctypes.c_float(0.1), 4, 8,
                                        ws, 16 << 20, None)
    assert step(ws=None) == -1
    assert step(H=0) == -1
    assert step(r=24) == -1
    assert step(maxpos=0) == -1


def test_binding_refuses_what_does_not_fit():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 1, 1, 18 * 64, dtype=torch.uint8)
    bt, sl = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gq.paged_decode_attn_int4(q, pool, bt, sl)
    with pytest.raises(ValueError, match="CUDA"):
        gq.quantize_pages_int4(q[None], q[None])
    with pytest.raises(ValueError, match="CUDA"):
        gq.rope_kv_append_int4(q, q[:, :1], q[:, :1], torch.zeros(4, 64), pool, bt, sl)
    with pytest.raises(ValueError, match="CUDA"):
        gq.decode_step_int4(q, q[:, :1], q[:, :1], pool, bt, sl, sl)
