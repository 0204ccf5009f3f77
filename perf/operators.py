"""Cases and plain forms of the 4-bit K/V cache and of the rotating appends.

Four operators of the paged cache are run here:

  rope     rotate q and k by position and append k, v to a bf16, e4m3 or 4-bit paged cache
  convert  a bf16 pool into the 4-bit pool, and the 4-bit pool back into bf16 values
  decode   attention of one query token per sequence over the 4-bit cache
  multi    attention of several query tokens per sequence over the 4-bit cache

Where `own` is false `run` computes them with elementary torch operations in 32 bits; where it
is true it makes the calls of gqa_decode_attention_04_b200.

The 4-bit pool.  For each token and kv head, K and V are cut into groups of 64 channels.  A group
holds its minimum and its step in bf16 and one code in 0..15 per channel; a cached value is
code * step + min.  The pool is [num_pages, num_kv_heads, page_size / 16, 18 * head_dim] bytes:
tiles of 16 tokens, each the K codes, the V codes, then (step, min) per token, K before V, per
group.  `_pack` and `_unpack` below spell out the order of the codes inside a tile.
"""
import math

import torch

own = False

GROUP = 64
TILE = 16


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat turn's single new token: the call whose latency counts
        dict(name="rope_one_token", op="rope", cache="bf16", seqs=1, tokens=1, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, page=16, longest=2048, fused=True),
        # one decode step of a continuous batch
        dict(name="rope_decode_batch", op="rope", cache="bf16", seqs=256, tokens=256, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, page=16, longest=1024, fused=True),
        # a ragged set of prompts into the 8-bit cache: partial, interleaved rotation, odd page size
        dict(name="rope_prompts_e4m3", op="rope", cache="e4m3", seqs=11, tokens=5987, heads=12, kv_heads=2, dim=64,
             rotary=32, interleaved=True, page=48, longest=1500, fused=False),
        # long prompts into the 4-bit cache, and the cache read back
        dict(name="rope_prompts_int4", op="rope", cache="int4", seqs=4, tokens=16384, heads=64, kv_heads=8, dim=128,
             rotary=128, interleaved=False, page=16, longest=8192, fused=True),
        # a few pages of a finished prompt moved into the 4-bit pool
        dict(name="convert_few_pages", op="convert", pages=37, kv_heads=8, dim=128, page=16),
        # a whole serving pool converted
        dict(name="convert_pool", op="convert", pages=9001, kv_heads=8, dim=128, page=16),
        # two short sequences, multi-query heads: latency
        dict(name="decode_tiny_mqa", op="decode", lengths="fixed", seqs=2, low=17, high=40, heads=4, kv_heads=1, dim=64,
             page=16, queries=1),
        # a serving batch
        dict(name="decode_gqa_batch", op="decode", lengths="uniform", seqs=32, low=512, high=4096, heads=32, kv_heads=8,
             dim=128, page=16, queries=1),
        # continuous batching: many lengths at once
        dict(name="decode_continuous", op="decode", lengths="log", seqs=256, low=1, high=32768, heads=32, kv_heads=8,
             dim=128, page=16, queries=1),
        # few very long contexts, some keys much larger than the rest
        dict(name="decode_long_context", op="decode", lengths="uniform", seqs=4, low=131072, high=131072, heads=64,
             kv_heads=8, dim=128, page=16, queries=1),
        # multi-query attention: 96 heads read one cached head
        dict(name="decode_mqa_batch", op="decode", lengths="uniform", seqs=64, low=8192, high=8192, heads=96, kv_heads=1,
             dim=128, page=64, queries=1),
        # drafts of four tokens verified at once
        dict(name="multi_verify_drafts", op="multi", lengths="uniform", seqs=32, low=512, high=4096, heads=32,
             kv_heads=8, dim=128, page=16, queries=4),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "convert", "decode", "decode", "decode", "multi"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op == "convert":
        return dict(op=op, pages=max(1, _log_int(rng, 16, 9000 * 128 * 16 * 8) // (page * dim * 8)),
                    kv_heads=rng.choice([1, 2, 3, 8]), dim=dim, page=page)
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        tokens = _log_int(rng, 1, 12000)
        seqs = min(tokens, _log_int(rng, 1, 300))
        step = rng.random() < 0.4
        if step:  # one token for each sequence
            seqs = tokens = min(tokens, 400)
        return dict(op=op, cache=rng.choice(["bf16", "e4m3", "int4"]), seqs=seqs, tokens=tokens,
                    heads=kv_heads * rng.choice([1, 2, 4, 7, 8]), kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, 16]), interleaved=rng.random() < 0.5, page=page,
                    longest=(2 * tokens) // seqs + rng.randrange(1, 500), fused=rng.random() < 0.5)
    if op == "multi":
        queries = rng.randrange(2, 9)
        group = rng.choice([g for g in (1, 2, 4, 6, 8, 16, 32) if g * queries <= 128])
    else:
        queries, group = 1, rng.choice([1, 2, 4, 4, 5, 8, 8, 12, 16, 24, 48, 96])
    seqs = _log_int(rng, 1, 256)
    room = 1_200_000 // max(1, kv_heads * group * queries // 16)  # tokens in all
    high = _log_int(rng, 20, max(21, min(131072, room // seqs)))
    lengths = rng.choice(["uniform", "log"])
    low = 0 if lengths == "uniform" and rng.random() < 0.2 else _log_int(rng, 1, high)
    return dict(op=op, lengths=lengths, seqs=seqs, low=low, high=high, heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, page=page, queries=queries)


# ----------------------------------------------------------------------------- the 4-bit format, plainly
def _quantize(x):
    """x [..., D] in 32 bits -> codes [..., D] (uint8), step and min [..., D / 64] (bf16)."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    low = lo.bfloat16()
    step = ((hi - lo) / 15).bfloat16()
    bad = ~(torch.isfinite(low) & torch.isfinite(step))
    low, step = low.masked_fill(bad, math.nan), step.masked_fill(bad, math.nan)
    s = step.to(x.dtype).unsqueeze(-1)
    code = ((g - low.to(x.dtype).unsqueeze(-1)) / s).round().clamp(0, 15)
    code = torch.where(s > 0, code, torch.zeros((), dtype=x.dtype, device=x.device))
    return code.to(torch.uint8).flatten(-2), step, low


def _rows(k, v):
    """K and V [..., D] of single tokens in 32 bits -> the bytes of each token [..., 18 D / 16]:
    K codes, V codes, (step, min) of K and of V."""
    (kc, ks, kl), (vc, vs, vl) = _quantize(k), _quantize(v)
    groups = k.shape[-1] // GROUP
    kc = kc.unflatten(-1, (groups, 4, 2, 8)).transpose(-4, -3)
    vc = vc.unflatten(-1, (groups, groups, 8 // groups, 8)).movedim(-4, -2)
    kc, vc = (c.flatten(-4).unflatten(-1, (-1, 2)) for c in (kc, vc))
    par = torch.stack([torch.stack([ks, kl], -1), torch.stack([vs, vl], -1)], -3).flatten(-3)
    return torch.cat([kc[..., 0] | (kc[..., 1] << 4), vc[..., 0] | (vc[..., 1] << 4), par.view(torch.uint8)], -1)


def _own_bytes(d, slot):
    """Places in a tile of the bytes of the token in each of `slot`, in _rows' order: [T, 18 D / 16]."""
    groups, dev = d // GROUP, slot.device
    slot = slot[:, None]
    k = slot * (d // 2) + torch.arange(d // 2, device=dev)
    row = (slot // 8) * 8 + (slot % 2) * 4 + (slot % 8) // 2
    v = 8 * d + (row * 32)[..., None] + torch.arange(groups, device=dev)[:, None] * 512 + torch.arange(32, device=dev)
    par = 16 * d + slot * (8 * groups) + torch.arange(8 * groups, device=dev)
    return torch.cat([k, v.flatten(1), par], 1)


def _pack(k, v):
    """K and V [N, 16, D] in 32 bits, N tiles of 16 tokens -> [N, 18 D] bytes of the pool."""
    place = _own_bytes(k.shape[-1], torch.arange(TILE, device=k.device)).flatten()
    return _rows(k, v).flatten(1)[:, place.argsort()]


def _fields(tiles):
    """Codes of K and V [N, 16, D] and (step, min) [N, 16, K/V, groups, 2] of tiles [N, 18 D]."""
    n, d = tiles.shape[0], tiles.shape[1] // 18
    groups = d // GROUP
    kc, vc, par = tiles.split([8 * d, 8 * d, 2 * d], 1)
    kc, vc = (torch.stack([c & 15, c >> 4], -1) for c in (kc, vc))
    kc = kc.reshape(n, 16, 4, groups, 2, 8).permute(0, 1, 3, 2, 4, 5).reshape(n, 16, d)
    vc = vc.reshape(n, groups, 2, 2, 4, 8 // groups, groups, 8).permute(0, 2, 4, 3, 6, 1, 5, 7).reshape(n, 16, d)
    return kc, vc, par.contiguous().view(torch.bfloat16).view(n, 16, 2, groups, 2)


def _unpack(tiles, dtype=torch.float32):
    """The values of K and V [N, 16, D] that tiles [N, 18 D] stand for."""
    kc, vc, par = _fields(tiles)
    par = par.to(dtype)
    return tuple((c.to(dtype).unflatten(-1, (-1, GROUP)) * par[:, :, i, :, :1] + par[:, :, i, :, 1:]).flatten(-2)
                 for i, c in enumerate((kc, vc)))


def _values(pool, dtype=torch.float32):
    """The whole pool as K and V pools [P, Hk, page, D]."""
    p, hk, tiles, b = pool.shape
    return tuple(x.view(p, hk, tiles * TILE, -1) for x in _unpack(pool.view(-1, b), dtype))


# ----------------------------------------------------------------------------- inputs
def _generator(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def _lengths(c, seed):
    g = _generator(seed, "cpu")
    n = c["seqs"]
    if c["lengths"] == "fixed":
        return [c["low"] + (c["high"] - c["low"]) * i // max(1, n - 1) for i in range(n)]
    if c["lengths"] == "log":
        u = torch.rand(n, generator=g, dtype=torch.float64)
        return [max(c["low"], min(c["high"], int(round(c["low"] * (c["high"] / c["low"]) ** float(x))))) for x in u]
    return torch.randint(c["low"], c["high"] + 1, (n,), generator=g).tolist()


def _table(lens, page, pages, seed):
    """A block table over a pool of so many pages, taken in shuffled order."""
    blocks = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=_generator(seed, "cpu"), dtype=torch.int64).to(torch.int32)
    table, at = torch.full((len(lens), max(1, max(blocks))), -1, dtype=torch.int32), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), pages


def _random_pool4(pages, kv_heads, page, d, g, spikes=False):
    """A 4-bit pool of normal keys and values, made a part at a time."""
    tiles = pages * kv_heads * page // TILE
    pool = torch.empty(tiles, 18 * d, dtype=torch.uint8, device="cuda")
    for at in range(0, tiles, 1 << 16):
        n = min(1 << 16, tiles - at)
        k, v = (torch.randn(n, TILE, d, generator=g, device="cuda") for _ in range(2))
        if spikes:
            k = k * (1 + 3 * (torch.rand(n, TILE, 1, generator=g, device="cuda") < 0.01))
        pool[at:at + n] = _pack(k, v)
    return pool.view(pages, kv_heads, page // TILE, 18 * d)


def _angles(positions, rotary):
    """cos and sin of every position, as models keep them: [positions, rotary] in 32 bits, cos first."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _room(c):
    """Positions that every sequence of a rope case has room for."""
    return max(c["longest"], 2 * c["tokens"] // c["seqs"] + 2)


def _pages(c):
    return c["seqs"] * -(-_room(c) // c["page"]) + 2


def _prepare_rope(c, seed):
    g, host = _generator(seed), _generator(seed, "cpu")
    n, t, d, hk, h = c["seqs"], c["tokens"], c["dim"], c["kv_heads"], c["heads"]
    # new tokens of each sequence: between half and twice the mean, one at least
    share = torch.rand(n, generator=host, dtype=torch.float64) * 2 / 3 + 2 / 3
    ends = (share.cumsum(0) / share.sum() * (t - n)).round().long() + torch.arange(1, n + 1)
    new = torch.diff(ends, prepend=ends.new_zeros(1)).tolist()
    room = _room(c)
    first = [int(torch.randint(0, room - x + 1, (1,), generator=host)) for x in new]
    table, pages = _table([f + x for f, x in zip(first, new)], c["page"], _pages(c), seed)
    ids = torch.repeat_interleave(torch.arange(n), torch.tensor(new)).to(torch.int32)
    pos = torch.cat([torch.arange(f, f + x) for f, x in zip(first, new)]).to(torch.int32)
    if c["fused"]:  # q, k and v as a fused projection leaves them
        qkv = torch.randn(t, h + 2 * hk, d, generator=g, device="cuda").bfloat16()
        q, k, v = qkv.split([h, hk, hk], 1)
    else:
        q, k, v = (torch.randn(t, x, d, generator=g, device="cuda").bfloat16() for x in (h, hk, hk))
    s = dict(case=c, q=q, k=k, v=v, cos_sin=_angles(room, c["rotary"]), table=table, pos=pos.cuda(), ids=ids.cuda(),
             q_out=torch.empty(t, h, d, dtype=torch.bfloat16, device="cuda"))
    shape = (pages, hk, c["page"], d)
    if c["cache"] == "bf16":
        s["k_pages"], s["v_pages"] = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
    elif c["cache"] == "e4m3":
        s["k_pages"], s["v_pages"] = (torch.randn(shape, generator=g, device="cuda").mul(60).to(torch.float8_e4m3fn)
                                      .view(torch.uint8) for _ in range(2))
        s["k_scale"], s["v_scale"] = (torch.rand(hk, generator=g, device="cuda") * 0.01 + 0.01 for _ in range(2))
    else:
        s["kv_pages"] = _random_pool4(pages, hk, c["page"], d, g)
        s["k_out"], s["v_out"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "rope":
        return _prepare_rope(c, seed)
    g, d, hk = _generator(seed), c["dim"], c["kv_heads"]
    if c["op"] == "convert":
        shape = (c["pages"], hk, c["page"], d)
        # keys have channels that are larger than the others and off zero
        bias = torch.randn(hk, 1, d, generator=g, device="cuda") * 0.5
        k = (torch.randn(shape, generator=g, device="cuda") + bias).bfloat16()
        v = torch.randn(shape, generator=g, device="cuda").bfloat16()
        return dict(case=c, k_pages=k, v_pages=v, k_out=torch.empty_like(k), v_out=torch.empty_like(v),
                    kv_pages=torch.empty(c["pages"], hk, c["page"] // TILE, 18 * d, dtype=torch.uint8, device="cuda"))
    lens = _lengths(c, seed)
    table, pages = _table(lens, c["page"], sum(-(-x // c["page"]) for x in lens) + 2, seed)
    n, h, m = c["seqs"], c["heads"], c["queries"]
    q = torch.randn(n, m, h, d, generator=g, device="cuda").bfloat16()
    s = dict(case=c, q=q if c["op"] == "multi" else q[:, 0], lens=lens, table=table,
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             kv_pages=_random_pool4(pages, hk, c["page"], d, g, spikes=min(lens) > 100000),
             out=torch.empty_like(q if c["op"] == "multi" else q[:, 0]),
             workspace=torch.zeros(16 << 20, dtype=torch.uint8, device="cuda"))
    return s


# ----------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rotary, interleaved):
    """x [T, heads, D] in 32 bits, cos and sin [T, rotary / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    r, rest = x[..., :rotary], x[..., rotary:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), rest], -1)


def _slots(s):
    """Page and slot of every new token."""
    page, pos = s["case"]["page"], s["pos"].long()
    return s["table"][s["ids"].long(), pos // page].long(), pos % page


def _plain_rope(s):
    c = s["case"]
    cos, sin = s["cos_sin"][s["pos"].long()].chunk(2, 1)
    q, k = (_rotate(s[x].float(), cos, sin, c["rotary"], c["interleaved"]) for x in "qk")
    v = s["v"].float()
    s["q_out"].copy_(q)
    page, slot = _slots(s)
    if c["cache"] == "bf16":
        s["k_pages"][page, :, slot] = k.bfloat16()
        s["v_pages"][page, :, slot] = v.bfloat16()
        return s["q_out"], s["k_pages"], s["v_pages"]
    if c["cache"] == "e4m3":
        for x, name in ((k, "k"), (v, "v")):
            code = (x / s[name + "_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_pages"][page, :, slot] = code
        return s["q_out"], s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn)
    hk, d = c["kv_heads"], c["dim"]
    tile = (page[:, None] * hk + torch.arange(hk, device="cuda")) * (c["page"] // TILE) + (slot // TILE)[:, None]
    place = tile[..., None] * (18 * d) + _own_bytes(d, slot % TILE)[:, None]  # [T, Hk, bytes of a token]
    s["kv_pages"].view(-1)[place] = _rows(k, v)
    kv, vv = _values(s["kv_pages"])
    s["k_out"].copy_(kv)
    s["v_out"].copy_(vv)
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_convert(s):
    c = s["case"]
    d = c["dim"]
    s["kv_pages"].copy_(_pack(*(s[x].float().view(-1, TILE, d) for x in ("k_pages", "v_pages"))).view(s["kv_pages"].shape))
    kv, vv = _values(s["kv_pages"])
    s["k_out"].copy_(kv)
    s["v_out"].copy_(vv)
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    c = s["case"]
    d, hk, page, m = c["dim"], c["kv_heads"], c["page"], c["queries"]
    group = c["heads"] // hk
    q = s["q"].view(c["seqs"], m, hk, group, d).permute(0, 2, 1, 3, 4).float() / math.sqrt(d)
    out = s["out"].view(c["seqs"], m, hk, group, d)
    buckets = {}
    for b, n in enumerate(s["lens"]):  # sequences of like lengths are attended together
        buckets.setdefault(max(n, 1).bit_length(), []).append(b)
    for at in buckets.values():
        blocks = max(1, -(-max(s["lens"][b] for b in at) // page))
        at = torch.tensor(at, device="cuda")
        tiles = s["kv_pages"][s["table"][at, :blocks].clamp(min=0).long()]  # [b, blocks, Hk, page / 16, 18 D]
        n = blocks * page
        tiles = tiles.permute(0, 2, 1, 3, 4).reshape(-1, 18 * d)
        k, v = (x.view(len(at), hk, n, d) for x in _unpack(tiles))
        score = q[at].flatten(2, 3) @ k.transpose(2, 3)  # [b, Hk, queries * group, n]
        ends = s["seq_lens"][at, None] - m + 1 + torch.arange(m, device="cuda")  # tokens that each query sees
        hidden = torch.arange(n, device="cuda") >= ends[..., None]
        score = score.unflatten(2, (m, group)).masked_fill(hidden[:, None, :, None], -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)
        p = (score - top).exp()
        o = (p.flatten(2, 3) @ v).unflatten(2, (m, group)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
        out[at] = o.permute(0, 2, 1, 3, 4).bfloat16()
    return s["out"]


# ----------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "convert": _plain_convert}.get(c["op"], _plain_attend)(s)
    import gqa_decode_attention_04_b200 as gq
    if c["op"] == "convert":
        gq.quantize_pages_int4(s["k_pages"], s["v_pages"], s["kv_pages"])
        gq.dequantize_pages_int4(s["kv_pages"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if c["op"] == "decode":
        return gq.paged_decode_attn_int4(s["q"], s["kv_pages"], s["table"], s["seq_lens"], s["out"],
                                         workspace=s["workspace"])
    if c["op"] == "multi":
        return gq.paged_multi_query_attn_int4(s["q"], s["kv_pages"], s["table"], s["seq_lens"], s["out"],
                                              workspace=s["workspace"])
    more = dict(seq_ids=s["ids"], interleaved=c["interleaved"], q_out=s["q_out"])
    new = (s["q"], s["k"], s["v"], s["cos_sin"])
    if c["cache"] == "bf16":
        gq.rope_kv_append(*new, s["k_pages"], s["v_pages"], s["table"], s["pos"], **more)
        return s["q_out"], s["k_pages"], s["v_pages"]
    if c["cache"] == "e4m3":
        gq.rope_kv_append_fp8(*new, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["pos"], **more)
        return s["q_out"], s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn)
    gq.rope_kv_append_int4(*new, s["kv_pages"], s["table"], s["pos"], **more)
    gq.dequantize_pages_int4(s["kv_pages"], s["k_out"], s["v_out"])
    return s["q_out"], s["k_out"], s["v_out"]


def work(case):
    c = case
    d, hk = c["dim"], c["kv_heads"]
    row4 = 9 * d / 8  # bytes of one token's K and V of one kv head in the 4-bit cache
    if c["op"] == "convert":
        rows = c["pages"] * c["page"] * hk
        return dict(bytes=rows * (8 * d + 2 * row4), flops=rows * d * 16)
    if c["op"] == "rope":
        t, h = c["tokens"], c["heads"]
        size = {"bf16": 4 * d, "e4m3": 2 * d, "int4": row4}[c["cache"]]
        total = t * ((2 * h + 2 * hk) * d * 2 + c["rotary"] * 4 + 12 + hk * size)
        if c["cache"] == "int4":  # the whole pool read back as bf16 values
            total += _pages(c) * c["page"] * hk * (row4 + 4 * d)
        return dict(bytes=total, flops=t * (h + hk) * c["rotary"] * 3)
    if c["lengths"] == "log":
        mean = (c["high"] - c["low"]) / math.log(c["high"] / c["low"]) if c["high"] > c["low"] else c["low"]
    else:
        mean = (c["low"] + c["high"]) / 2
    tokens = c["seqs"] * mean
    rows = c["seqs"] * c["queries"] * c["heads"] * d * 4
    return dict(bytes=tokens * hk * row4 + rows + 4 * tokens / c["page"], flops=4 * d * tokens * c["heads"] * c["queries"])


# ----------------------------------------------------------------------------- from the definition, in 64 bits
def _exact_row4(x):
    """The 4-bit cache's values of rows x [..., D] in 64 bits: bf16 step and minimum belong to the format."""
    out = torch.empty_like(x)
    for at in range(0, x.shape[-1], GROUP):
        g = x[..., at:at + GROUP]
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        low, step = lo.to(torch.bfloat16).double(), ((hi - lo) / 15).to(torch.bfloat16).double()
        code = torch.where(step > 0, torch.round((g - low) / torch.where(step > 0, step, 1.0)), 0.0)
        out[..., at:at + GROUP] = low + step * code.clamp(0, 15)
    return out


def _exact_rope(s):
    c = s["case"]
    r, pos = c["rotary"], s["pos"].long()
    angle = s["cos_sin"].double()[pos]
    turn = torch.complex(angle[:, :r // 2], angle[:, r // 2:])[:, None]
    new = []
    for x in (s["q"].double(), s["k"].double()):
        y = x.clone()
        first, second = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        new.append(y)
    q, k = new
    v = s["v"].double()
    page, slot = _slots(s)
    if c["cache"] == "int4":
        pools = list(_values(s["kv_pages"], torch.float64))
        rows = (_exact_row4(k), _exact_row4(v))
    elif c["cache"] == "bf16":
        pools, rows = [s["k_pages"].double(), s["v_pages"].double()], (k, v)
    else:
        pools = [s[x].view(torch.float8_e4m3fn).double() for x in ("k_pages", "v_pages")]
        rows = [(x / s[n].double()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()
                for x, n in ((k, "k_scale"), (v, "v_scale"))]
    for pool, x in zip(pools, rows):
        pool[page, :, slot] = x
    return q, *pools


def _exact_attend(s):
    c = s["case"]
    d, hk, page, m = c["dim"], c["kv_heads"], c["page"], c["queries"]
    group = c["heads"] // hk
    q = s["q"].view(c["seqs"], m, hk, group, d)
    out = torch.zeros(c["seqs"], m, hk, group, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // page)].long()
        for j in range(hk):
            k, v = (x.reshape(-1, d)[:n] for x in _unpack(s["kv_pages"][pages, j].reshape(-1, 18 * d), torch.float64))
            for i in range(m):
                seen = n - m + 1 + i
                if seen > 0:
                    p = torch.softmax(q[b, i, j].double() @ k[:seen].T * d ** -0.5, -1)
                    out[b, i, j] = p @ v[:seen]
    return out.view(s["out"].shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "convert":
        return tuple(_exact_row4(s[x].double()) for x in ("k_pages", "v_pages"))
    return _exact_attend(s)
