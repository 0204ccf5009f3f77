// Decode attention over the 4-bit paged cache (include/gqa_int4.h), one or several query
// tokens per sequence.
//
// Mathematics.  With c the code, s the step and m the minimum of a group (k = c s + m),
//   <q, k_t> = sum_g s_tg <q_g, c_tg> + m_tg sum(q_g)
//   O        = sum_t (p_t s_t) c_t + sum_t p_t m_t
// so the tensor cores multiply bare codes and the steps and minima meet them as scalars per
// token.  A nibble masked out of its 32-bit word, two at a time, IS a pair of fp16 numbers:
// bits 0-3 of a half are the subnormal c * 2^-24, bits 4-7 are c * 2^-20.  So widening costs one
// logical operation per two codes (plus a shift per four), no conversion and no subtraction;
// fp16 MMAs take subnormals exactly, and the powers of two are folded into q (for K: the odd
// nibbles' channels of q are scaled by 2^-4) and into the output (for V).
//   q is scaled by a power of two per row so that its largest element lies in [2^14, 2^15):
// exact in fp16 for elements within 2^-28 of it (bf16 has 8 significant bits), and the products
// with c * 2^-24 stay normal in fp32.
//   p s is rounded to fp16.  Steps may be of any size, so each row carries a power of two F per
// group that keeps p s F below 2^15; it moves with the running maximum.  Scores, sums and
// outputs are fp32.
//
// Bound: HBM at small groups -- 9/8 D bytes per token and kv head.  At that rate a tile of 16
// tokens has to be done every ~100 cycles per SM, which leaves about 400 issue slots a tile,
// and that is what the shape is for: warps that never wait for one another.
//
// Work.  The list of tiles (sequence, kv head, row tile, 16-token tile), in that order, is cut
// into one equal contiguous range per WARP.  Each warp streams its range through its own ring
// of kStages tiles in shared memory (one bulk copy per tile: K, V and parameters lie together),
// and keeps the running maximum, sum and output of its current segment in registers; there is no
// producer warp and no barrier in the loop.  A segment wholly inside a warp's range is written out
// at once.  What a range cuts is left in shared memory (at most the first and the last segment of
// a warp), merged over the CTA's warps after one __syncthreads, and over CTAs through two
// workspace slots per CTA: the last CTA to arrive at a segment's counter merges it.
//
// The S tile is computed transposed, S^T = K Q^T (tokens on the MMA's 16-row side, 8 query
// rows on the other), so a group of 4 or 8 heads needs no padding to 16.
//
// Safety: every wait is bounded; a warp whose wait runs out sets the error word, treats the rest
// of its range as masked, drains its own copies (bounded) and still takes part in the merges, so
// no counter is left behind.  Page ids and lengths are range-checked before use.
#include <type_traits>

#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

namespace {

constexpr int kWarps = 8;
constexpr float kNone = -3.0e38f;   // reference of a row that has seen no token

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;              // query rows of a segment
  static constexpr int kGroups = D / 64;
  static constexpr int kTileBytes = 18 * D;
  static constexpr int kUnitBytes = 2 * kTileBytes;
  static constexpr int kStages = NT == 1 ? 2 : 4;
  static constexpr int kCtas = NT == 1 ? 2 : 1;     // per SM
  static constexpr int kRecFloats = kRows * (D + 2);  // a piece: [rows][D], then (reference, sum)
  static constexpr int kRingBytes = kStages * kUnitBytes;
  static_assert(kRingBytes >= kRecFloats * 4, "the last piece of a warp is left in its ring");
  static constexpr int kRecBytes = (kRecFloats * 4 + 127) / 128 * 128;
  static constexpr int kSmem = kWarps * (kRingBytes + kRecBytes);
};

// A piece that a warp's range cut off.
struct Piece {
  int64_t start;  // position of the segment's first unit in the list
  int units;      // of the segment; 0: no piece
  int b, seg;     // sequence and segment in it
};

constexpr int kUnit = 2 * int4::kTile;  // tokens per step of a warp

__device__ __forceinline__ int units_of(int len) { return (len + kUnit - 1) / kUnit; }

// The length of sequence b, 0 if it is out of range.
__device__ __forceinline__ int checked_len(const Int4DecodeParams& p, int b) {
  const int L = __ldg(p.seq_lens + b);
  return L < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(p.max_blocks) * p.page_size ? 0 : L;
}

// Moves b on to the next sequence that has tokens; its length.  (There is one, unless the
// lengths changed under the call: then the last sequence is taken again.)
__device__ __forceinline__ int next_len(const Int4DecodeParams& p, int& b) {
  int len = 1;
  while (b + 1 < p.num_seqs && (len = checked_len(p, ++b)) == 0) {
  }
  return max(len, 1);
}

// The query token of row r of a kv head.
__device__ __forceinline__ int token_of(const Int4DecodeParams& p, int r) { return p.q_len == 1 ? 0 : r / p.group; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ void st_bf16x4(uint16_t* dst, const float4& o, float inv) {
  uint2 w;
  w.x = ptx::pack_bf16x2(o.x * inv, o.y * inv);
  w.y = ptx::pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(dst) = w;
}

// 2^-floor(log2 m) for m > 0 (finite), between 2^-126 and 2^126; 2^100 for 0 or less.
__device__ __forceinline__ float inverse_pow2(float m) {
  if (!(m > 0.0f)) return 0x1p100f;
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;  // (a subnormal counts as 2^-127)
  e = max(-126, min(126, e));
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, (Cfg<D, NT>::kCtas)) decode_int4_kernel(const Int4DecodeParams p) {
  using C = Cfg<D, NT>;
  using L4 = int4::Layout<D>;
  constexpr int G = C::kGroups;
  constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;

  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t excl[32 * kWarps];  // tiles of the sequences before each thread's chunk
  __shared__ int64_t scan[kWarps];
  __shared__ __align__(8) uint64_t full[kWarps][C::kStages];
  __shared__ Piece pieces[2 * kWarps];
  __shared__ int last_of[2];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  unsigned char* ring = smem + warp * C::kRingBytes;
  float* rec_of[2];
  rec_of[0] = reinterpret_cast<float*>(smem + kWarps * C::kRingBytes + warp * C::kRecBytes);
  rec_of[1] = reinterpret_cast<float*>(ring);

  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) ptx::mbar_init(ptx::smem_u32(&full[warp][s]), 2);  // lanes 0 and 1
    ptx::fence_mbarrier_init();
    pieces[2 * warp].units = 0;
    pieces[2 * warp + 1].units = 0;
  }

  // ---- the split: tiles before each thread's chunk of sequences
  const int segs = p.num_kv_heads * p.n_rt;  // segments per sequence
  const int chunk = (p.num_seqs + 32 * kWarps - 1) / (32 * kWarps);
  {
    int64_t mine = 0;
    const int b0 = threadIdx.x * chunk, b1 = min(p.num_seqs, b0 + chunk);
    for (int b = b0; b < b1; ++b) mine += units_of(checked_len(p, b));
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += scan[w];
    excl[threadIdx.x] = before + incl - mine;
    __syncthreads();
  }
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) total += scan[w];
  total *= segs;
  // as many warps as there are tiles, if that is fewer
  const int64_t workers = min(static_cast<int64_t>(gridDim.x) * kWarps, total);
  auto start_of = [&](int64_t w) { return w >= workers ? total : total * w / workers; };
  auto owner_of = [&](int64_t tile) { return ((tile + 1) * workers - 1) / total; };
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  int64_t pos = start_of(me);
  const int64_t end = start_of(me + 1);

  ptx::pdl_wait_prerequisites();  // q and the pool may be written by the preceding append

  // Rows of sequences without a token (a length out of range counts as none and is reported).
  for (int64_t b = me; b < p.num_seqs; b += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int raw = __ldg(p.seq_lens + b);
    if (checked_len(p, static_cast<int>(b)) != 0) continue;
    if (raw != 0 && lane == 0) atomicOr(p.err, kErrBounds);
    uint4* o = reinterpret_cast<uint4*>(p.out + b * p.q_len * p.num_heads * D);
    for (int i = lane; i < p.q_len * p.num_heads * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
  }

  if (pos < end) {
    // ---- find the first tile: the chunk, then the sequence in it
    const int64_t unit = pos / segs;  // in tiles per row tile
    int ci = 0;
    for (int i = 0; i < kWarps; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, excl[32 * i + lane] <= unit);
      ci += __popc(m);
    }
    int b = (ci - 1) * chunk;
    int64_t base = excl[ci - 1];
    int len = 0;
    for (;; b += 32) {
      const int mine = b + lane < p.num_seqs ? checked_len(p, b + lane) : 0;
      int64_t incl = units_of(mine);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + incl > unit);
      if (past != 0) {
        const int at = __ffs(past) - 1;
        b += at;
        len = __shfl_sync(0xffffffffu, mine, at);
        base += __shfl_sync(0xffffffffu, incl, at) - units_of(len);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      if (b + 32 >= p.num_seqs) break;  // only if the lengths changed under the call
    }
    if (len == 0) pos = end;
    int seg = static_cast<int>((pos - base * segs) / max(1, units_of(len)));
    int unit0 = static_cast<int>(pos - base * segs - static_cast<int64_t>(seg) * units_of(len));
    int left = static_cast<int>(min(end - pos, int64_t{INT32_MAX}));  // units to do

    // ---- the copies' cursor runs kStages units ahead of the arithmetic's.  Lanes 0 and 1 bring
    // one tile each of a unit.
    int pb = b, phead = seg / p.n_rt, prt = seg - phead * p.n_rt, punit = unit0, plen = len, pleft = left;
    int win = -1, win_b = -1;  // first block and sequence of the block-table window (one entry per lane)
    int entry = 0, pstage = 0;
    uint32_t bad = 0, phase = 0;  // two bits per stage: no data behind the tile; bit per stage: parity to wait for
    const uint32_t ring_at = ptx::smem_u32(ring), bar_at = ptx::smem_u32(&full[warp][0]);
    auto produce = [&]() {
      if (pleft <= 0) return;
      const int ptile = 2 * punit + (lane & 1);
      const int block = p.tpp_magic != 0 ? fast_div(ptile, p.tpp_magic, p.tpp_shift) : ptile;
      const int block0 = p.tpp_magic != 0 ? fast_div(2 * punit, p.tpp_magic, p.tpp_shift) : 2 * punit;
      // (31: the unit's second tile may be in the next block)
      if (pb != win_b || static_cast<unsigned>(block0 - win) >= 31u) {
        win = block0;
        win_b = pb;
        entry = win + lane < p.max_blocks ? __ldg(p.block_table + static_cast<int64_t>(pb) * p.max_blocks + win + lane) : -1;
      }
      const int page = __shfl_sync(0xffffffffu, entry, block - win);
      const bool wanted = ptile * int4::kTile < plen;  // (the last unit may be one tile)
      const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
      const unsigned lost = __ballot_sync(0xffffffffu, !ok || !wanted) & 3u;
      bad = (bad & ~(3u << (2 * pstage))) | (lost << (2 * pstage));
      if (lane < 2) {
        const uint32_t bar = bar_at + 8 * pstage;
        if (ok && wanted) {
          const uint32_t at = (static_cast<uint32_t>(page) * p.num_kv_heads + phead) * p.tiles_per_page +
                              (ptile - block * p.tiles_per_page);
          ptx::mbar_arrive_expect_tx(bar, C::kTileBytes);
          if (!p.arm_without_copy)
            ptx::bulk_load(ring_at + pstage * C::kUnitBytes + lane * C::kTileBytes,
                           p.pool + static_cast<uint64_t>(at) * C::kTileBytes, C::kTileBytes, bar);
        } else {
          if (wanted) atomicOr(p.err, kErrBounds);
          ptx::mbar_arrive(bar);
        }
      }
      pstage = pstage + 1 == C::kStages ? 0 : pstage + 1;
      --pleft;
      if (++punit == units_of(plen)) {
        punit = 0;
        if (++prt == p.n_rt) {
          prt = 0;
          if (++phead == p.num_kv_heads) {
            phead = 0;
            if (pleft > 0) plen = next_len(p, pb);
          }
        }
      }
    };
    __syncwarp();
    for (int s = 0; s < C::kStages; ++s) produce();

    int stage = 0;
    bool dead = false;
    while (left > 0) {
      // ---- a piece: units [unit0, unit0 + count) of segment (b, seg)
      const int n = units_of(len);
      const int count = min(n - unit0, left);
      const int head = seg / p.n_rt, row0 = (seg - head * p.n_rt) * C::kRows;

      // q fragments (B operand: k = channels, n = rows), row sums and scales
      uint32_t qf[NT][2 * G * 2][2];
      uint32_t qsum[NT];  // B operand of the minima's product: k = t holds group t % G, its upper then lower bits
      float h[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        uint4 w[2 * G];
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) w[i] = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
          const int tok = token_of(p, r);
          const uint16_t* src = p.q + ((static_cast<int64_t>(b) * p.q_len + tok) * p.num_heads +
                                       static_cast<int64_t>(head) * p.group + (r - tok * p.group)) * D;
#pragma unroll
          for (int i = 0; i < 2 * G; ++i)
            w[i] = *reinterpret_cast<const uint4*>(src + 64 * (i / 2) + 16 * t + 8 * (i % 2));
        }
        float x[2 * G][8], top = 0.0f, sum[G];
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
          int4::unpack8(w[i], x[i]);
          if (i % 2 == 0) sum[i / 2] = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            top = int4::max_nan(top, fabsf(x[i][e]));
            sum[i / 2] += x[i][e];
          }
        }
        top = int4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = int4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
#pragma unroll
        for (int u = 0; u < G; ++u) {
          sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 1);
          sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 2);
        }
        // up = 2^e with top * 2^e in [2^14, 2^15), |e| <= 100
        const int top_e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int e = max(-100, min(100, 14 - top_e));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        float down = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 24 - e) << 23);
        if (!(top < INFINITY)) down = __uint_as_float(0x7fffffffu);  // the row is NaN
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
          float* y = x[i];
          const float up4 = up * 0.0625f;
          qf[nt][2 * i][0] = ptx::pack_f16x2(y[0] * up, y[4] * up);
          qf[nt][2 * i][1] = ptx::pack_f16x2(y[1] * up4, y[5] * up4);
          qf[nt][2 * i + 1][0] = ptx::pack_f16x2(y[2] * up, y[6] * up);
          qf[nt][2 * i + 1][1] = ptx::pack_f16x2(y[3] * up4, y[7] * up4);
        }
        // The sum of q in the units of the codes' products, cut into two parts of 11 bits, which
        // tf32 holds exactly: the minima (bf16) times them lose 2^-22 at most.
        const float mine = (G == 2 && (t & 1) ? sum[G - 1] : sum[0]) * up * 0x1p-24f;
        const float upper = __uint_as_float(__float_as_uint(mine) & 0xffffe000u);
        const float lower = __uint_as_float(__float_as_uint(mine - upper) & 0xffffe000u);
        qsum[nt] = __float_as_uint(t / G == 0 ? upper : (t / G == 1 ? lower : 0.0f));
        // this thread's score columns are rows 2 t and 2 t + 1 of the row tile
#pragma unroll
        for (int c = 0; c < 2; ++c) h[nt][c] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * c);
      }

      float o[G * 4][NT][4], l[NT][2], pm[NT][G][2], ref[NT][2], F[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < G * 4; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[m][nt][x] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[nt][c] = 0.0f;
          ref[nt][c] = kNone;
          F[nt][c] = 1.0f;
#pragma unroll
          for (int u = 0; u < G; ++u) pm[nt][u][c] = 0.0f;
        }
      }

      // One tile whose first token is tok0.  ENDS: some row's window ends in it.
      auto attend = [&](const unsigned char* at, int tok0, auto ends_tag) {
        constexpr bool ENDS = decltype(ends_tag)::value;
        // ---- S^T = K Q^T per group, and the minima's part of it
        float s[NT][G][4], bias[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            bias[nt][x] = 0.0f;
#pragma unroll
            for (int u = 0; u < G; ++u) s[nt][u][x] = 0.0f;
          }
        uint32_t ka[2 * G], kb[2 * G];
        uint32_t par[2][2 * G];  // tokens g, g + 8: (step, low) of K's groups, then V's
        if (G == 2) {
          const uint4 a = *reinterpret_cast<const uint4*>(at + g * 64 + t * 16);
          const uint4 c = *reinterpret_cast<const uint4*>(at + (g + 8) * 64 + t * 16);
          ka[0] = a.x; ka[1] = a.y; ka[2 * G - 2] = a.z; ka[2 * G - 1] = a.w;
          kb[0] = c.x; kb[1] = c.y; kb[2 * G - 2] = c.z; kb[2 * G - 1] = c.w;
          const uint4 pa = *reinterpret_cast<const uint4*>(at + L4::kParams + g * 16);
          const uint4 pc = *reinterpret_cast<const uint4*>(at + L4::kParams + (g + 8) * 16);
          par[0][0] = pa.x; par[0][1] = pa.y; par[0][2 * G - 2] = pa.z; par[0][2 * G - 1] = pa.w;
          par[1][0] = pc.x; par[1][1] = pc.y; par[1][2 * G - 2] = pc.z; par[1][2 * G - 1] = pc.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(at + g * 32 + t * 8);
          const uint2 c = *reinterpret_cast<const uint2*>(at + (g + 8) * 32 + t * 8);
          ka[0] = a.x; ka[1] = a.y;
          kb[0] = c.x; kb[1] = c.y;
          const uint2 pa = *reinterpret_cast<const uint2*>(at + L4::kParams + g * 8);
          const uint2 pc = *reinterpret_cast<const uint2*>(at + L4::kParams + (g + 8) * 8);
          par[0][0] = pa.x; par[0][1] = pa.y;
          par[1][0] = pc.x; par[1][1] = pc.y;
        }
        {
          const uint32_t low_a = (G == 2 && (t & 1) ? par[0][G - 1] : par[0][0]) & 0xffff0000u;
          const uint32_t low_c = (G == 2 && (t & 1) ? par[1][G - 1] : par[1][0]) & 0xffff0000u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ptx::mma_tf32_1684(bias[nt], low_a, low_c, qsum[nt]);
        }
#pragma unroll
        for (int w = 0; w < 2 * G; ++w) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a = half ? ka[w] >> 8 : ka[w], c = half ? kb[w] >> 8 : kb[w];
            const uint32_t frag[4] = {a & kLo, c & kLo, a & kHi, c & kHi};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              ptx::mma_f16_16816(s[nt][w / 2], frag, qf[nt][2 * w + half][0], qf[nt][2 * w + half][1]);
          }
        }
        float step[2][G], low[2][G];  // of V: [token g, g + 8][group]
        float sc[NT][4];              // scores, in units of log2 once multiplied by h
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int u = 0; u < G; ++u) {
            step[r][u] = __uint_as_float(par[r][G + u] << 16);
            low[r][u] = __uint_as_float(par[r][G + u] & 0xffff0000u);
            const float ks = __uint_as_float(par[r][u] << 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                sc[nt][2 * r + c] = fmaf(ks, s[nt][u][2 * r + c], u == 0 ? bias[nt][2 * r + c] : sc[nt][2 * r + c]);
          }
          if (ENDS && tok0 + g + 8 * r >= len) {  // past the sequence: no parameters
#pragma unroll
            for (int u = 0; u < G; ++u) step[r][u] = low[r][u] = 0.0f;
          }
        }
        bool seen[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            seen[nt][x] = true;
            if (ENDS) {
              const int lim = min(len, len - p.q_len + 1 + token_of(p, row0 + nt * 8 + 2 * t + x % 2));
              seen[nt][x] = tok0 + g + 8 * (x / 2) < lim;
            }
          }
        // ---- weights; the reference moves only when a score passes it by 2^8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t hh = ptx::f2_pack(h[nt][0], h[nt][1]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint64_t y = ptx::f2_mul(ptx::f2_pack(sc[nt][2 * r], sc[nt][2 * r + 1]), hh);
            ptx::f2_unpack(y, sc[nt][2 * r], sc[nt][2 * r + 1]);
          }
        }
        float pr[NT][4], w[NT][G][4];
        bool up;
        auto weigh = [&]() {
          float big = 0.0f, top = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              // (packed pairs: the two rows of a token)
              float y[2];
              ptx::f2_unpack(ptx::f2_sub(ptx::f2_pack(sc[nt][2 * r], sc[nt][2 * r + 1]), ptx::f2_pack(ref[nt][0], ref[nt][1])), y[0], y[1]);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                pr[nt][2 * r + c] = ptx::ex2(y[c]);
                if (ENDS && !seen[nt][2 * r + c]) pr[nt][2 * r + c] = 0.0f;
              }
              ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(pr[nt][2 * r], pr[nt][2 * r + 1]), ptx::f2_pack(F[nt][0], F[nt][1])), y[0], y[1]);
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int u = 0; u < G; ++u) {
                  w[nt][u][2 * r + c] = y[c] * step[r][u];
                  if (ENDS && !seen[nt][2 * r + c]) w[nt][u][2 * r + c] = 0.0f;
                }
            }
            top = ptx::max3(top, pr[nt][0], pr[nt][1]);
            top = ptx::max3(top, pr[nt][2], pr[nt][3]);
#pragma unroll
            for (int u = 0; u < G; ++u) {
              big = ptx::max3(big, w[nt][u][0], w[nt][u][1]);
              big = ptx::max3(big, w[nt][u][2], w[nt][u][3]);
            }
          }
          up = top > 256.0f || big > 32768.0f;
        };
        weigh();
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = ref[nt][c], at0 = sc[nt][c], at1 = sc[nt][c + 2];
              if (seen[nt][c]) top = fmaxf(top, at0);
              if (seen[nt][c + 2]) top = fmaxf(top, at1);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              const float a = ptx::ex2(ref[nt][c] - top);
              ref[nt][c] = top;
              l[nt][c] *= a;
              float big = 0.0f;
#pragma unroll
              for (int u = 0; u < G; ++u) {
                pm[nt][u][c] *= a;
                if (seen[nt][c]) big = fmaxf(big, ptx::ex2(at0 - top) * step[0][u]);
                if (seen[nt][c + 2]) big = fmaxf(big, ptx::ex2(at1 - top) * step[1][u]);
              }
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
              // the largest weight so far in [2^6, 2^8): 2^8 below the bound, as far as scores may pass
              // the reference, and 2^20 above fp16's subnormals
              const float before = a / F[nt][c];
              const float f = inverse_pow2(fmaxf(big * 0x1p-6f, before));
              const float scale = before * f;
              F[nt][c] = f;
#pragma unroll
              for (int m = 0; m < 4 * G; ++m) {
                o[m][nt][c] *= scale;
                o[m][nt][c + 2] *= scale;
              }
            }
          weigh();
        }
        uint32_t pb16[NT][G][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            ptx::f2_unpack(ptx::f2_add(ptx::f2_pack(l[nt][0], l[nt][1]), ptx::f2_pack(pr[nt][2 * r], pr[nt][2 * r + 1])), l[nt][0], l[nt][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
#pragma unroll
            for (int u = 0; u < G; ++u)
              if (!ENDS || seen[nt][x]) pm[nt][u][x % 2] = fmaf(pr[nt][x], low[x / 2][u], pm[nt][u][x % 2]);
          }
#pragma unroll
          for (int u = 0; u < G; ++u) {
            pb16[nt][u][0] = ptx::movmatrix_trans(ptx::pack_f16x2(w[nt][u][0], w[nt][u][1]));
            pb16[nt][u][1] = ptx::movmatrix_trans(ptx::pack_f16x2(w[nt][u][2], w[nt][u][3]));
          }
        }
        // ---- O^T += V^T P^T: tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of this thread's channels
        uint32_t v[4][G];
        const unsigned char* vat = at + L4::kVCodes + (g / (8 / G)) * 512 + t * 32 + (g % (8 / G)) * (4 * G);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (G == 2) {
            const uint2 a = *reinterpret_cast<const uint2*>(vat + q * 128);
            v[q][0] = a.x;
            v[q][G - 1] = a.y;
          } else {
            v[q][0] = *reinterpret_cast<const uint32_t*>(vat + q * 128);
          }
        }
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t sel = m < 2 ? 0x5410u : 0x7632u;
            uint32_t a = prmt(v[0][u], v[1][u], sel), c = prmt(v[2][u], v[3][u], sel);
            if (m % 2) {
              a >>= 8;
              c >>= 8;
            }
            const uint32_t frag[4] = {a & kLo, a & kHi, c & kLo, c & kHi};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ptx::mma_f16_16816(o[4 * u + m][nt], frag, pb16[nt][u][0], pb16[nt][u][1]);
          }
      };

      for (int i = 0; i < count; ++i) {
        if (!dead) {
          const bool ok = ptx::mbar_wait_bounded(bar_at + 8 * stage, (phase >> stage) & 1u, p.wait_limit_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            dead = true;
            if (lane == 0) atomicOr(p.err, kErrTimeout);
            if (!p.arm_without_copy) {  // nothing may still be landing when the ring is written or given up
              const int in_flight = left - pleft - i;
              for (int k = 0, st = stage; k < in_flight; ++k, st = st + 1 == C::kStages ? 0 : st + 1)
                ptx::mbar_wait_bounded(bar_at + 8 * st, (phase >> st) & 1u, p.wait_limit_ns);
              __syncwarp();
            }
          }
        }
        if (!dead) {
          const unsigned char* at = ring + stage * C::kUnitBytes;
          const int tok0 = (unit0 + i) * kUnit;
          const uint32_t lost = (bad >> (2 * stage)) & 3u;
          if (lost == 0 && tok0 + kUnit <= len - p.q_len + 1) {
#pragma unroll 1
            for (int k = 0; k < 2; ++k) attend(at + k * C::kTileBytes, tok0 + k * int4::kTile, std::false_type{});
          } else {
#pragma unroll 1
            for (int k = 0; k < 2; ++k)
              if ((lost >> k & 1u) == 0) attend(at + k * C::kTileBytes, tok0 + k * int4::kTile, std::true_type{});
          }
        }
        phase ^= 1u << stage;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
        __syncwarp();  // every lane has read the stage
        if (!dead) produce();
      }

      // ---- end of the piece
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], d);
#pragma unroll
            for (int u = 0; u < G; ++u) pm[nt][u][c] += __shfl_xor_sync(0xffffffffu, pm[nt][u][c], d);
          }
      const bool whole = count == n;
      // only the first piece of a range can be cut and not reach its end; at the end the ring is idle
      float* rec = rec_of[count < left ? 0 : 1];
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t + c;  // row of the row tile
          const float inv = l[nt][c] != 0.0f ? 1.0f / l[nt][c] : 0.0f;  // NaN stays NaN
#pragma unroll
          for (int u = 0; u < G; ++u) {
            const float even = 0x1p24f / F[nt][c], odd = 0x1p20f / F[nt][c];
            float y[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              y[2 * m] = fmaf(o[4 * u + m][nt][c], even, pm[nt][u][c]);
              y[2 * m + 1] = fmaf(o[4 * u + m][nt][c + 2], odd, pm[nt][u][c]);
            }
            if (whole) {
              if (row0 + r < p.rows) {
                const int tok = token_of(p, row0 + r);
                uint16_t* dst = p.out + ((static_cast<int64_t>(b) * p.q_len + tok) * p.num_heads +
                                         static_cast<int64_t>(head) * p.group + (row0 + r - tok * p.group)) * D + 64 * u + 8 * g;
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] *= inv;
                *reinterpret_cast<uint4*>(dst) = int4::pack8(y);
              }
            } else {
              float4* dst = reinterpret_cast<float4*>(rec + r * D + 64 * u + 8 * g);
              dst[0] = make_float4(y[0], y[1], y[2], y[3]);
              dst[1] = make_float4(y[4], y[5], y[6], y[7]);
            }
          }
          if (!whole && g == 0) {
            rec[C::kRows * D + 2 * r] = ref[nt][c];
            rec[C::kRows * D + 2 * r + 1] = l[nt][c];
          }
        }
      if (!whole && lane == 0) {
        Piece& pc = pieces[2 * warp + (rec == rec_of[1])];
        pc.start = pos - unit0;
        pc.units = n;
        pc.b = b;
        pc.seg = seg;
      }
      pos += count;
      left -= count;
      unit0 = 0;
      if (left > 0 && ++seg == segs) {
        seg = 0;
        len = next_len(p, b);
      }
    }
  }
  __syncthreads();

  // ---- merge what the ranges cut: over the CTA's warps, then over CTAs
  const int64_t cta_start = start_of(static_cast<int64_t>(blockIdx.x) * kWarps);
  const int64_t cta_end = start_of(static_cast<int64_t>(blockIdx.x + 1) * kWarps);
  auto record = [&](int i) {
    return reinterpret_cast<const float*>((i & 1) ? smem + (i / 2) * C::kRingBytes
                                                  : smem + kWarps * C::kRingBytes + (i / 2) * C::kRecBytes);
  };
  auto out_row = [&](int b, int seg, int r, bool& valid) {
    const int head = seg / p.n_rt, row = (seg - head * p.n_rt) * C::kRows + r;
    valid = row < p.rows;
    const int tok = token_of(p, row);
    return p.out + ((static_cast<int64_t>(b) * p.q_len + tok) * p.num_heads + static_cast<int64_t>(head) * p.group +
                    (row - tok * p.group)) * D;
  };
  const int64_t slot_floats = C::kRecFloats;
  int outward[2] = {-1, -1};  // pieces whose segment goes on in another CTA: started before, ends after
  for (int i = 0; i < 2 * kWarps;) {
    if (pieces[i].units == 0) {
      ++i;
      continue;
    }
    const Piece pc = pieces[i];
    uint32_t mine = 0;  // records of this segment
    int j = i;
    for (; j < 2 * kWarps && (pieces[j].units == 0 || pieces[j].start == pc.start); ++j)
      if (pieces[j].units != 0) mine |= 1u << j;
    const bool inside = pc.start >= cta_start && pc.start + pc.units <= cta_end;
    const int slot = pc.start < cta_start ? 0 : 1;
    if (!inside) outward[slot] = i;
    for (int r = warp; r < C::kRows; r += kWarps) {
      bool valid;
      uint16_t* dst = out_row(pc.b, pc.seg, r, valid);
      if (!valid) continue;
      float top = kNone;
      for (uint32_t m = mine; m; m &= m - 1) top = fmaxf(top, record(__ffs(m) - 1)[C::kRows * D + 2 * r]);
      float sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t m = mine; m; m &= m - 1) {
        const float* rec = record(__ffs(m) - 1);
        const float a = ptx::ex2(rec[C::kRows * D + 2 * r] - top);
        sum = fmaf(a, rec[C::kRows * D + 2 * r + 1], sum);
        if (lane < D / 4) {
          const float4 y = *reinterpret_cast<const float4*>(rec + r * D + 4 * lane);
          acc.x = fmaf(a, y.x, acc.x);
          acc.y = fmaf(a, y.y, acc.y);
          acc.z = fmaf(a, y.z, acc.z);
          acc.w = fmaf(a, y.w, acc.w);
        }
      }
      if (inside) {
        if (lane < D / 4) st_bf16x4(dst + 4 * lane, acc, sum != 0.0f ? 1.0f / sum : 0.0f);
      } else {
        float* ws = p.slots + (2 * static_cast<int64_t>(blockIdx.x) + slot) * slot_floats;
        if (lane < D / 4) __stcg(reinterpret_cast<float4*>(ws + r * D + 4 * lane), acc);
        if (lane == 0) __stcg(reinterpret_cast<float2*>(ws + C::kRows * D + 2 * r), make_float2(top, sum));
      }
    }
    i = j;
  }
  if (outward[0] < 0 && outward[1] < 0) return;  // (the same in every thread)
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {
    int last = 0;
    const int i = outward[threadIdx.x];
    if (i >= 0) {
      const Piece pc = pieces[i];
      const int first = static_cast<int>(owner_of(pc.start) / kWarps);
      const int ctas = static_cast<int>(owner_of(pc.start + pc.units - 1) / kWarps) - first + 1;
      last = atomicAdd(p.counters + first, 1) == ctas - 1;
    }
    last_of[threadIdx.x] = last;
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (!last_of[k]) continue;
    __threadfence();
    const Piece pc = pieces[outward[k]];
    const int first = static_cast<int>(owner_of(pc.start) / kWarps);
    const int last = static_cast<int>(owner_of(pc.start + pc.units - 1) / kWarps);
    if (threadIdx.x == 0) p.counters[first] = 0;
    for (int r = warp; r < C::kRows; r += kWarps) {
      bool valid;
      uint16_t* dst = out_row(pc.b, pc.seg, r, valid);
      if (!valid) continue;
      // the first CTA's part is its second slot, the others' their first
      auto part = [&](int c) { return p.slots + (2 * static_cast<int64_t>(c) + (c == first)) * slot_floats; };
      float top = kNone;
      for (int c = first + lane; c <= last; c += 32) top = fmaxf(top, __ldcg(part(c) + C::kRows * D + 2 * r));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int c = first; c <= last; ++c) {
        const float* ws = part(c);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(ws + C::kRows * D + 2 * r));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(ws + r * D + 4 * (lane % (D / 4))));
        const float a = ptx::ex2(ml.x - top);
        sum = fmaf(a, ml.y, sum);
        acc.x = fmaf(a, y.x, acc.x);
        acc.y = fmaf(a, y.y, acc.y);
        acc.z = fmaf(a, y.z, acc.z);
        acc.w = fmaf(a, y.w, acc.w);
      }
      if (lane < D / 4) st_bf16x4(dst + 4 * lane, acc, sum != 0.0f ? 1.0f / sum : 0.0f);
    }
  }
}

namespace {

template <int D, int NT>
Int4Plan plan_of() {
  using C = Cfg<D, NT>;
  return {NT, C::kCtas, static_cast<size_t>(C::kSmem), static_cast<size_t>(C::kRecFloats) * 2 * sizeof(float)};
}

template <int D, int NT>
cudaError_t launch(const Int4DecodeParams& p, int grid, cudaStream_t stream, bool overlap) {
  const auto kernel = decode_int4_kernel<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = Cfg<D, NT>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// 8 rows per segment while a kv head has no more than that, else 16.
Int4Plan plan_decode_int4(int head_dim, int rows) {
  if (head_dim == 64) return rows <= 8 ? plan_of<64, 1>() : plan_of<64, 2>();
  return rows <= 8 ? plan_of<128, 1>() : plan_of<128, 2>();
}

cudaError_t launch_decode_int4(const Int4DecodeParams& p, const Int4Plan& plan, int head_dim, int grid,
                               cudaStream_t stream, bool overlap) {
  if (head_dim == 64) return plan.n_tiles == 1 ? launch<64, 1>(p, grid, stream, overlap) : launch<64, 2>(p, grid, stream, overlap);
  return plan.n_tiles == 1 ? launch<128, 1>(p, grid, stream, overlap) : launch<128, 2>(p, grid, stream, overlap);
}

}  // namespace gqa
