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
// with c * 2^-24 stay normal in fp32.  Any finite q has such a power.  A score in the units of these products,
// the sum over g above times 2^(e - 24), is some 2^-9 |k|: the tensor core may drop what of the minima's part
// lies below 2^-126, which is 2^-126 scale log2(e) 2^(24 - e) < 2^-15 of a score while |scale q| < 2^100.
//   The minima's part of a score is one more MMA of depth 4 per tile, in tf32: m is exact there, and
// sum(q_g) goes in as two parts of 11 bits.
//   p s is rounded to fp16.  Steps may be of any size, so each row carries a power of two F for each group of V
// that keeps p s F below 2^15 (F is 2^115 at most, so steps below 2^-112 lose bits: 2^-25 / F = 2^-140 absolutely for
// each token's weight); they move with the running maximum, which itself moves only when a score
// passes it by 2^12.  (One F for both groups of a row would leave a group that is 2^-18 of the other, or less
// beside one token of great weight, in fp16's subnormals.)  Scores, sums and outputs are fp32.
//
// Bound: HBM at small groups on paper -- 9/8 D bytes per token and kv head -- but in fact the
// instructions that turn codes into MMA operands, whatever the number of query rows: about 315 per
// tile of 16 tokens and row tile, about half of them on the integer pipe at half rate, issued at 0.55 a cycle:
// what a warp waits for most is the latency of the one before.  4 sequences of 131072 tokens, 8 kv heads, 8 rows
// each: 130 us (4.6 TB/s, 71 % of a copy's rate), 107 with the copies alone.  256 sequences of 1 to 32768 tokens:
// 180 us (5.2 TB/s, 79 %).  More rows widen each tile again for every 16: 96 rows (64 sequences of 8192
// tokens, one kv head) 144 us, 0.18 PFLOP/s.  (Times here are of calls replayed in a graph.)
//
// Work.  The list of units (sequence, kv head, row tile, 32 tokens), in that order, is cut into one
// contiguous range of equal cost per WARP.  Each warp streams its range through its own ring of
// kStages units in shared memory (one bulk copy per tile of 16 tokens: K, V and parameters lie
// together), and keeps the running maximum, sum and output of its current segment in registers;
// there is no producer warp and no barrier in the loop.  The copies' cursor runs kStages units ahead;
// lane i holds the address of the i-th tile of a window of 32, so a unit costs no index arithmetic.
// (One producer warp for the CTA instead, with registers moved to the others, against the kernel of its
// time: 142 us for 135, and 42 for 36 on 32 sequences of 512 to 4096 tokens.)  A segment wholly inside a warp's range is written
// out at once.  What a range cuts is left in shared memory or the workspace (at most the first and the
// last segment of a warp), merged over the CTA's warps after one __syncthreads, and over CTAs through
// two workspace slots per CTA: the warp that is last to arrive at the counter of a segment's two rows
// merges those.  (With a barrier of the CTA and one counter a segment, then: 33.4 us for 31.8 on that batch.)
// Which order the CTAs arrive in changes nothing: the parts are summed in the order of the list.
//
// The S tile is computed transposed, S^T = K Q^T (tokens on the MMA's 16-row side, 8 query
// rows on the other), so a group of 4 or 8 heads needs no padding to 16.
//
// Safety: every wait is bounded; a warp whose wait runs out sets the error word, treats the rest
// of its range as masked, drains its own copies (bounded) and still takes part in the merges, so
// no counter is left behind.  Page ids and lengths are range-checked before use.
#include <atomic>
#include <type_traits>

#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

namespace {

constexpr int kWarps = 8;
static_assert((2 * kWarps & (2 * kWarps - 1)) == 0 && 2 * kWarps <= 32, "a lane per piece of the CTA");
constexpr float kNone = -3.0e38f;   // reference of a row that has seen no token

// Rows of a merge, and records whose rows are loaded at a time (what a merge waits for is the way to L2,
// but each costs its instructions where there are fewer): 32 sequences of 512 to 4096 tokens take 32.8 us
// with (2, 5), 32.7 with (2, 4), 32.6 with (2, 2), 34.0 with (1, 4); with four query tokens 49.9, 49.6, 48.3,
// 55.5; 4 of 131072 130.2, 130.5, 130.5, 134.3; 64 of 8192 with 96 heads 144.3, 144.1, 143.5, 152.9; one of 131072
// beside 20 of 2000, one kv head, 30.2, 30.8, 34.8 with (2, 2).
constexpr int kMergeRows = 2, kFlight = 5;

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;              // query rows of a segment
  static constexpr int kGroups = D / 64;
  static constexpr int kTileBytes = 18 * D;
  static constexpr int kUnitBytes = 2 * kTileBytes;
  static constexpr int kStages = 3;
  static constexpr int kCtas = NT == 1 ? 2 : 1;     // per SM
  static constexpr int kCounters = kRows / kMergeRows;  // of a CTA
  static constexpr int kRecFloats = kRows * (D + 2);  // a piece: [rows][D], then (reference, sum)
  static constexpr int kRingBytes = kStages * kUnitBytes;
  static_assert(kRingBytes >= kRecFloats * 4, "the last piece of a warp is left in its ring");
  // Where a piece that a range cuts at the front is left: in shared memory if there is room beside the
  // rings (one CTA per SM), else in the workspace.
  static constexpr bool kRecHere = NT > 1;
  static constexpr int kRecBytes = (kRecFloats * 4 + 127) / 128 * 128;
  static constexpr int kSmem = kWarps * (kRingBytes + (kRecHere ? kRecBytes : 0));
};

// A piece that a warp's range cut off.
struct Piece {
  int64_t start;  // position of the segment's first unit in the list
  int units;      // of the segment; 0: no piece
  int b, seg;     // sequence and segment in it
};

constexpr int kUnit = 2 * int4::kTile;  // tokens per step of a warp

// What a segment costs a warp beside its units, in units: fetching q, ending and leaving a piece.
// The list is cut by it, since some warps get dozens of short sequences: 256 sequences of 1 to 32768
// tokens take 187 us with 2, 180 with 3, 181 with 4 (266 with 0 and 208 with 1 in an earlier state); a batch of 32
// of 512 to 4096 tokens 33.5, 32.8, 32.8, and with four query tokens 50.1, 49.9, 47.1.
constexpr int kSegCost = 3;

__device__ __forceinline__ int units_of(int len) {
  return static_cast<int>((static_cast<unsigned>(len) + (kUnit - 1)) / kUnit);  // (len may be near 2^31)
}
// Whether a sequence of len tokens has a tile of this number.
__device__ __forceinline__ bool has_tile(int tile, int len) {
  return static_cast<unsigned>(tile) * int4::kTile < static_cast<unsigned>(len);
}
__device__ __forceinline__ int cost_of(int len) { return len > 0 ? units_of(len) + kSegCost : 0; }

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

// a / b, both not negative; in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// How the list of `total` units is cut: the first `rem` workers take per + 1 units, the others per.
struct Split {
  int64_t total, workers, per, rem;
  __device__ __forceinline__ int64_t start(int64_t w) const { return w >= workers ? total : w * per + min(w, rem); }
  __device__ __forceinline__ int64_t owner(int64_t unit) const {
    const int64_t cut = rem * (per + 1);
    return unit < cut ? quotient(unit, per + 1) : rem + quotient(unit - cut, per);
  }
};

// The query token of row r of a kv head.
__device__ __forceinline__ int token_of(const Int4DecodeParams& p, int r) { return p.q_len == 1 ? 0 : r / p.group; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ void st_bf16x4(uint16_t* dst, const float4& o, float inv) {
  uint2 w;
  w.x = ptx::pack_bf16x2(o.x * inv, o.y * inv);
  w.y = ptx::pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(dst) = w;
}

// 2^-floor(log2 m) for finite m, between 2^-126 and 2^115 (which 0 gives, too).  Not more: times a weight of up to
// 2^12, before it meets a step that may be 0, it has to be finite.
__device__ __forceinline__ float inverse_pow2(float m) {
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;  // (a subnormal counts as 2^-127)
  e = max(-115, min(126, e));
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
  __shared__ int64_t excl[32 * kWarps];  // cost of the sequences before each thread's chunk
  __shared__ int64_t scan[kWarps];
  __shared__ int longest[kWarps];
  __shared__ __align__(8) uint64_t full[kWarps][C::kStages];
  __shared__ Piece pieces[2 * kWarps];
  __shared__ Split kept;  // for the merges: the loop has no registers for it

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  unsigned char* ring = smem + warp * C::kRingBytes;
  // A warp's pieces: one cut at the end stays in its ring, which is idle by then.
  auto record = [&](int i) {
    if (i & 1) return reinterpret_cast<float*>(smem + (i / 2) * C::kRingBytes);
    if (C::kRecHere) return reinterpret_cast<float*>(smem + kWarps * C::kRingBytes + (i / 2) * C::kRecBytes);
    return p.slots + (2 * static_cast<int64_t>(gridDim.x) + static_cast<int64_t>(blockIdx.x) * kWarps + i / 2) * C::kRecFloats;
  };

  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) ptx::mbar_init(ptx::smem_u32(&full[warp][s]), 2);  // the lanes of a unit's two tiles
    ptx::fence_mbarrier_init();
    pieces[2 * warp].units = 0;
    pieces[2 * warp + 1].units = 0;
  }

  // ---- the split: cost before each thread's chunk of sequences
  const int segs = p.num_kv_heads * p.n_rt;  // segments per sequence
  const int chunk = (p.num_seqs + 32 * kWarps - 1) / (32 * kWarps);
  {
    int64_t mine = 0;
    int most = 0;
    const int b0 = threadIdx.x * chunk, b1 = min(p.num_seqs, b0 + chunk);
    for (int b = b0; b < b1; ++b) {
      const int cost = cost_of(checked_len(p, b));
      mine += cost;
      most = max(most, cost);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) {
      scan[warp] = incl;
      longest[warp] = most;
    }
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += scan[w];
    excl[threadIdx.x] = before + incl - mine;
    __syncthreads();
  }
  Split split;
  {
    int64_t total = 0;
    int most = 0;
    for (int w = 0; w < kWarps; ++w) {
      total += scan[w];
      most = max(most, longest[w]);
    }
    split.total = total * segs;
    // Least work of a warp.  Few long segments are not cut into more than is merged in the time that it
    // saves: a unit takes 0.8 us, a warp merges eight CTAs' parts of a segment in 1 us, and n units a
    // segment in ranges of x make n / 8 x parts: x = sqrt(n / 52).  The longest segment's n, since segments
    // are merged side by side; sequences without tokens do not count.  (One sequence of 131072 tokens and one
    // kv head: 29 us, and 57 cut as finely as there are warps; three of 30000 19 and 31.)  A batch of a few
    // units is not cut finer than a segment of one: two sequences of 17 and 40 tokens take 6.2 us whole
    // and 7.9 cut.
    int64_t least = static_cast<int64_t>(sqrtf(static_cast<float>(most) * (1.0f / 52.0f)));
    least = max(least, split.total <= 4 * kWarps ? int64_t{kSegCost + 1} : int64_t{1});
    split.workers = min(static_cast<int64_t>(gridDim.x) * kWarps, quotient(split.total + least - 1, least));
    split.per = split.total == 0 ? 0 : quotient(split.total, split.workers);
    split.rem = split.total - split.per * split.workers;
    if (threadIdx.x == 0) kept = split;
  }
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  int64_t pos = split.start(me);
  const int64_t end = split.start(me + 1);

  ptx::pdl_wait_prerequisites();  // q and the pool may be written by the preceding append

  if (pos < end) {
    // ---- find the first unit: the chunk, then the sequence in it
    const int64_t unit = quotient(pos, segs);  // in units of a sequence's one segment
    int ci = 0;
    for (int i = 0; i < kWarps; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, excl[32 * i + lane] <= unit);
      ci += __popc(m);
    }
    int b = (ci - 1) * chunk, len = 0;
    int64_t base = excl[ci - 1];
    if (chunk == 1) {
      len = checked_len(p, b);
    } else {
      for (;; b += 32) {
        const int mine = b + lane < p.num_seqs ? checked_len(p, b + lane) : 0;
        int64_t incl = cost_of(mine);
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
          base += __shfl_sync(0xffffffffu, incl, at) - cost_of(len);
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
        if (b + 32 >= p.num_seqs) break;  // only if the lengths changed under the call
      }
    }
    // The position lies in segment seg's own cost (then its first unit is the next) or is a unit of it.
    int seg = static_cast<int>(quotient(pos - base * segs, max(1, cost_of(len))));
    const int into = static_cast<int>(pos - base * segs - static_cast<int64_t>(seg) * cost_of(len));
    int unit0 = max(0, into - kSegCost);
    int64_t first = pos - into + kSegCost;  // the position of the segment's first unit
    // positions from unit0 to the end of the range
    int left = len == 0 ? 0 : static_cast<int>(min(end - first - unit0, int64_t{INT32_MAX}));

    // ---- the copies' cursor runs kStages units ahead of the arithmetic's.  Lane i holds the address
    // of tile win + i of the cursor's segment (0: none) and issues that tile's copy itself.
    int pb = b, phead = seg / p.n_rt, prt = seg - phead * p.n_rt, plen = len, pleft = left;
    int punits = units_of(len) - unit0;  // units of the segment not issued yet
    int win = 2 * unit0, in_win = 16;    // the window's first tile; its next unit (16: past it)
    int ahead = -1;                      // this lane's page of the next window
    uint32_t bad = 0;                    // two bits per stage: no data behind the tile
    uint64_t addr = 0;
    const uint32_t ring_at = ptx::smem_u32(ring) + (lane & 1) * C::kTileBytes, bar_at = ptx::smem_u32(&full[warp][0]);
    auto page_of = [&](int tile) {
      const int block = p.tpp_magic != 0 ? fast_div(tile, p.tpp_magic, p.tpp_shift) : tile;
      return has_tile(tile, plen) ? __ldg(p.block_table + static_cast<int64_t>(pb) * p.max_blocks + block) : -1;
    };
    auto produce = [&](int pstage) {  // into the stage that is free
      if (pleft <= 0) return;
      if (in_win == 16) {  // the next 32 tiles
        const int tile = win + lane;
        const int block = p.tpp_magic != 0 ? fast_div(tile, p.tpp_magic, p.tpp_shift) : tile;
        const int page = ahead;
        const bool wanted = has_tile(tile, plen);
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
        const uint32_t at = (static_cast<uint32_t>(page) * p.num_kv_heads + phead) * p.tiles_per_page +
                            (tile - block * p.tiles_per_page);
        addr = ok && wanted ? reinterpret_cast<uint64_t>(p.pool) + static_cast<uint64_t>(at) * C::kTileBytes : 0;
        // (only tiles of this warp's range are its to report)
        if (wanted && !ok && lane < 2 * min(pleft, 16)) atomicOr(p.err, kErrBounds);
        in_win = 0;
        win += 32;
        ahead = page_of(win + lane);
      }
      const uint32_t here = __ballot_sync(0xffffffffu, addr != 0) >> (2 * in_win);
      bad = (bad & ~(3u << (2 * pstage))) | ((~here & 3u) << (2 * pstage));
      if ((lane >> 1) == in_win) {
        const uint32_t bar = bar_at + 8 * pstage;
        if (addr != 0) {
          ptx::mbar_arrive_expect_tx(bar, C::kTileBytes);
          if (!p.arm_without_copy)
            ptx::bulk_load(ring_at + pstage * C::kUnitBytes, reinterpret_cast<const void*>(addr), C::kTileBytes, bar);
        } else {
          ptx::mbar_arrive(bar);
        }
      }
      ++in_win;
      --pleft;
      if (--punits == 0) {  // the next segment
        pleft -= kSegCost;
        if (++prt == p.n_rt) {
          prt = 0;
          if (++phead == p.num_kv_heads) {
            phead = 0;
            if (pleft > 0) plen = next_len(p, pb);
          }
        }
        punits = units_of(plen);
        win = 0;
        in_win = 16;
        if (pleft > 0) ahead = page_of(lane);
      }
    };
    ahead = page_of(win + lane);
    __syncwarp();
    for (int s = 0; s < C::kStages; ++s) produce(s);

    // this lane's places in a tile
    const uint32_t at_k = g * (D / 2) + t * (D / 8), at_par = L4::kParams + g * (8 * G);
    const uint32_t at_v = L4::kVCodes + (g / (8 / G)) * 512 + t * 32 + (g % (8 / G)) * (4 * G);
    const uint32_t ring0 = ptx::smem_u32(ring);
    int stage = 0;
    uint32_t parity = 0;
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
#pragma unroll
          for (int e = 0; e < 8; ++e) top = int4::max_nan(top, fabsf(x[i][e]));
        }
        top = int4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = int4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // up = 2^e with top * 2^e in [2^14, 2^15), for every finite top down to 2^-112 (a smaller one, a multiple
        // of bf16's least number, is exact all the same).  The sums are taken after it: they stay finite.
        const int top_e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const int e = min(126, 14 - top_e);  // -114 (not finite) and above
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
          if (i % 2 == 0) sum[i / 2] = 0.0f;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            x[i][c] *= up;
            sum[i / 2] += x[i][c];
          }
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
          sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 1);
          sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 2);
        }
        // scale log2(e) 2^(24 - e); the power in two factors, as it may pass fp32's range where the product does not
        const int e0 = (24 - e) >> 1, e1 = 24 - e - e0;
        float down = p.scale * __uint_as_float(static_cast<uint32_t>(127 + e0) << 23) * 1.4426950408889634f *
                     __uint_as_float(static_cast<uint32_t>(127 + e1) << 23);
        if (!(top < INFINITY)) down = __uint_as_float(0x7fffffffu);  // the row is NaN
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
          const float* y = x[i];
          qf[nt][2 * i][0] = ptx::pack_f16x2(y[0], y[4]);
          qf[nt][2 * i][1] = ptx::pack_f16x2(y[1] * 0.0625f, y[5] * 0.0625f);
          qf[nt][2 * i + 1][0] = ptx::pack_f16x2(y[2], y[6]);
          qf[nt][2 * i + 1][1] = ptx::pack_f16x2(y[3] * 0.0625f, y[7] * 0.0625f);
        }
        // The sum of q in the units of the codes' products, cut into two parts of 11 bits, which
        // tf32 holds exactly: the minima (bf16) times them lose 2^-22 at most.
        const float mine = (G == 2 && (t & 1) ? sum[G - 1] : sum[0]) * 0x1p-24f;
        const float upper = __uint_as_float(__float_as_uint(mine) & 0xffffe000u);
        const float lower = __uint_as_float(__float_as_uint(mine - upper) & 0xffffe000u);
        qsum[nt] = __float_as_uint(t / G == 0 ? upper : (t / G == 1 ? lower : 0.0f));
        // this thread's score columns are rows 2 t and 2 t + 1 of the row tile
#pragma unroll
        for (int c = 0; c < 2; ++c) h[nt][c] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * c);
      }

      float o[G * 4][NT][4], l[NT][2], pm[NT][G][2], ref[NT][2], F[NT][G][2];
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
#pragma unroll
          for (int u = 0; u < G; ++u) {
            pm[nt][u][c] = 0.0f;
            F[nt][u][c] = 1.0f;
          }
        }
      }

      // One tile whose first token is tok0.  ENDS: some row's window ends in it.
      auto attend = [&](uint32_t at, int tok0, auto ends_tag) {
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
          const uint4 a = ptx::lds128(at + at_k), c = ptx::lds128(at + at_k + 8 * 64);
          ka[0] = a.x; ka[1] = a.y; ka[2 * G - 2] = a.z; ka[2 * G - 1] = a.w;
          kb[0] = c.x; kb[1] = c.y; kb[2 * G - 2] = c.z; kb[2 * G - 1] = c.w;
          const uint4 pa = ptx::lds128(at + at_par), pc = ptx::lds128(at + at_par + 8 * 16);
          par[0][0] = pa.x; par[0][1] = pa.y; par[0][2 * G - 2] = pa.z; par[0][2 * G - 1] = pa.w;
          par[1][0] = pc.x; par[1][1] = pc.y; par[1][2 * G - 2] = pc.z; par[1][2 * G - 1] = pc.w;
        } else {
          const uint2 a = ptx::lds64(at + at_k), c = ptx::lds64(at + at_k + 8 * 32);
          ka[0] = a.x; ka[1] = a.y;
          kb[0] = c.x; kb[1] = c.y;
          const uint2 pa = ptx::lds64(at + at_par), pc = ptx::lds64(at + at_par + 8 * 8);
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
        // ---- weights; the reference moves only when a score passes it by 12 (in units of log2)
        // (not in packed pairs: the compiler may contract a packed product and difference, and a score
        // has to be the same number here and where the reference is taken from it)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[nt][x] = __fmul_rn(sc[nt][x], h[nt][x % 2]);
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
#pragma unroll
              for (int u = 0; u < G; ++u) {
                ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(pr[nt][2 * r], pr[nt][2 * r + 1]), ptx::f2_pack(F[nt][u][0], F[nt][u][1])), y[0], y[1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  w[nt][u][2 * r + c] = y[c] * step[r][u];
                  if (ENDS && !seen[nt][2 * r + c]) w[nt][u][2 * r + c] = 0.0f;
                }
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
          up = top > 4096.0f || big > 32768.0f;
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
#pragma unroll
              for (int u = 0; u < G; ++u) {
                pm[nt][u][c] *= a;
                float big = 0.0f;
                if (seen[nt][c]) big = fmaxf(big, ptx::ex2(at0 - top) * step[0][u]);
                if (seen[nt][c + 2]) big = fmaxf(big, ptx::ex2(at1 - top) * step[1][u]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
                // the largest weight so far in [2^2, 2^3): 2^12 below the bound, as far as scores may pass
                // the reference, and 2^16 above fp16's subnormals
                const float before = a / F[nt][u][c];
                const float f = inverse_pow2(fmaxf(big * 0x1p-2f, before));
                const float scale = before * f;
                F[nt][u][c] = f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  o[4 * u + m][nt][c] *= scale;
                  o[4 * u + m][nt][c + 2] *= scale;
                }
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
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (G == 2) {
            const uint2 a = ptx::lds64(at + at_v + q * 128);
            v[q][0] = a.x;
            v[q][G - 1] = a.y;
          } else {
            v[q][0] = ptx::lds32(at + at_v + q * 128);
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

      // units whose tokens every row sees
      const int open = max(0, len - p.q_len + 1) / kUnit - unit0;
      for (int i = 0; i < count && !dead; ++i) {
        const bool landed = ptx::mbar_wait_bounded(bar_at + 8 * stage, parity, p.wait_limit_ns);
        if (!__all_sync(0xffffffffu, landed)) {
          dead = true;
          if (lane == 0) atomicOr(p.err, kErrTimeout);
          if (!p.arm_without_copy) {  // nothing may still be landing when the ring is written or given up
            // (a stage that nothing was sent to is waited for in vain)
#pragma unroll 1
            for (int k = 0; k < C::kStages; ++k) {
              ptx::mbar_wait_bounded(bar_at + 8 * stage, parity, p.wait_limit_ns);
              if (++stage == C::kStages) stage = 0, parity ^= 1;
            }
          }
          __syncwarp();
          break;
        }
        const uint32_t at = ring0 + stage * C::kUnitBytes;
        const int tok0 = (unit0 + i) * kUnit;
        const uint32_t lost = (bad >> (2 * stage)) & 3u;
        if (lost == 0 && i < open) {
#pragma unroll 1
          for (int k = 0; k < 2; ++k) attend(at + k * C::kTileBytes, tok0 + k * int4::kTile, std::false_type{});
        } else {
#pragma unroll 1
          for (int k = 0; k < 2; ++k)
            if ((lost >> k & 1u) == 0) attend(at + k * C::kTileBytes, tok0 + k * int4::kTile, std::true_type{});
        }
        __syncwarp();  // every lane has read the stage
        produce(stage);
        if (++stage == C::kStages) stage = 0, parity ^= 1;
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
      // only the first piece of a range can be cut and not reach its end
      const int which = 2 * warp + (count < left ? 0 : 1);
      float* rec = record(which);
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = nt * 8 + 2 * t + c;  // row of the row tile
          const float inv = l[nt][c] != 0.0f ? 1.0f / l[nt][c] : 0.0f;  // NaN stays NaN
#pragma unroll
          for (int u = 0; u < G; ++u) {
            // 1 / F: a power of two in [2^-115, 2^126], so it does not take the codes' 2^24 as well
            const float over = __uint_as_float((254u << 23) - __float_as_uint(F[nt][u][c]));
            float y[8];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              y[2 * m] = fmaf(o[4 * u + m][nt][c] * 0x1p24f, over, pm[nt][u][c]);
              y[2 * m + 1] = fmaf(o[4 * u + m][nt][c + 2] * 0x1p20f, over, pm[nt][u][c]);
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
        Piece& pc = pieces[which];
        pc.start = first;
        pc.units = n;
        pc.b = b;
        pc.seg = seg;
      }
      first += n + kSegCost;
      left -= count + kSegCost;
      unit0 = 0;
      if (left > 0 && ++seg == segs) {
        seg = 0;
        len = next_len(p, b);
      }
    }
  }
  // Rows of sequences without a token (a length out of range counts as none and is reported).
  for (int64_t b = me; b < p.num_seqs; b += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int raw = __ldg(p.seq_lens + b);
    if (checked_len(p, static_cast<int>(b)) != 0) continue;
    if (raw != 0 && lane == 0) atomicOr(p.err, kErrBounds);
    uint4* o = reinterpret_cast<uint4*>(p.out + b * p.q_len * p.num_heads * D);
    for (int i = lane; i < p.q_len * p.num_heads * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
  }

  __syncthreads();

  // ---- merge what the ranges cut: over the CTA's warps, then over CTAs
  const int64_t cta_start = kept.start(static_cast<int64_t>(blockIdx.x) * kWarps);
  const int64_t cta_end = kept.start(static_cast<int64_t>(blockIdx.x + 1) * kWarps);
  auto out_row = [&](int b, int seg, int r) -> uint16_t* {
    const int head = seg / p.n_rt, row = (seg - head * p.n_rt) * C::kRows + r;
    if (row >= p.rows) return nullptr;
    const int tok = token_of(p, row);
    return p.out + ((static_cast<int64_t>(b) * p.q_len + tok) * p.num_heads + static_cast<int64_t>(head) * p.group +
                    (row - tok * p.group)) * D;
  };
  constexpr int kMl = C::kRows * D;  // (reference, sum) of the rows, behind the rows
  const int col = 4 * (lane % (D / 4));
  constexpr int MR = kMergeRows;
  // Merges rows r0 .. r0 + MR - 1 (of `rows`) of a segment's records -- record_of(i), i < count, of the
  // first 16 only those with bit i of `some` set -- into their output rows, or into the rows of `into`.
  // Lane i looks after record i % 16 of 16, of row r0 + i / 16.
  auto merge = [&](int b, int seg, int r0, int rows, int count, uint32_t some, auto record_of, auto load2, auto load4, float* into) {
    float top = kNone, sum = 0.0f;
    float4 acc[MR];
#pragma unroll
    for (int k = 0; k < MR; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int my_row = r0 + lane / 16;
#pragma unroll 1
    for (int c = 0; c < count; c += 16) {
      const int i0 = lane & 15;
      const bool mine = c + i0 < count && (some >> i0 & 1);
      float2 ml = make_float2(kNone, 0.0f);
      if (mine && my_row < rows) ml = load2(record_of(c + i0) + kMl + 2 * my_row);
      uint32_t todo = __ballot_sync(0xffffffffu, mine) & 0xffffu;
      float a = 0.0f;
      bool weighed = false;
#pragma unroll 1
      while (todo) {
        float4 y[kFlight][MR];
        int from[kFlight];
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
          from[q] = todo ? __ffs(todo) - 1 : -1;
          todo &= todo - 1;
          const float* rec = record_of(c + max(0, from[q])) + r0 * D + col;
#pragma unroll
          for (int k = 0; k < MR; ++k) {
            y[q][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from[q] >= 0 && (k == 0 || r0 + k < rows)) y[q][k] = load4(rec + k * D);
          }
        }
        if (!weighed) {  // (after the first loads are on their way)
          weighed = true;
          float now = fmaxf(top, ml.x);
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
          const float before = ptx::ex2(top - now);
          a = ptx::ex2(ml.x - now);
          top = now;
          float part = a * ml.y;
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
          sum = fmaf(sum, before, part);
#pragma unroll
          for (int k = 0; k < MR; ++k) {
            const float f = __shfl_sync(0xffffffffu, before, 16 * k);
            acc[k].x *= f;
            acc[k].y *= f;
            acc[k].z *= f;
            acc[k].w *= f;
          }
        }
#pragma unroll
        for (int q = 0; q < kFlight; ++q)
#pragma unroll
          for (int k = 0; k < MR; ++k) {
            float w = __shfl_sync(0xffffffffu, a, 16 * k + max(0, from[q]));
            if (from[q] < 0) w = 0.0f;
            acc[k].x = fmaf(w, y[q][k].x, acc[k].x);
            acc[k].y = fmaf(w, y[q][k].y, acc[k].y);
            acc[k].z = fmaf(w, y[q][k].z, acc[k].z);
            acc[k].w = fmaf(w, y[q][k].w, acc[k].w);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < MR; ++k) {
      const float t = __shfl_sync(0xffffffffu, top, 16 * k);
      const float l = __shfl_sync(0xffffffffu, sum, 16 * k);
      if (k > 0 && r0 + k >= rows) break;
      if (into == nullptr) {
        if (lane < D / 4) st_bf16x4(out_row(b, seg, r0 + k) + col, acc[k], l != 0.0f ? 1.0f / l : 0.0f);
      } else {
        if (lane < D / 4) *reinterpret_cast<float4*>(into + (r0 + k) * D + col) = acc[k];
        if (lane == 0) *reinterpret_cast<float2*>(into + kMl + 2 * (r0 + k)) = make_float2(t, l);
      }
    }
  };
  // rows of the segment's row tile
  auto rows_of = [&](int seg) { return min(C::kRows, p.rows - seg % p.n_rt * C::kRows); };

  // Lane i looks after piece i; (segment, MR rows) go to the warps in turn: first what the CTA has of the
  // rows, then, where the segment goes on in other CTAs, the arrival at their counter.  The last CTA's warp to
  // arrive merges those rows' parts, so no warp waits for another, nor for other rows.
  const int64_t its_start = lane < 2 * kWarps ? pieces[lane].start : 0;
  uint32_t todo = __ballot_sync(0xffffffffu, lane < 2 * kWarps && pieces[lane & (2 * kWarps - 1)].units != 0);
  int turn = MR * warp;
#pragma unroll 1
  while (todo) {
    const int i = __ffs(todo) - 1;
    const Piece pc = pieces[i];
    const uint32_t mine = todo & __ballot_sync(0xffffffffu, its_start == pc.start);
    todo &= ~mine;
    const bool inside = pc.start >= cta_start && pc.start + pc.units <= cta_end;
    const int slot = pc.start < cta_start ? 0 : 1;  // it started in an earlier CTA; it goes on in a later one
    float* into = inside ? nullptr : p.slots + (2 * static_cast<int64_t>(blockIdx.x) + slot) * C::kRecFloats;
    const int rows = rows_of(pc.seg);
#pragma unroll 1
    for (; turn < rows; turn += MR * kWarps) {
      merge(pc.b, pc.seg, turn, rows, 2 * kWarps, mine, record, [](const float* x) { return *reinterpret_cast<const float2*>(x); },
            [](const float* x) { return *reinterpret_cast<const float4*>(x); }, into);
      if (inside) continue;
      const int from = static_cast<int>(kept.owner(pc.start) / kWarps);
      const int to = static_cast<int>(kept.owner(pc.start + pc.units - 1) / kWarps);
      int32_t* counter = p.counters + from * C::kCounters + turn / MR;
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(counter, 1) == to - from;
      if (__shfl_sync(0xffffffffu, last, 0) == 0) continue;
      __threadfence();
      if (lane == 0) *counter = 0;
      // the first CTA's part is its second slot, the others' their first
      merge(pc.b, pc.seg, turn, rows, to - from + 1, 0xffffu,
            [&](int c) { return p.slots + (2 * static_cast<int64_t>(from + c) + (c == 0)) * C::kRecFloats; },
            [](const float* x) { return __ldcg(reinterpret_cast<const float2*>(x)); },
            [](const float* x) { return __ldcg(reinterpret_cast<const float4*>(x)); }, nullptr);
    }
    turn -= (rows + MR - 1) / MR * MR;
  }
}

namespace {

template <int D, int NT>
Int4Plan plan_of() {
  using C = Cfg<D, NT>;
  return {NT, kWarps, C::kCtas, static_cast<size_t>(C::kRecFloats) * (C::kRecHere ? 2 : 2 + kWarps) * sizeof(float),
          kInt4Counters / C::kCounters};
}

template <int D, int NT>
cudaError_t launch(const Int4DecodeParams& p, int grid, cudaStream_t stream, bool overlap) {
  const auto kernel = decode_int4_kernel<D, NT>;
  // the attribute is kept per device: set by the first call on each
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || (set.load(std::memory_order_relaxed) >> dev & 1) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  }
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

// 8 rows per segment while a kv head has no more than that, else 16, which widen each tile once for both
// halves but leave registers for half the warps: a kv head with 16 rows (32 sequences of 512 to 4096
// tokens, four query tokens) takes 50 us with 16 and 55 with 8; one with 96 (64 of 8192 tokens) 144 and
// 189 us, and 154 (then) with 24 rows a segment, whose output no longer fits the registers.
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
