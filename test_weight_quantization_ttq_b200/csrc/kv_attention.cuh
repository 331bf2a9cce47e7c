// Attention of a few new tokens per sequence over the quantised paged cache
// (ttq_kv_attention).
//
//   t_j = scale <q, K_j>  (capped: cap tanh(t_j / cap));  y = sum_j softmax(t)_j V_j
// with K_j = s (c - z) D_k^{-1/2} per group of channels, V_j likewise.
//
// Work.  The rows of one key/value head (its query heads x the sequence's
// new tokens) form tiles of 8 NT rows, or of 256 where there are many
// (kv_attention_wide.cuh); a segment is one (sequence, head,
// tile) with all blocks of 16 tokens that it may see.  All segments'
// blocks, laid end to end, are cut into equal runs, one per thread block of
// the grid, so that contexts of any lengths load the SMs evenly.  The warps
// of a block share out its part of a segment, keep softmax states of their
// own and merge them at its end.  Of a segment that several runs share each
// leaves a partial result (offset, sum and accumulator) in the
// workspace, and the one whose ticket is the segment's last merges them in
// their order, so that the result does not depend on who is last; where
// there are many, groups of them are merged before the whole.
// (One run per warp, with no barrier between warps, was measured too: it
// left every cut to a single warp's merge, 6 us at 2 to 9 results, and took
// 97 us where this takes 87 for 64 contexts of up to 8192.)
//
// A warp brings its blocks through a ring of shared memory stages by bulk
// copies, one per block (codes and pairs of K and V are contiguous).
// Products are m16n8k16 with the codes as the A operand:
//   S^T [16 tokens x 8 rows] = (c - z)_K Q^T   per group of channels, scaled
//       by the token's s_K in fp32;
//   O^T [channels x 8 rows] += (c - z)_V^T (p s_V)^T.
// An INT field's code c is taken where it stands: masked out of its word and
// put under an exponent whose unit it counts, it reads as 1024 + c, 256 + c,
// 64 + c or 16 + c, and those above 64 are brought down to 64 or 16 (exact).
// The offsets and zeros are taken off the sums instead of every element:
// S - sum(offset q) - z sum(q) with the sums of q formed once per segment,
// and for the second product sum(p s (offset + z)), one more accumulator per
// group with offset + z as the operand.  (Codes read as subnormals would
// need neither offset nor exponent, but the matrix instruction aligns its
// sums by the operands' exponents and keeps some 8 bits less of those: errors
// of 2^-15 of the raw sums, measured.)  With more than 8 rows those
// accumulators would not fit the registers; there V's operand is c - z itself.
// p s_V moves from the accumulator layout (tokens along the lanes' rows) to
// the B operand's by an 8 x 8 transposition within the warp.
//
// Numerics.  Each row of q (times D_k^{-1/2}) is scaled by a power of two to
// [1, 2) and rounded to binary16, or to a sum of two (QP).  Scores t (in
// powers of two), the row's offset and the sum l are fp32.  What is rounded to
// binary16 is p s_V, so the offset in p = 2^(t - offset) is not the largest
// score but the largest t + e of the tokens that the row sees, 2^e the power of
// two in the token's largest scale of V (its groups share it): p s_V of the
// weightiest token is near 1, whatever the scales are, and a token that the row
// does not see, or that has no probability, takes no bits from the others.
// The offset moves only when a t + e exceeds it by more than 8, which keeps
// p s_V below 2^9; products under 2^-14 are binary16's subnormal numbers.
#pragma once

#include <atomic>
#include <type_traits>

#include "kv_device.cuh"
#include "ttq_kernels.h"

namespace ttq {

constexpr float kKvLog2e = 1.4426950408889634f;
constexpr float kKvFloor = -3.4e38f;  // a row's offset before any score
constexpr float kKvSlack = 8.f;
constexpr float kKvLeastScale = 5.9604645e-08f;   // 2^-24, binary16's least: what a token without a scale counts for

// The exponent of a positive float: the integer put under 2^23's exponent, which counts it.
__device__ __forceinline__ float kv_exponent(float x) {
  return __uint_as_float(__float_as_uint(x) >> 23 | 0x4B000000u) - 8388735.f;   // 2^23 + 127
}

// QP: the binary16 numbers that an element of Q is taken as, 1 or 2 (kv_api.cu
// says when).  Two are two sets of fragments, whose products add to the same
// scores.
template <int HD, int BITS, int NG, int NT, int QP>
struct KvAttention {
  using F = KvFormat<HD, BITS, NG>;
  static constexpr int W = kKvAttentionWarps;       // warps of a block
  static constexpr int ROWS = 8 * NT;               // query rows of a tile
  static constexpr int KS = HD / 16;                // k steps of the first product
  static constexpr int MT = HD / 16;                // m tiles of the second
  static constexpr int FRAGS = NT * KS * 32 * 8;    // fragments of one part of the tile's Q
  static constexpr int QPART = FRAGS + ROWS * 8 * NG;   // with the sums of its groups
  static constexpr int QFRAG = QP * QPART;
  static constexpr int ROWINFO = ROWS * 16;         // what is known of the rows
  static constexpr int LDO = HD + 4;                // padded row of the accumulators in shared memory
  static constexpr int TILE = ROWS * LDO * 4;       // their bytes
  // whether V's codes are taken raw and their zeros off the sums (see above)
  static constexpr bool VRAW = BITS != 8 && NT == 1 && NG <= 2;
  // what even and odd fields of a half word are offset by
  static constexpr uint32_t EVEN = 0x54005400u, ODD = BITS == 4 ? 0x54005400u : 0x4C004C00u;   // 64; 64 or 16
  // Blocks of threads per SM: by registers 4 where a thread's HD NT / 4
  // accumulators are at most 32 (128 registers), 3 for 64 (168), else 2; fewer
  // where their rings would not have two stages.
  static constexpr int SM_BYTES = 212 * 1024;
  static constexpr int room(int ctas) { return (SM_BYTES / ctas - QFRAG - ROWINFO - 2048) / W; }
  static constexpr int fits(int ctas) { return room(ctas) >= 2 * F::BLOCK && room(ctas) >= TILE; }
  static constexpr int BY_REGS = HD * NT / 4 <= 32 ? 4 : HD * NT / 4 <= 64 ? 3 : 2;
  static constexpr int CTAS = BY_REGS >= 4 && fits(4) ? 4 : BY_REGS >= 3 && fits(3) ? 3 : 2;
  static constexpr int STAGES = room(CTAS) >= 4 * F::BLOCK ? 4 : 2;
  static_assert(fits(CTAS), "the ring needs two stages, the accumulators their place");
  // a warp's region: its ring; at a segment's end its accumulators
  static constexpr int RING = STAGES * F::BLOCK;
  static constexpr int WARP_BYTES = RING > TILE ? RING : TILE;
  static constexpr int MOST = 25;                   // results (or groups of results) merged at a time
  static_assert((MOST * (2 * ROWS + 1) + ROWS) * 4 <= W * WARP_BYTES, "their weights fit the regions");
  // dynamic shared memory: the warps' regions, the tile's, 16 bytes a sequence
  static constexpr int SMEM = W * WARP_BYTES + QFRAG + ROWINFO;
  // a partial result: accumulators, m and l, m and l of the group merged here
  static constexpr int SLOT = ROWS * (HD + 4);
  // what a segment costs besides its blocks, in blocks: its rows of Q, the
  // first copies' latency, the merge of the warps' results and of the cuts'.
  // (8 / 16 / 24 / 32 of them: 64 contexts of up to 8192, 8 rows, 98 / 88 /
  // 89 / 90 us; trees of 24 over 8 contexts of 4099, 32 rows, 128 / 101 / 88 /
  // 85 us.)
  static constexpr int OVERHEAD = NT == 1 ? 16 : 32;
  // the least units a run has: few, long runs cost a short context its
  // latency, many short ones their merge (6 / 10 / 14 / 24: 32 heads of 517
  // positions 10.1 / 10.6 / 11.2 / 14 us, 8 heads of 2000 14.2 / 13.7 / 12.7 /
  // 14.4, a chain of 16 over 700 17.9 / 18.1 / 17.9 / 23.3)
  static constexpr int LEAST = 12;
};

__device__ __forceinline__ void kv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t kv_transpose(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float kv_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float kv_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// cap tanh(x) in powers of two: cap (1 - 2 / (1 + e^{2 x})).  That is off by some
// 2^-22 of the cap: `fine`, for caps of which that is too much for a score,
// takes tanh of less than 1 / 4 from its series up to x^9 (the next term is
// under 2^-26 of it), so that the score is off by 2^-19 of itself at most.
constexpr float kKvFineCap = 256.f;   // 2^-22 of it moves a probability by 2^-14, an eighth of its rounding
__device__ __forceinline__ float kv_cap(float x, float cap, bool fine) {
  float y = 1.f - 2.f * kv_rcp(1.f + kv_exp2(x * (2.f * kKvLog2e)));
  if (fine) {
    const float u = x * x;
    const float z = fmaf(u, fmaf(u, fmaf(u, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
    y = fabsf(x) < 0.25f ? fmaf(x * u, z, x) : y;
  }
  return cap * kKvLog2e * y;
}

// t = sum * what this gives, or tanh's argument: the row's power of two and the
// call's factor.  Held finite, so that a score of zero stays one.
__device__ __forceinline__ float kv_row_factor(float factor, int exponent) {
  return fminf(fmaxf(factor * __uint_as_float(static_cast<uint32_t>(exponent) << 23), -3.4e38f), 3.4e38f);
}

// w = 0 where p = 0.  (Left to the compiler, what few blocks need becomes a
// select for all of them.)
__device__ __forceinline__ void kv_zero_with(float& w, float p) {
  asm volatile("{\n\t.reg .pred z;\n\tsetp.eq.f32 z, %1, 0f00000000;\n\t@z mov.f32 %0, 0f00000000;\n\t}" : "+f"(w) : "f"(p));
}

// v read from shared memory as N words.
template <int N>
__device__ __forceinline__ void kv_lds(uint32_t addr, uint32_t* v) {
  static_assert(N == 1 || N == 2 || N == 4, "1, 2 or 4 words");
  if constexpr (N == 1)
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
  else
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// The offset pairs of a word: p[i] holds the i-th field of the low and of
// the high half, plus 64 (even fields) or 64 / 16 (odd fields of INT4 / INT2).
template <int BITS>
__device__ __forceinline__ void kv_offset_pairs(uint32_t w, const KvMagic<BITS>& c, uint32_t* p) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = i ? w >> 8 : w;
    if constexpr (BITS == 4) {
      p[2 * i] = h2_as_u32(__hadd2(kv_field<0x000F000Fu>(u, c.v[0]), u32_as_h2(0xE380E380u)));       // 1024 - 960
      p[2 * i + 1] = h2_as_u32(kv_field<0x00F000F0u>(u, c.v[1]));
    } else {
      p[4 * i] = h2_as_u32(__hadd2(kv_field<0x00030003u>(u, c.v[0]), u32_as_h2(0xE380E380u)));       // 1024 - 960
      p[4 * i + 1] = h2_as_u32(__hadd2(kv_field<0x000C000Cu>(u, c.v[2]), u32_as_h2(0xDB80DB80u)));   // 256 - 240
      p[4 * i + 2] = h2_as_u32(kv_field<0x00300030u>(u, c.v[1]));
      p[4 * i + 3] = h2_as_u32(kv_field<0x00C000C0u>(u, c.v[3]));
    }
  }
}

struct KvSegment {
  int b, h, tile;        // sequence, key/value head, tile of rows
  int row0, n, kv;       // the sequence's first row, its rows and positions
  int first;             // its first block that may be seen
  int blocks;            // and how many there are
};

// N (1, 2, 4 or 8) consecutive words.
template <int N>
__device__ __forceinline__ void kv_load_words(const void* p, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 u = *static_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 u = static_cast<const uint4*>(p)[i / 4];
      w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
    }
  }
}

// Four consecutive elements, rounded to the type.
__device__ __forceinline__ void kv_store4(void* p, int type, int64_t at, float4 v) {
  if (type == kRowF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = v;
  } else {
    const uint2 b = make_uint2(kv_pack2<kRowBF16>(v.x, v.y), kv_pack2<kRowBF16>(v.z, v.w));
    const uint2 h = make_uint2(kv_pack2<kRowF16>(v.x, v.y), kv_pack2<kRowF16>(v.z, v.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = type == kRowBF16 ? b : h;
  }
}

// A float4 that other SMs wrote in this launch, past the L1 cache.
__device__ __forceinline__ float4 kv_load_shared_result(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// Stores 4 channels of a row: O / l, times D_v^{-1/2}; at: the row's first
// element in Y.
template <int HD>
__device__ __forceinline__ void kv_store_row(const KvAttentionArgs& a, int64_t at, int h, int ch, float4 o, float l) {
  const float f = l > 0.f ? 1.f / l : l;            // l = 0: nothing seen, O = 0; NaN stays
  o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.Dv != nullptr) {
    const float4 d = __ldg(reinterpret_cast<const float4*>(a.Dv + h * HD + ch));
    o = make_float4(o.x * d.x, o.y * d.y, o.z * d.z, o.w * d.w);
  }
  kv_store4(a.Y, a.y_type, at + ch, o);
}

// a / b for a, b >= 0, by 32-bit division where both fit; the 64-bit one is
// long, and out of line.
static __device__ __noinline__ int64_t kv_div64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t kv_div(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return kv_div64(a, b);
}

// How the units of work are cut into runs: run i is [start(i), start(i + 1)).
struct KvRuns {
  int64_t total, each;
  int runs, more;                                   // the first `more` runs have one unit more
  __device__ __forceinline__ int64_t start(int i) const { return i * each + min(i, more); }
  __device__ __forceinline__ int of(int64_t unit) const {
    const int64_t cut = more * (each + 1);
    return static_cast<int>(unit < cut ? kv_div(unit, each + 1) : more + kv_div(unit - cut, each));
  }
};

// Which of its sequence's n new tokens row i_new sees, as bits.  What a tree's
// mask has beyond them stands for no token.
__device__ __forceinline__ uint64_t kv_new_tokens(const KvAttentionArgs& a, int row0, int n, int i_new) {
  return a.tree != nullptr ? a.tree[row0 + i_new] & ~0ull >> (64 - n) : (2ull << i_new) - 1ull;
}

// Which of block blk's 16 tokens a row sees (bit t): of the old tokens all, of
// the new ones those of its mask, with a window those less than `window` back.
__device__ __forceinline__ uint32_t kv_visible(const KvAttentionArgs& a, int row0, int old, int kv, int blk, uint64_t mask,
                                               int pos) {
  const int p0 = blk * 16, there = min(kv - p0, 16), j0 = old - p0;
  auto below = [](int64_t n) { return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u; };
  uint32_t before = below(j0), since = 0;         // of the old tokens, of the new ones
  if (j0 < 16) since = static_cast<uint32_t>(j0 >= 0 ? mask << j0 : mask >> min(-j0, 63)) & ~below(j0);
  if (a.window > 0) {
    const uint32_t far = below(pos - a.window + 1 - p0);
    before &= ~far;
    if (a.tree == nullptr) {
      since &= ~far;
    } else {
#pragma unroll 1
      for (int j = max(j0, 0); j < there; ++j) {
        const int k_new = j - j0;
        if (pos - old - __popcll(kv_new_tokens(a, row0, kv - old, k_new) & ~(1ull << k_new)) >= a.window) since &= ~(1u << j);
      }
    }
  }
  return (before | since) & below(there);
}

}  // namespace ttq

#include "kv_attention_wide.cuh"

namespace ttq {

// A block's shape: NT tiles of 8 rows a warp's products, or (NT = 16) the 256 rows of kv_attention_wide.cuh.
template <int HD, int BITS, int NG, int NT, int QP>
struct KvShape {
  using A = KvAttention<HD, BITS, NG, NT, QP>;
};
template <int HD, int BITS, int NG>
struct KvShape<HD, BITS, NG, 16, 1> {
  using A = KvWide<HD, BITS, NG>;
};

template <int HD, int BITS, int NG, int NT, int QP>
__global__ void __launch_bounds__(KvShape<HD, BITS, NG, NT, QP>::A::W * 32, KvShape<HD, BITS, NG, NT, QP>::A::CTAS)
    kv_attention_kernel(const KvAttentionArgs a) {
  using A = typename KvShape<HD, BITS, NG, NT, QP>::A;
  using F = typename A::F;
  constexpr bool WIDE = NT == 16;
  constexpr int W = A::W, ROWS = A::ROWS, OV = A::OVERHEAD;
  constexpr int PARTS = WIDE ? 1 : W;           // accumulators of a part: the warps', or the block's
  extern __shared__ __align__(1024) uint8_t dynamic_smem[];
  // (operands of tcgen05 stand on 1024-byte boundaries)
  uint8_t* const smem = WIDE ? dynamic_smem + (-smem_addr(dynamic_smem) & 1023u) : dynamic_smem;
  __shared__ __align__(8) uint64_t all_bars[WIDE ? 1 : W * A::STAGES];
  __shared__ int all_absent[WIDE ? 1 : W * A::STAGES];   // the stage's block has no page
  __shared__ __align__(8) KvWideBars wide_bars;
  __shared__ uint32_t tmem_at;
  __shared__ float warp_m[PARTS][ROWS], warp_l[PARTS][ROWS];
  __shared__ KvRuns runs_s;
  __shared__ int abort_flag, last_flag;
  const KvGeometry& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* row_mask = reinterpret_cast<uint64_t*>(smem + PARTS * A::WARP_BYTES + A::QFRAG);
  float* q_factor = reinterpret_cast<float*>(row_mask + ROWS);   // t = <row, (c - z) s> * q_factor
  int* row_pos = reinterpret_cast<int*>(q_factor + ROWS);
  // {end of its work in blocks of one head (56 bits), n (8 bits); kv; row0}
  int4* seqs = reinterpret_cast<int4*>(dynamic_smem + A::SMEM);
  auto pack = [](int64_t end, int n, int kv, int row0) {
    return make_int4(static_cast<int>(end), static_cast<int>((end >> 32) & 0xFFFFFF) | n << 24, kv, row0);
  };
  auto end_of = [](int4 v) {
    return static_cast<int64_t>(static_cast<uint32_t>(v.x)) | static_cast<int64_t>(v.y & 0xFFFFFF) << 32;
  };

  allow_dependents_launch();
  if constexpr (WIDE) {
    if (tid == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&wide_bars.op_full[s], 8);
        mbar_init(&wide_bars.op_free[s], 1);
        mbar_init(&wide_bars.s_full[s], 1);
        mbar_init(&wide_bars.s_free[s], 8);
      }
      mbar_init(&wide_bars.p_full, 8);
      mbar_init(&wide_bars.pv_done, 1);
      mbar_init(&wide_bars.drain, 1);
      fence_barrier_init();
    }
  } else if (lane == 0) {
    for (int s = 0; s < A::STAGES; ++s) mbar_init(&all_bars[warp * A::STAGES + s], 1);
    fence_barrier_init();
  }
  if (tid == 0) abort_flag = 0;
  grid_dependency_wait();

  // ---- the work of every sequence, its running sum, and the runs
  auto first_block = [&](int kv, int n) -> int {   // of those a new token may see
    if (a.window <= 0) return 0;
    const int64_t p = static_cast<int64_t>(kv) - n - a.window + 1;
    return p > 0 ? static_cast<int>(p >> 4) : 0;
  };
  auto tiles_of = [&](int n) { return (n * a.per + ROWS - 1) / ROWS; };
  if (warp == 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < g.batch; b0 += 32) {
      const int b = b0 + lane;
      KvSequence s = {};
      int64_t v = 0;
      if (b < g.batch) {
        if (kv_sequence(g, b, s)) {
          if (s.n > 0) v = static_cast<int64_t>(((s.kv - 1) >> 4) + 1 - first_block(s.kv, s.n) + OV) * tiles_of(s.n);
        } else {
          if (blockIdx.x == 0 && s.n != 0) set_flag(g.status, TTQ_FLAG_BAD_INDEX);
          s.n = 0;
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < g.batch) seqs[b] = pack(base + v, s.n, s.kv, s.row0);
      base += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      const int64_t total = base * g.kv_heads, most = kv_div(total + A::LEAST - 1, A::LEAST);
      const int runs = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
      runs_s.total = total;
      runs_s.runs = runs;
      runs_s.each = runs > 0 ? kv_div(total, runs) : 0;
      runs_s.more = static_cast<int>(total - runs_s.each * runs);
    }
  }
  __syncthreads();
  const KvRuns runs = runs_s;
  const int run = blockIdx.x;
  if (run >= runs.runs) return;
  int64_t x = runs.start(run);
  const int64_t x1 = runs.start(run + 1);

  // ---- the segment at x; a segment's blocks follow OV units of its own
  // cost, so a run that begins within those begins with its first block
  KvSegment seg = {};
  int tiles = 1;
  int64_t left = 0;                             // units of the segment from x on
  auto enter = [&](int b) {                     // sequence b's first segment
    while (((seqs[b].y >> 24) & 0xFF) == 0) ++b;   // there is one: x < total
    const int4 q = seqs[b];
    seg.b = b, seg.h = 0, seg.tile = 0, seg.kv = q.z, seg.row0 = q.w, seg.n = q.y >> 24;
    seg.first = first_block(seg.kv, seg.n);
    seg.blocks = ((seg.kv - 1) >> 4) + 1 - seg.first;
    tiles = tiles_of(seg.n);
  };
  {
    const int64_t per_head_x = kv_div(x, g.kv_heads);
    int lo = 0, hi = g.batch - 1;               // first b with end * kv_heads > x
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end_of(seqs[mid]) > per_head_x) hi = mid; else lo = mid + 1;
    }
    enter(lo);
    const int64_t rest = x - (lo > 0 ? end_of(seqs[lo - 1]) * g.kv_heads : 0);
    const int64_t units = seg.blocks + OV, tile = kv_div(rest, units);
    left = units - (rest - tile * units);
    seg.h = static_cast<int>(tile) / tiles;
    seg.tile = static_cast<int>(tile) - seg.h * tiles;
  }

  const KvMagic<BITS> magic;
  int turn = 0;                                 // blocks (wide: steps) waited for so far: stage and parity of the ring
  if constexpr (WIDE) {
    if (warp == W - 1) {
      tmem_alloc(&tmem_at, A::COLUMNS);
      tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
  }
  // nothing of tensor memory is in use any more
  auto leave = [&]() {
    if constexpr (WIDE) {
      tc_fence_before_sync();
      __syncthreads();
      if (warp == W - 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_at, A::COLUMNS);
      }
    }
  };
  for (bool started = false; x < x1; started = true) {
    if (started && left == 0) {                 // the next segment
      if (++seg.tile == tiles) {
        seg.tile = 0;
        if (++seg.h == g.kv_heads) enter(seg.b + 1);
      }
      left = seg.blocks + OV;
    }
    // blocks [from, from + part) of it are this run's; none if only some of
    // its overhead is
    const int64_t take = x1 - x < left ? x1 - x : left;
    const int from = seg.blocks - static_cast<int>(left < seg.blocks ? left : seg.blocks);
    x += take;
    left -= take;
    const int part = seg.blocks - static_cast<int>(left < seg.blocks ? left : seg.blocks) - from;
    if (part == 0) continue;
    const int old = seg.kv - seg.n;             // positions before the new ones
    const int R = seg.n * a.per, r0 = seg.tile * ROWS;
    const int here = min(R - r0, ROWS);         // rows of the tile
    const float factor = a.scale * (a.cap > 0.f ? kv_rcp(a.cap) : kKvLog2e);
    // of `count` blocks from blk0 on, [plain0, plain1) need no masks: not those
    // that the window of the last new token does not cover, nor those that
    // reach the new tokens
    auto unmasked = [&](int blk0, int count, int& plain0, int& plain1) {
      plain0 = 0;
      if (a.window > 0 && seg.kv > a.window) {
        const int64_t past = static_cast<int64_t>(seg.kv) - a.window;   // p >= past is in every row's window
        const int64_t need = (past + 15) / 16 - blk0;                   // first block wholly in it
        plain0 = need <= 0 ? 0 : need >= count ? count : static_cast<int>(need);
      }
      plain1 = (old >> 4) - blk0;                                       // blocks before the new tokens
    };
    if constexpr (WIDE) {
      float* tables = reinterpret_cast<float*>(row_pos + ROWS);
      KvWidePart<HD, BITS, NG> p{a, wide_bars, &abort_flag, smem, row_mask, q_factor, row_pos, tables,
                                 tables + 2 * NG * A::STEP, reinterpret_cast<int*>(tables + 4 * NG * A::STEP), tmem_at};
      p.b = seg.b, p.h = seg.h, p.row0 = seg.row0, p.n = seg.n, p.kv = seg.kv, p.old = old;
      p.blk0 = seg.first + from, p.count = part, p.steps = (part + 3) / 4, p.here = here, p.r0 = r0, p.turn0 = turn;
      unmasked(p.blk0, part, p.plain0, p.plain1);
      p.rows(tid, factor);
      __syncthreads();
      if (warp < 8) p.softmax(tid, &warp_m[0][tid], &warp_l[0][tid]);
      else p.unpack(warp - 8);
      turn += p.steps;
    } else {
    constexpr int KS = A::KS, MT = A::MT, STAGES = A::STAGES;
    constexpr int PW = F::PIECE / 4;            // words of a lane's piece
    const int gr = lane >> 2, tq = lane & 3;    // row group and quarter of the MMA fragments
    uint8_t* ring = smem + warp * A::WARP_BYTES;
    uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + W * A::WARP_BYTES);
    // behind a part's fragments: [NG][ROWS] sums of a row's group, and the same with the fields' offsets as weights
    float* q_sum = reinterpret_cast<float*>(smem + W * A::WARP_BYTES + A::FRAGS);
    float* q_off = q_sum + NG * ROWS;
    uint64_t* bars = all_bars + warp * STAGES;
    int* absent = all_absent + warp * STAGES;
    // of these this warp's: [blk0, blk0 + count)
    const int mine0 = static_cast<int>(static_cast<int64_t>(part) * warp / W);
    const int count = static_cast<int>(static_cast<int64_t>(part) * (warp + 1) / W) - mine0;
    const int blk0 = seg.first + from + mine0;

    // ---- the tile's rows, 2 NT to a warp: their loads from Q are on their
    // way while the pages are looked up and the copies start
    constexpr int E = HD / 32;                  // consecutive channels of a lane
    constexpr int OWN = ROWS / W;               // rows that a warp prepares
    const bool wide = a.q_type == kRowF32;
    uint32_t raw[OWN][E] = {};                  // E words of float32, E / 2 of 16-bit elements
    {
      int64_t q_at = 0;                         // row OWN warp + lane of the tile in Q
      if (lane < OWN) {
        const int r = OWN * warp + lane, rr = min(r0 + r, R - 1), i_new = rr / a.per;
        const int64_t row = seg.row0 + i_new;
        q_at = row * a.q_row + (seg.h * a.per + rr - i_new * a.per) * a.q_head;
        const uint64_t mask = kv_new_tokens(a, seg.row0, seg.n, i_new);
        row_mask[r] = mask;
        row_pos[r] = old + __popcll(mask & ~(1ull << i_new));
      }
      const uint8_t* q = static_cast<const uint8_t*>(a.Q) + lane * (wide ? 4 * E : 2 * E);
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        const int64_t at = __shfl_sync(0xffffffffu, q_at, k);   // (of rows that are not there: the last one)
        if (wide) kv_load_words<E>(q + at * 4, raw[k]);
        else kv_load_words<E / 2>(q + at * 2, raw[k]);
      }
    }

    // ---- start the copies
    const uint8_t* src = nullptr;               // this lane's block 32 k + lane
    bool any_absent = false;
    const int turn0 = turn;
    auto look_up = [&](int i) {                 // blocks i to i + 31
      const int j = i + lane, blk = blk0 + j;
      src = nullptr;
      if (j < count) {
        const int pg = g.page_of(blk);
        const int page = g.table[seg.b * g.table_stride + pg];
        if (page >= 0 && page < g.num_pages)
          src = g.pages + page * g.page_bytes +
                (static_cast<int64_t>(seg.h) * g.page_blocks + (blk - pg * g.page_blocks)) * F::BLOCK;
        else
          set_flag(g.status, TTQ_FLAG_BAD_INDEX);
      }
      any_absent = __any_sync(0xffffffffu, j < count && src == nullptr) || any_absent;
    };
    auto issue = [&](int i) {                   // by the whole warp; one lane does it
      if (lane == (i & 31)) {
        const int s = (turn0 + i) % STAGES;
        absent[s] = src == nullptr;
        if (src != nullptr) {
          mbar_arrive_expect_tx(&bars[s], F::BLOCK);
          bulk_load(smem_addr(ring + s * F::BLOCK), src, F::BLOCK, &bars[s]);
        } else {
          mbar_arrive(&bars[s]);
        }
      }
    };
    int issued = 0;
    look_up(0);
#pragma unroll
    for (; issued < STAGES; ++issued)
      if (issued < count) issue(issued);

    // ---- the rows as B fragments: scaled by a power of two to [1, 2) and
    // rounded; rows that are not there are zero
    {
      float dk[E];
#pragma unroll
      for (int e = 0; e < E; ++e) dk[e] = a.Dk != nullptr ? __ldg(a.Dk + seg.h * HD + lane * E + e) : 1.f;
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        const int r = OWN * warp + k;
        float v[E], big = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t w = raw[k][e / 2];
          const float bf = __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
          const float hf = __half2float(e & 1 ? u32_as_h2(w).y : u32_as_h2(w).x);
          const float q = wide ? __uint_as_float(raw[k][e]) : a.q_type == kRowBF16 ? bf : hf;
          v[e] = r < here ? q * dk[e] : 0.f;
          big = fmaxf(big, fabsf(v[e]));
        }
        // the row's largest magnitude: bits of non-negative floats order as integers
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);   // 2^-(ex - 127)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int c = lane * E + e, kg = c / F::G, j = c % F::G;
          const int quarter = j / (F::G / 4), idx = kg * (F::G / 4) + j % (F::G / 4);
          // two k steps of a lane stand side by side
          uint32_t* at = qfrag + (((r >> 3) * (KS / 2) + idx / 8) * 32 + 4 * (r & 7) + quarter) * 4 + (idx % 8) / 2;
          const __half2 q = __floats2half2_rn(v[e] * down, v[e + 1] * down);
          *at = h2_as_u32(q);
          if constexpr (QP == 2) {              // what that rounding left (exact in fp32)
            const float2 f = __half22float2(q);
            at[A::QPART / 4] = h2_as_u32(__floats2half2_rn(fmaf(v[e], down, -f.x), fmaf(v[e + 1], down, -f.y)));
          }
        }
        if (lane == 0) q_factor[r] = kv_row_factor(factor, ex);
      }
    }
    __syncthreads();
    if constexpr (BITS != 8) {
      // the sums of each group of the rounded rows: the first product with
      // ones, and (INT2, whose fields' offsets differ) with the offsets, as codes
#pragma unroll 1
      for (int kn = warp; kn < QP * NG * NT; kn += W) {
        const int k = kn / NT % NG, nt = kn % NT, part = kn / (NG * NT) * (A::QPART / 4);
        float one[4] = {}, off[4] = {};
#pragma unroll
        for (int j = 0; j < KS / NG; ++j) {
          const int ks = k * (KS / NG) + j;
          const uint2 bq = *reinterpret_cast<const uint2*>(qfrag + part + ((nt * (KS / 2) + ks / 2) * 32 + lane) * 4 + ks % 2 * 2);
          kv_mma(one, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, bq.x, bq.y);
          if constexpr (BITS == 2) kv_mma(off, A::EVEN, A::EVEN, A::ODD, A::ODD, bq.x, bq.y);
        }
        if (gr == 0) {
          *reinterpret_cast<float2*>(q_sum + part + k * ROWS + 8 * nt + 2 * tq) = make_float2(one[0], one[1]);
          if constexpr (BITS == 2)
            *reinterpret_cast<float2*>(q_off + part + k * ROWS + 8 * nt + 2 * tq) = make_float2(off[0], off[1]);
        }
      }
      __syncthreads();
    }

    // ---- the loop over this warp's blocks
    float o[MT][NT][4] = {};
    float off[NT][2] = {}, l[NT][2] = {};
    constexpr uint32_t ALL = (1u << (2 * NT)) - 1;
    uint32_t seen = 0;                          // columns (bit 2 nt + c) whose offset is a token's
    bool all_seen = false;                      // all columns of all lanes
    float zs[A::VRAW ? NG : 1][4] = {};         // sums of p s (the fields' offset + z) per group
    int plain0, plain1;
    unmasked(blk0, count, plain0, plain1);
    const uint32_t q_frags = smem_addr(qfrag) + lane * 16;

#pragma unroll 1
    for (int done = 0; done < count; ++done) {
      const int stage = (turn0 + done) % STAGES, blk = blk0 + done;
      // (the lanes go on together or not at all)
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[stage], ((turn0 + done) / STAGES) & 1, &abort_flag))) {
        // a copy did not arrive in time: say so and wait, with the same limit,
        // for the copies still in flight; the results are not right any more
        if (lane == 0) {
          set_flag(g.status, TTQ_FLAG_TIMEOUT);
          abort_flag = 1;
#pragma unroll 1
          for (int i = done; i < min(issued, count); ++i) {
            int never = 0;
            mbar_wait(&bars[(turn0 + i) % STAGES], ((turn0 + i) / STAGES) & 1, &never);
          }
        }
        __syncwarp();
        break;
      }
      const uint32_t st = smem_addr(ring + stage * F::BLOCK);
      const bool gone = any_absent && absent[stage] != 0;
      const bool masked = gone || done < plain0 || done >= plain1;
      // -- scores
      float s[NT][4];
      if constexpr (QP == 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      }
      uint32_t kp[2][NG];
      kv_lds<NG>(st + F::CODES + gr * NG * 4, kp[0]);
      kv_lds<NG>(st + F::CODES + (gr + 8) * NG * 4, kp[1]);
      constexpr int KSG = KS / NG;              // k steps of a group
      constexpr int KSW = BITS == 8 ? 1 : 32 / BITS / 4;   // k steps of a word
      uint32_t kw[2][PW], pa[2][2 * KSW];
#pragma unroll 1
      for (int part = 0; part < A::QFRAG; part += A::QPART) {   // of Q: its offset
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          float acc[NT][4];
          uint32_t bq[NT][4];                     // Q's fragments of two k steps
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
          for (int j = 0; j < KSG; ++j) {
            const int ks = k * KSG + j, w = ks / KSW, in = ks % KSW;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (in == 0 && w % PW == 0)
                kv_lds<PW>(st + (w / PW * 2 + r) * 32 * F::PIECE + lane * F::PIECE, kw[r]);
              if (in == 0) {
                if constexpr (BITS == 8) kv_e4m3x4(kw[r][w % PW], pa[r][0], pa[r][1]);
                else kv_offset_pairs<BITS>(kw[r][w % PW], magic, pa[r]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (ks % 2 == 0) kv_lds<4>(q_frags + part + (nt * (KS / 2) + ks / 2) * 512, bq[nt]);
              kv_mma(acc[nt], pa[0][2 * in], pa[1][2 * in], pa[0][2 * in + 1], pa[1][2 * in + 1], bq[nt][ks % 2 * 2],
                     bq[nt][ks % 2 * 2 + 1]);
            }
          }
          const float2 p0 = __half22float2(u32_as_h2(kp[0][k])), p1 = __half22float2(u32_as_h2(kp[1][k]));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (BITS != 8) {
              const float2 qs = *reinterpret_cast<const float2*>(q_sum + part / 4 + k * ROWS + 8 * nt + 2 * tq);
              float z0 = p0.y, z1 = p1.y;
              if constexpr (BITS == 4) {          // both fields are offset by 64
                z0 += 64.f, z1 += 64.f;
              } else {
                const float2 qo = *reinterpret_cast<const float2*>(q_off + part / 4 + k * ROWS + 8 * nt + 2 * tq);
                acc[nt][0] -= qo.x, acc[nt][1] -= qo.y, acc[nt][2] -= qo.x, acc[nt][3] -= qo.y;
              }
              acc[nt][0] = fmaf(-z0, qs.x, acc[nt][0]);
              acc[nt][1] = fmaf(-z0, qs.y, acc[nt][1]);
              acc[nt][2] = fmaf(-z1, qs.x, acc[nt][2]);
              acc[nt][3] = fmaf(-z1, qs.y, acc[nt][3]);
            }
            if (QP == 1 && k == 0) {
              s[nt][0] = acc[nt][0] * p0.x, s[nt][1] = acc[nt][1] * p0.x;
              s[nt][2] = acc[nt][2] * p1.x, s[nt][3] = acc[nt][3] * p1.x;
            } else {
              s[nt][0] = fmaf(acc[nt][0], p0.x, s[nt][0]);
              s[nt][1] = fmaf(acc[nt][1], p0.x, s[nt][1]);
              s[nt][2] = fmaf(acc[nt][2], p1.x, s[nt][2]);
              s[nt][3] = fmaf(acc[nt][3], p1.x, s[nt][3]);
            }
          }
        }
      }
      // -- V's scales of tokens gr and gr + 8, and zeros of 2 tq, 2 tq + 1 (+ 8)
      float vs[2][NG];
      [[maybe_unused]] uint32_t vz[2][NG], keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      const uint32_t vst = st + F::V_OFFSET;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t vp[NG];
        kv_lds<NG>(vst + F::CODES + (gr + 8 * r) * NG * 4, vp);
#pragma unroll
        for (int k = 0; k < NG; ++k) vs[r][k] = __half2float(u32_as_h2(vp[k]).x);
        if constexpr (BITS != 8) {
          uint32_t e[2 * NG];                   // both tokens' pairs are contiguous
          kv_lds<NG == 1 ? 2 : 4>(vst + F::CODES + (2 * tq + 8 * r) * NG * 4, e);
          if constexpr (NG == 4) kv_lds<4>(vst + F::CODES + (2 * tq + 8 * r) * NG * 4 + 16, e + 4);
#pragma unroll
          for (int k = 0; k < NG; ++k) vz[r][k] = __byte_perm(e[k], e[NG + k], 0x7632);
        }
      }
      // -- scores in powers of two less the row's offset
      auto scaled = [&](auto of) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 f = *reinterpret_cast<const float2*>(q_factor + 8 * nt + 2 * tq);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nt][i] = of(s[nt][i], (i & 1) ? f.y : f.x, off[nt][i & 1]);
        }
      };
      if (!(a.cap > 0.f)) scaled([](float x, float f, float o) { return fmaf(x, f, -o); });
      else if (a.cap > kKvFineCap) scaled([&](float x, float f, float o) { return kv_cap(x * f, a.cap, true) - o; });
      else scaled([&](float x, float f, float o) { return kv_cap(x * f, a.cap, false) - o; });
      // -- masks: lane r finds which of the block's tokens row r sees; tokens
      // that are not there count for nothing, whatever their bytes are
      if (masked) {
        const int there = gone ? 0 : min(seg.kv - blk * 16, 16);
        const uint32_t vis =
            gone ? 0u : kv_visible(a, seg.row0, old, seg.kv, blk, row_mask[lane % ROWS], row_pos[lane % ROWS]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t v = __shfl_sync(0xffffffffu, vis, 8 * nt + 2 * tq + c) >> gr;
            if (!(v & 1u)) s[nt][c] = -INFINITY;
            if (!(v & 256u)) s[nt][c + 2] = -INFINITY;
          }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t0 = 2 * tq + 8 * r;
          keep[r] = (t0 < there ? 0xFFFFu : 0u) | (t0 + 1 < there ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            if (gr + 8 * r >= there) vs[r][k] = 0.f;
            if constexpr (BITS != 8) vz[r][k] &= keep[r];
          }
        }
      }
      // -- the offsets move only when a t + e is well above one (and to a
      // column's first); whether one may is asked of the lane's largest score
      // and scale (NaN aside) first
      float top[2] = {kKvLeastScale, kKvLeastScale}, most = s[0][0];
#pragma unroll
      for (int k = 0; k < NG; ++k) top[0] = fmaxf(top[0], vs[0][k]), top[1] = fmaxf(top[1], vs[1][k]);
#pragma unroll
      for (int i = 1; i < 4 * NT; ++i) most = fmaxf(most, s[i / 4][i % 4]);
      if (__any_sync(0xffffffffu, !all_seen || most + kv_exponent(fmaxf(top[0], top[1])) > kKvSlack)) {
        const float e0 = kv_exponent(top[0]), e1 = kv_exponent(top[1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float up = fmaxf(s[nt][c] + e0, s[nt][c + 2] + e1);
            up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
            up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
            up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
            const uint32_t bit = 1u << (2 * nt + c);
            // (each column by its own tokens, so that no row's result depends on another's)
            if (!(up > -INFINITY) || ((seen & bit) && up <= kKvSlack)) up = 0.f;
            else seen |= bit;
            // (before the first score l and o are zero, or NaN)
            const float f = up < 0.f ? 1.f : kv_exp2(-up);
            off[nt][c] += up;
            s[nt][c] -= up;
            s[nt][c + 2] -= up;
            l[nt][c] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][nt][c] *= f;
              o[mt][nt][c + 2] *= f;
            }
            if constexpr (A::VRAW) {
#pragma unroll
              for (int k = 0; k < NG; ++k) {
                zs[k][c] *= f;
                zs[k][c + 2] *= f;
              }
            }
          }
        all_seen = __all_sync(0xffffffffu, seen == ALL);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[nt][i] = kv_exp2(s[nt][i]);
          l[nt][i & 1] += s[nt][i];
        }
      // -- p s_V as the B operand, and the second product
      constexpr int MTG = MT / NG;              // m tiles of a group
      constexpr int MTW = BITS == 8 ? 1 : 16 / BITS / 2;   // m tiles of a word
      uint32_t vw[2][PW], pv[2][BITS == 8 ? 2 : 16 / BITS];
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w0 = s[nt][0] * vs[0][k], w1 = s[nt][1] * vs[0][k], w2 = s[nt][2] * vs[1][k], w3 = s[nt][3] * vs[1][k];
          if (masked) {                         // a NaN scale reaches only those that see its token
            kv_zero_with(w0, s[nt][0]);
            kv_zero_with(w1, s[nt][1]);
            kv_zero_with(w2, s[nt][2]);
            kv_zero_with(w3, s[nt][3]);
          }
          b[nt][0] = kv_transpose(h2_as_u32(__floats2half2_rn(w0, w1)));
          b[nt][1] = kv_transpose(h2_as_u32(__floats2half2_rn(w2, w3)));
        }
        [[maybe_unused]] KvZero<BITS> z[2];
        if constexpr (A::VRAW) {
          // rows of even fields, then of odd ones
          const uint32_t e0 = h2_as_u32(__hadd2(u32_as_h2(vz[0][k]), u32_as_h2(A::EVEN)));
          const uint32_t e1 = h2_as_u32(__hadd2(u32_as_h2(vz[1][k]), u32_as_h2(A::EVEN)));
          if constexpr (BITS == 4) {
            kv_mma(zs[k], e0, e0, e1, e1, b[0][0], b[0][1]);
          } else {
            const uint32_t d0 = h2_as_u32(__hadd2(u32_as_h2(vz[0][k]), u32_as_h2(A::ODD)));
            const uint32_t d1 = h2_as_u32(__hadd2(u32_as_h2(vz[1][k]), u32_as_h2(A::ODD)));
            kv_mma(zs[k], e0, d0, e1, d1, b[0][0], b[0][1]);
          }
        } else if constexpr (BITS != 8) {
#pragma unroll
          for (int r = 0; r < 2; ++r) z[r].set(vz[r][k]);
        }
#pragma unroll
        for (int j = 0; j < MTG; ++j) {
          const int mt = k * MTG + j, w = mt / MTW, in = mt % MTW;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (in == 0 && w % PW == 0) {
              kv_lds<PW>(vst + (w / PW * 2 + r) * 32 * F::PIECE + lane * F::PIECE, vw[r]);
              if (BITS == 8 && masked) {        // (any INT code is finite; an E4M3 one may be a NaN)
#pragma unroll
                for (int i = 0; i < PW; ++i) vw[r][i] &= keep[r];
              }
            }
            if (in == 0 || (!A::VRAW && j == 0)) {
              if constexpr (BITS == 8)          // bytes: even token's two channels, then the odd one's
                kv_e4m3x4(__byte_perm(vw[r][w % PW], 0, 0x3120), pv[r][0], pv[r][1]);
              else if constexpr (A::VRAW)
                kv_offset_pairs<BITS>(vw[r][w % PW], magic, pv[r]);
              else
                kv_int_pairs<BITS>(vw[r][w % PW], z[r], magic, pv[r]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            kv_mma(o[mt][nt], pv[0][2 * in], pv[0][2 * in + 1], pv[1][2 * in], pv[1][2 * in + 1], b[nt][0], b[nt][1]);
        }
      }
      __syncwarp();
      if (issued < count) {
        if ((issued & 31) == 0) look_up(issued);
        issue(issued++);
      }
      if constexpr (A::VRAW) {
        // the offsets and zeros are taken off the accumulators, often enough
        // that the sums of offset codes do not grow much past their difference
        if ((done & 15) == 15 || done + 1 == count) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][0][i] -= zs[mt / (MT / NG)][i];
#pragma unroll
          for (int k = 0; k < NG; ++k) zs[k][0] = zs[k][1] = zs[k][2] = zs[k][3] = 0.f;
        }
      }
    }
    turn = turn0 + count;

    // ---- the end of the segment, or of this run's part of it: the warps'
    // accumulators go to their regions, the rows' results from there to Y or,
    // of a part, to the workspace
    {
      float* tile = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * nt + 2 * tq + c;
          float v = l[nt][c];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (gr == 0) {
            warp_l[warp][r] = v;
            warp_m[warp][r] = (seen >> (2 * nt + c) & 1u) ? off[nt][c] : kKvFloor;
          }
#pragma unroll
          for (int mt = 0; mt < MT; mt += 2) {
            // the four channels of m tiles mt and mt + 1 that this lane holds of the row
            const int ch = 2 * mt / (F::G / 8) * F::G + gr * (F::G / 8) + 2 * mt % (F::G / 8);
            *reinterpret_cast<float4*>(tile + r * A::LDO + ch) =
                make_float4(o[mt][nt][c], o[mt][nt][c + 2], o[mt + 1][nt][c], o[mt + 1][nt][c + 2]);
          }
        }
    }
    }
    __syncthreads();
    const bool failed = *static_cast<volatile int*>(&abort_flag) != 0;
    const bool whole = part == seg.blocks;
    auto store_row = [&](int r, int ch, float4 acc, float sum) {
      const int rr = r0 + r, i_new = rr / a.per;
      const int64_t row = static_cast<int64_t>(seg.row0 + i_new) * a.heads + seg.h * a.per + rr - i_new * a.per;
      kv_store_row<HD>(a, row * HD, seg.h, ch, acc, sum);
    };
    // a part's result is in the run's first place if the segment began in an
    // earlier run, else in its second
    float* slot = a.part + (2 * static_cast<int64_t>(run) + (from > 0 ? 0 : 1)) * A::SLOT;
#pragma unroll 1
    for (int i = tid; i < here * (HD / 4); i += W * 32) {
      const int r = i / (HD / 4), ch = (i % (HD / 4)) * 4;
      float mx = warp_m[0][r], sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 1; w < PARTS; ++w) mx = fmaxf(mx, warp_m[w][r]);
#pragma unroll
      for (int w = 0; w < PARTS; ++w) {
        const float f = kv_exp2(warp_m[w][r] - mx);
        const float4 v = *reinterpret_cast<const float4*>(smem + w * A::WARP_BYTES + (r * A::LDO + ch) * 4);
        sum = fmaf(warp_l[w][r], f, sum);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        store_row(r, ch, acc, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(slot + r * HD + ch), acc);
        if (ch == 0) {
          __stcg(slot + ROWS * HD + r, mx);
          __stcg(slot + ROWS * (HD + 1) + r, sum);
        }
      }
    }
    if (!whole) {
      // ---- the segment's results are those of runs first to last.  Tickets:
      // the last of a group of results merges it, the last group the segment.
      // Groups of about the root of all results, where there are more than 12
      // (there are some 600 at most).
      const int64_t end = x + left, begin = end - seg.blocks;   // the units of its blocks
      const int first = runs.of(begin), results = runs.of(end - 1) - first + 1;
      auto place_of = [&](int k) { return 2 * (first + k) + (k == 0 ? 1 : 0); };
      int group = results;
      if (results > 12)
        for (group = 4; group * group < results;) ++group;
      const int groups = (results + group - 1) / group;
      float* ms = reinterpret_cast<float*>(smem);     // weights that a merge gives the results
      float* ls = ms + A::MOST * ROWS;
      float* sums = ls + A::MOST * ROWS;
#pragma unroll 1
      for (int level = groups > 1 ? 0 : 1; level < 2; ++level) {
        // results k0, k0 + step, ...: n of them, their own or their groups'
        const int k0 = level == 0 ? (run - first) / group * group : 0;
        const int step = level == 1 && groups > 1 ? group : 1;
        const int n = level == 0 ? min(group, results - k0) : step > 1 ? groups : results;
        __syncthreads();                        // all of the result is written
        // (a group of one may share its ticket with the next segment's first: it takes none)
        if (level == 1 || n > 1) {
          if (tid == 0) {
            uint32_t* ticket = a.tickets + (level == 0 ? gridDim.x + first + k0 : first);
            __threadfence();
            const bool last = atomicAdd(ticket, 1u) == static_cast<uint32_t>(n - 1);
            if (last) {
              *ticket = 0;                      // left at zero
              __threadfence();
            }
            last_flag = last;
          }
          __syncthreads();
          if (!last_flag) break;
        }
        const int mls = ROWS * (step > 1 ? HD + 2 : HD);
        for (int i = tid; i < n * ROWS; i += W * 32) {
          const float* p = a.part + static_cast<int64_t>(place_of(k0 + i / ROWS * step)) * A::SLOT + mls + i % ROWS;
          ms[i] = __ldcg(p);
          ls[i] = __ldcg(p + ROWS);
        }
        __syncthreads();
        float* to = a.part + static_cast<int64_t>(place_of(k0)) * A::SLOT;   // a group's result
        if (tid < here) {
          float mx = kKvFloor, sum = 0.f;
#pragma unroll 1
          for (int i = 0; i < n; ++i) mx = fmaxf(mx, ms[i * ROWS + tid]);
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            const float f = kv_exp2(ms[i * ROWS + tid] - mx);
            ms[i * ROWS + tid] = f;
            sum = fmaf(ls[i * ROWS + tid], f, sum);
          }
          sums[tid] = sum;
          if (level == 0) {
            __stcg(to + ROWS * (HD + 2) + tid, mx);
            __stcg(to + ROWS * (HD + 3) + tid, sum);
          }
        }
        __syncthreads();
        // 16 loads at a time that do not wait for one another
#pragma unroll 1
        for (int i0 = tid; i0 < here * (HD / 4); i0 += 4 * W * 32) {
          float4 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int j0 = 0; j0 < n; j0 += 4) {
            float4 v[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                const int i = i0 + e * W * 32;
                if (j0 + j < n && i < here * (HD / 4))
                  v[j][e] = kv_load_shared_result(a.part + static_cast<int64_t>(place_of(k0 + (j0 + j) * step)) * A::SLOT + i * 4);
              }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = i0 + e * W * 32;
                const float f = j0 + j < n && i < here * (HD / 4) ? ms[(j0 + j) * ROWS + i / (HD / 4)] : 0.f;
                acc[e].x = fmaf(v[j][e].x, f, acc[e].x);
                acc[e].y = fmaf(v[j][e].y, f, acc[e].y);
                acc[e].z = fmaf(v[j][e].z, f, acc[e].z);
                acc[e].w = fmaf(v[j][e].w, f, acc[e].w);
              }
          }
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * W * 32;
            const float4 v = e == 0 ? acc[0] : e == 1 ? acc[1] : e == 2 ? acc[2] : acc[3];
            if (i < here * (HD / 4)) {
              if (level == 1) store_row(i / (HD / 4), (i % (HD / 4)) * 4, v, sums[i / (HD / 4)]);
              else __stcg(reinterpret_cast<float4*>(to + i * 4), v);   // read by this thread alone
            }
          }
        }
      }
    }
    if (failed) {                               // (set before the barrier above: the same for all threads)
      if (WIDE && tid == 8 * 32) {              // no product is under way when tensor memory is freed
        int never = 0;
        mma_commit(&wide_bars.drain);
        mbar_wait(&wide_bars.drain, 0, &never);
      }
      leave();
      return;
    }
    fence_proxy_async_smem();                   // the regions are the copies' again
    __syncthreads();
  }
  leave();
}

// One head size's kernels (a source file each).
cudaError_t kv_attention_hd64(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
cudaError_t kv_attention_hd128(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
cudaError_t kv_attention_hd256(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
// Blocks per SM of the same kernels; 0 if the format is not built.
int kv_attention_ctas_hd64(int bits, int group, int nt, int q_parts);
int kv_attention_ctas_hd128(int bits, int group, int nt, int q_parts);
int kv_attention_ctas_hd256(int bits, int group, int nt, int q_parts);

// Calls f(BITS, NG, NT, QP) as constants for one head size; false if not built.
template <int HD, typename Fn>
bool kv_with_format(int bits, int group, int nt, int q_parts, Fn&& f) {
  auto tiles = [&](auto BITSc, auto NGc) {
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 2> two{};
    if (nt == 1) return q_parts == 1 ? f(BITSc, NGc, one, one) : f(BITSc, NGc, one, two), true;
    if (nt == 2) return q_parts == 1 ? f(BITSc, NGc, two, one) : f(BITSc, NGc, two, two), true;
    if constexpr (HD <= 128) {
      constexpr std::integral_constant<int, 4> four{};
      if (nt == 4) return q_parts == 1 ? f(BITSc, NGc, four, one) : f(BITSc, NGc, four, two), true;
      if (nt == 3 && q_parts == 1) return f(BITSc, NGc, std::integral_constant<int, 3>{}, one), true;
    }
    if constexpr (HD <= 128 && decltype(NGc)::value <= 2)
      if (nt == 16 && q_parts == 1) return f(BITSc, NGc, std::integral_constant<int, 16>{}, one), true;
    return false;
  };
  auto groups = [&](auto BITSc) {
    const int ng = HD / group;
    if (ng == 1) return tiles(BITSc, std::integral_constant<int, 1>{});
    if (ng == 2) return tiles(BITSc, std::integral_constant<int, 2>{});
    if constexpr (HD >= 128)
      if (ng == 4) return tiles(BITSc, std::integral_constant<int, 4>{});
    return false;
  };
  if (bits == 2) return groups(std::integral_constant<int, 2>{});
  if (bits == 4) return groups(std::integral_constant<int, 4>{});
  if (bits == 8) return groups(std::integral_constant<int, 8>{});
  return false;
}

template <int HD>
int kv_attention_ctas(int bits, int group, int nt, int q_parts) {
  int n = 0;
  kv_with_format<HD>(bits, group, nt, q_parts, [&](auto B, auto G, auto N, auto P) {
    n = KvShape<HD, decltype(B)::value, decltype(G)::value, decltype(N)::value, decltype(P)::value>::A::CTAS;
  });
  return n;
}

template <int HD>
cudaError_t kv_attention_launch(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p,
                                cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  kv_with_format<HD>(bits, group, p.nt, p.q_parts, [&](auto Bc, auto Gc, auto Nc, auto Pc) {
    constexpr int BITS = decltype(Bc)::value, NG = decltype(Gc)::value, NT = decltype(Nc)::value, QP = decltype(Pc)::value;
    using A = typename KvShape<HD, BITS, NG, NT, QP>::A;
    auto* kernel = kv_attention_kernel<HD, BITS, NG, NT, QP>;
    const int smem = A::SMEM + 16 * a.g.batch;
    static std::atomic<uint64_t> set{0};
    if ((e = kv_allow_smem(reinterpret_cast<const void*>(kernel), A::SMEM + 16 * kKvMaxBatch, set)) != cudaSuccess) return;
    e = launch_kernel(kernel, dim3(p.grid), dim3(A::W * 32), smem, stream, true, a);
  });
  return e;
}

}  // namespace ttq
