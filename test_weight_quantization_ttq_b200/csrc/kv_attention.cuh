// Attention of a few new tokens per sequence over the quantised paged cache
// (ttq_kv_attention).
//
//   t_j = scale <q, K_j>  (capped: cap tanh(t_j / cap));  y = sum_j softmax(t)_j V_j
// with K_j = s (c - z) D_k^{-1/2} per group of channels, V_j likewise.
//
// Work.  The rows of one key/value head (its query heads x the sequence's
// new tokens) form tiles of 8 NT rows; a segment is one (sequence, head,
// tile) with all blocks of 16 tokens that it may see.  All segments'
// blocks, laid end to end, are cut into equal runs, one per thread block of
// the grid, so that contexts of any lengths load the SMs evenly; a segment
// cut by a run's end leaves partial results (running maximum, sum and
// accumulator) in the workspace, which kv_join_kernel merges in order.
//
// A warp takes every W-th block of its segment through a ring of shared
// memory stages, one bulk copy per block (codes and pairs of K and V
// together), and keeps its own softmax state; the warps' states are merged
// once per segment.  Products are m16n8k16 with the codes as the A operand:
//   S^T [16 tokens x 8 rows] = (c - z)_K Q^T   per group of channels, then
//       scaled by the token's s_K in fp32;
//   O^T [channels x 8 rows] += (c - z)_V^T (p s_V)^T.
// c - z is exact in binary16 and is formed in two instructions per pair of
// codes: the code bits are put under an exponent whose unit they count
// (1024 + c, 256 + c, 64 + c or 16 + c by their place in the word), and that
// offset + z is subtracted.  p s_V moves from the accumulator layout (tokens
// along the lanes' rows) to the B operand's by an 8 x 8 transposition within
// the warp.
//
// Numerics.  Each row of q (times D_k^{-1/2}) is scaled by a power of two to
// [1, 2) and rounded to binary16.  Scores, the running maximum m and the sum
// l are fp32.  m moves only when a score exceeds it by more than 8 (in
// powers of two), which keeps p <= 256; p s_V is rounded to binary16 after
// scaling by 2^-E, E the running maximum of the exponents of s_V, so that
// scales of any size use binary16's normal range.
#pragma once

#include <atomic>
#include <type_traits>

#include "kv_device.cuh"
#include "ttq_kernels.h"

namespace ttq {

constexpr float kKvLog2e = 1.4426950408889634f;
constexpr float kKvFloor = -1e30f;    // running maximum before any score
constexpr float kKvSlack = 8.f;

template <int HD, int BITS, int NG, int NT>
struct KvAttention {
  using F = KvFormat<HD, BITS, NG>;
  static constexpr int W = 4;                       // warps of a block
  static constexpr int ROWS = 8 * NT;               // query rows of a tile
  static constexpr int KS = HD / 16;                // k steps of the first product
  static constexpr int MT = HD / 16;                // m tiles of the second
  // blocks per SM by registers (HD NT / 4 accumulators a thread) and memory
  static constexpr int SM_BYTES = 208 * 1024;
  static constexpr int LDO = HD + 4;                // padded row of the merge buffer
  static constexpr int MERGE = W * ROWS * LDO * 4;
  static constexpr int QFRAG = NT * KS * 32 * 8;
  static constexpr int OTHER = QFRAG + 4096;        // static arrays, and 16 bytes a sequence
  static constexpr int room(int ctas) { return SM_BYTES / ctas - OTHER; }
  static constexpr int fits(int ctas) { return room(ctas) >= W * 2 * F::BLOCK && room(ctas) >= MERGE; }
  static constexpr int CTAS = HD * NT / 4 <= 64 ? (fits(4) ? 4 : fits(3) ? 3 : 2) : 2;
  static constexpr int STAGES_FIT = room(CTAS) / (W * F::BLOCK);
  static constexpr int STAGES = STAGES_FIT > 4 ? 4 : STAGES_FIT;
  static_assert(STAGES >= 2, "the ring needs two stages");
  static constexpr int RING = W * STAGES * F::BLOCK;
  static constexpr int UNION = RING > MERGE ? RING : MERGE;
  // dynamic shared memory: ring / merge | Q fragments | sequences (16 B each)
  static constexpr int SMEM = UNION + QFRAG;
  static constexpr int SLOT = ROWS * (HD + 2);      // floats of a partial result
  // what a segment costs besides its blocks, in blocks: its rows of Q, the
  // first copy's latency and the merge
  static constexpr int OVERHEAD = 8;
};

__device__ __forceinline__ void kv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
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

// A lane's words of one half of a part.
template <int LB, int PIECE>
__device__ __forceinline__ void kv_lane_words(uint32_t part, int lane, int half, uint32_t* v) {
#pragma unroll
  for (int c = 0; c < LB / PIECE; ++c)
    kv_lds<PIECE / 4>(part + (c * 2 + half) * 32 * PIECE + lane * PIECE, v + c * (PIECE / 4));
}

// The offsets + zero that the pairs of a word carry: o[i] for the i-th place.
template <int BITS>
struct KvZero {
  static constexpr int N = BITS == 8 ? 1 : 8 / BITS;   // different places of a half word's byte
  __half2 o[N];
  __device__ __forceinline__ void set(uint32_t z) {    // two binary16 zeros
    if constexpr (BITS == 4) {
      o[0] = __hadd2(u32_as_h2(z), u32_as_h2(0x64006400u));   // 1024 + z
      o[1] = __hadd2(u32_as_h2(z), u32_as_h2(0x54005400u));   // 64 + z
    } else if constexpr (BITS == 2) {
      o[0] = __hadd2(u32_as_h2(z), u32_as_h2(0x64006400u));   // 1024 + z
      o[1] = __hadd2(u32_as_h2(z), u32_as_h2(0x5C005C00u));   // 256 + z
      o[2] = __hadd2(u32_as_h2(z), u32_as_h2(0x54005400u));   // 64 + z
      o[3] = __hadd2(u32_as_h2(z), u32_as_h2(0x4C004C00u));   // 16 + z
    }
  }
};

// The pairs (c - z) of a word of INT codes: p[i] holds the i-th field of the
// low and of the high half.
template <int BITS>
__device__ __forceinline__ void kv_int_pairs(uint32_t w, const KvZero<BITS>& z, uint32_t* p) {
  if constexpr (BITS == 4) {
    const uint32_t u = w >> 8;
    p[0] = h2_as_u32(__hsub2(u32_as_h2((w & 0x000F000Fu) | 0x64006400u), z.o[0]));
    p[1] = h2_as_u32(__hsub2(u32_as_h2((w & 0x00F000F0u) | 0x54005400u), z.o[1]));
    p[2] = h2_as_u32(__hsub2(u32_as_h2((u & 0x000F000Fu) | 0x64006400u), z.o[0]));
    p[3] = h2_as_u32(__hsub2(u32_as_h2((u & 0x00F000F0u) | 0x54005400u), z.o[1]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = i ? w >> 8 : w;
      p[4 * i] = h2_as_u32(__hsub2(u32_as_h2((u & 0x00030003u) | 0x64006400u), z.o[0]));
      p[4 * i + 1] = h2_as_u32(__hsub2(u32_as_h2((u & 0x000C000Cu) | 0x5C005C00u), z.o[1]));
      p[4 * i + 2] = h2_as_u32(__hsub2(u32_as_h2((u & 0x00300030u) | 0x54005400u), z.o[2]));
      p[4 * i + 3] = h2_as_u32(__hsub2(u32_as_h2((u & 0x00C000C0u) | 0x4C004C00u), z.o[3]));
    }
  }
}

struct KvSegment {
  int b, h, tile;        // sequence, key/value head, tile of rows
  int row0, n, kv;       // the sequence's first row, its rows and positions
  int first;             // its first block that may be seen
  int blocks;            // and how many there are
};

// E (2, 4 or 8) consecutive elements of a row tensor of the given type.
template <int E>
__device__ __forceinline__ void kv_load_lane(const void* p, int type, int64_t at, float (&v)[E]) {
  if (type == kRowF32) {
    const float2* s = reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 f = s[e];
      v[2 * e] = f.x, v[2 * e + 1] = f.y;
    }
    return;
  }
  uint32_t w[E / 2];
  const uint16_t* s = static_cast<const uint16_t*>(p) + at;
  if constexpr (E == 2) w[0] = *reinterpret_cast<const uint32_t*>(s);
  if constexpr (E == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(s);
    w[0] = u.x, w[1] = u.y;
  }
  if constexpr (E == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(s);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    if (type == kRowBF16) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(u32_as_h2(w[e]));
      v[2 * e] = f.x, v[2 * e + 1] = f.y;
    }
  }
}
// Four consecutive elements, rounded to the type.
__device__ __forceinline__ void kv_store4(void* p, int type, int64_t at, float4 v) {
  if (type == kRowF32)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = v;
  else if (type == kRowBF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
        make_uint2(kv_pack2<kRowBF16>(v.x, v.y), kv_pack2<kRowBF16>(v.z, v.w));
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) =
        make_uint2(kv_pack2<kRowF16>(v.x, v.y), kv_pack2<kRowF16>(v.z, v.w));
}

// Stores 4 channels of a row of a segment: O / l, times D_v^{-1/2}.
template <int HD>
__device__ __forceinline__ void kv_store_row(const KvAttentionArgs& a, int row0, int h, int r, int ch, float4 o,
                                             float l) {
  const float f = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // l = 0: nothing seen; NaN stays
  o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.Dv != nullptr) {
    const float4 d = __ldg(reinterpret_cast<const float4*>(a.Dv + h * HD + ch));
    o = make_float4(o.x * d.x, o.y * d.y, o.z * d.z, o.w * d.w);
  }
  const int64_t row = row0 + r / a.per;
  const int head = h * a.per + r % a.per;
  kv_store4(a.Y, a.y_type, (row * a.heads + head) * HD + ch, o);
}

template <int HD, int BITS, int NG, int NT>
__global__ void __launch_bounds__(KvAttention<HD, BITS, NG, NT>::W * 32, KvAttention<HD, BITS, NG, NT>::CTAS)
    kv_attention_kernel(const KvAttentionArgs a) {
  using A = KvAttention<HD, BITS, NG, NT>;
  using F = typename A::F;
  constexpr int W = A::W, ROWS = A::ROWS, KS = A::KS, MT = A::MT, STAGES = A::STAGES;
  constexpr int WORDS = F::LB / 4;              // words of a lane's half
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W * STAGES];
  __shared__ int absent[W * STAGES];            // the stage's block has no page
  __shared__ float q_factor[ROWS];              // t = <row, (c - z) s> * q_factor
  __shared__ int row_pos[ROWS];
  __shared__ uint64_t row_mask[ROWS];
  __shared__ int new_pos[kKvMaxNew];
  __shared__ float warp_m[W][ROWS], warp_l[W][ROWS];
  __shared__ int abort_flag;
  const KvGeometry& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, tq = lane & 3;      // row group and quarter of the MMA fragments
  uint8_t* ring = smem + warp * STAGES * F::BLOCK;
  uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + A::UNION);
  // {end of its work in blocks of one head (56 bits), n (8 bits); kv; row0}
  int4* seqs = reinterpret_cast<int4*>(smem + A::UNION + A::QFRAG);
  auto pack = [](int64_t end, int n, int kv, int row0) {
    return make_int4(static_cast<int>(end), static_cast<int>((end >> 32) & 0xFFFFFF) | n << 24, kv, row0);
  };
  auto end_of = [](int4 v) {
    return static_cast<int64_t>(static_cast<uint32_t>(v.x)) | static_cast<int64_t>(v.y & 0xFFFFFF) << 32;
  };

  allow_dependents_launch();
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bars[warp * STAGES + s], 1);
      absent[warp * STAGES + s] = 0;
    }
    fence_barrier_init();
  }
  if (tid == 0) abort_flag = 0;
  grid_dependency_wait();

  // ---- the work of every sequence and its running sum
  auto first_block = [&](int kv, int n) -> int {   // of those a new token may see
    if (a.window <= 0) return 0;
    const int64_t p = static_cast<int64_t>(kv) - n - a.window + 1;
    return p > 0 ? static_cast<int>(p >> 4) : 0;
  };
  auto tiles_of = [&](int n) { return (n * a.per + ROWS - 1) / ROWS; };
  for (int b = tid; b < g.batch; b += W * 32) {
    KvSequence s;
    int64_t w = 0;
    if (kv_sequence(g, b, s)) {
      if (s.n > 0) w = static_cast<int64_t>(((s.kv - 1) >> 4) + 1 - first_block(s.kv, s.n) + A::OVERHEAD) * tiles_of(s.n);
    } else {
      if (blockIdx.x == 0 && s.n != 0) set_flag(g.status, TTQ_FLAG_BAD_INDEX);
      s.n = 0;
    }
    seqs[b] = pack(w, s.n, s.kv, s.row0);
  }
  __syncthreads();
  if (warp == 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < g.batch; b0 += 32) {
      const int b = b0 + lane;
      const int4 q = b < g.batch ? seqs[b] : make_int4(0, 0, 0, 0);
      int64_t v = end_of(q);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < g.batch) seqs[b] = pack(base + v, q.y >> 24, q.z, q.w);
      base += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int64_t total = g.batch > 0 ? end_of(seqs[g.batch - 1]) * g.kv_heads : 0;
  // no run shorter than a segment's overhead and 2 blocks a warp, so that short
  // contexts are not cut into pieces whose merge costs more than they do
  constexpr int LEAST = A::OVERHEAD + 2 * W;
  const int64_t most = (total + LEAST - 1) / LEAST;
  const int64_t runs = most < static_cast<int64_t>(gridDim.x) ? most : static_cast<int64_t>(gridDim.x);
  int4* meta = a.meta + 2 * blockIdx.x;
  if (tid == 0) meta[0] = make_int4(-1, 0, 0, 0);
  if (blockIdx.x >= runs) return;
  int64_t x = blockIdx.x * total / runs;
  const int64_t x1 = (blockIdx.x + 1) * total / runs;

  // ---- the segment at x; a segment's blocks follow A::OVERHEAD units of its
  // own cost, so a run that begins within those begins with its first block
  KvSegment seg;
  int from, tiles;
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
    const int64_t per_head_x = x / g.kv_heads;
    int lo = 0, hi = g.batch - 1;               // first b with end * kv_heads > x
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end_of(seqs[mid]) > per_head_x) hi = mid; else lo = mid + 1;
    }
    enter(lo);
    const int64_t rest = x - (lo > 0 ? end_of(seqs[lo - 1]) * g.kv_heads : 0);
    const int64_t units = seg.blocks + A::OVERHEAD, tile = rest / units;
    left = units - (rest - tile * units);
    seg.h = static_cast<int>(tile / tiles);
    seg.tile = static_cast<int>(tile - static_cast<int64_t>(seg.h) * tiles);
  }
  uint32_t phases = 0;                          // bit s: parity of stage s
  for (bool started = false; x < x1; started = true) {
    if (started && left == 0) {                 // the next segment
      if (++seg.tile == tiles) {
        seg.tile = 0;
        if (++seg.h == g.kv_heads) enter(seg.b + 1);
      }
      left = seg.blocks + A::OVERHEAD;
    }
    // blocks [from, from + count) of it are this run's; none if only a part
    // of its overhead is
    const int64_t take = x1 - x < left ? x1 - x : left;
    const int end = seg.blocks - static_cast<int>(left - take < seg.blocks ? left - take : seg.blocks);
    from = seg.blocks - static_cast<int>(left < seg.blocks ? left : seg.blocks);
    const int count = end - from;
    x += take;
    left -= take;
    if (count == 0) continue;
    const bool whole = from == 0 && count == seg.blocks;
    const int old = seg.kv - seg.n;             // positions before the new ones
    const int R = seg.n * a.per, r0 = seg.tile * ROWS;
    if (started) {
      // the ring was the merge buffer: order those accesses before the copies
      fence_proxy_async_smem();
      __syncthreads();
    }

    // ---- start this warp's copies: blocks from + warp, + W, ...
    const int mine = count > warp ? (count - warp + W - 1) / W : 0;
    auto block_of = [&](int i) { return seg.first + from + warp + i * W; };
    int page_of_lane = -1;                      // page of this warp's block 32 k + lane
    auto load_pages = [&](int i0) {
      const int i = i0 + lane;
      page_of_lane = i < mine ? g.table[seg.b * g.table_stride + block_of(i) / g.page_blocks] : -1;
    };
    auto issue = [&](int i) {                   // by the whole warp
      const int page = __shfl_sync(0xffffffffu, page_of_lane, i & 31);
      if (lane == 0) {
        const int s = i % STAGES;
        uint64_t* bar = &bars[warp * STAGES + s];
        if (page >= 0 && page < g.num_pages) {
          const uint8_t* src = g.pages + page * g.page_bytes +
                               (static_cast<int64_t>(seg.h) * g.page_blocks + block_of(i) % g.page_blocks) * F::BLOCK;
          absent[warp * STAGES + s] = 0;
          mbar_arrive_expect_tx(bar, F::BLOCK);
          bulk_load(smem_addr(ring + s * F::BLOCK), src, F::BLOCK, bar);
        } else {
          absent[warp * STAGES + s] = 1;
          set_flag(g.status, TTQ_FLAG_BAD_INDEX);
          mbar_arrive(bar);
        }
      }
    };
    load_pages(0);
    int issued = 0;
    for (; issued < STAGES && issued < mine; ++issued) issue(issued);

    // ---- the tile's rows of Q as B fragments, and what each row sees
    {
      constexpr int E = HD / 32;                // consecutive channels of a lane
      constexpr int RW = ROWS / W;              // rows of a warp
      float v[RW][E];
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int rr = r0 + warp * RW + k;
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = 0.f;
        if (rr < R) {
          const int i_new = rr / a.per;
          kv_load_lane<E>(a.Q, a.q_type,
                          (seg.row0 + i_new) * a.q_row + (seg.h * a.per + rr - i_new * a.per) * a.q_head + lane * E, v[k]);
        }
      }
      float dk[E];
#pragma unroll
      for (int e = 0; e < E; ++e) dk[e] = a.Dk != nullptr ? __ldg(a.Dk + seg.h * HD + lane * E + e) : 1.f;
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int r = warp * RW + k;
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[k][e] *= dk[e];
          big = fmaxf(big, fabsf(v[k][e]));
        }
        // the row's largest magnitude: bits of non-negative floats order as integers
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);   // 2^-(ex - 127)
        const float up = __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int c = lane * E + e, kg = c / F::G, j = c % F::G;
          const int quarter = j / (F::G / 4), idx = kg * (F::G / 4) + j % (F::G / 4);
          qfrag[(((r >> 3) * KS + idx / 4) * 32 + 4 * (r & 7) + quarter) * 2 + (idx % 4) / 2] =
              h2_as_u32(__floats2half2_rn(v[k][e] * down, v[k][e + 1] * down));
        }
        if (lane == 0) q_factor[r] = a.scale * up * (a.cap > 0.f ? 1.f / a.cap : kKvLog2e);
      }
      if (tid < ROWS) {
        const int rr = r0 + tid, i_new = rr / a.per;
        uint64_t mask = 0;
        if (rr < R) mask = a.tree != nullptr ? a.tree[seg.row0 + i_new] : (2ull << i_new) - 1ull;
        row_mask[tid] = mask;
        row_pos[tid] = old + __popcll(mask & ~(1ull << (i_new & 63)));
      }
      if (tid >= 64 && tid - 64 < seg.n) {
        const int i = tid - 64;
        const uint64_t mask = a.tree != nullptr ? a.tree[seg.row0 + i] : (2ull << i) - 1ull;
        new_pos[i] = old + __popcll(mask & ~(1ull << i));
      }
    }
    __syncthreads();

    // ---- the loop over this warp's blocks
    float o[MT][NT][4] = {};
    float m[NT][2], l[NT][2] = {};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = kKvFloor;
    int e_run = 0;                              // running exponent field of V's scales
    bool ok = true;

    auto process = [&](auto masked_c, uint32_t st, int blk, bool gone) {
      constexpr bool MASKED = decltype(masked_c)::value;
      // -- scores
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      uint32_t kw[2][WORDS];
      kv_lane_words<F::LB, F::PIECE>(st, lane, 0, kw[0]);
      kv_lane_words<F::LB, F::PIECE>(st, lane, 1, kw[1]);
      uint32_t kp[2][NG];
      kv_lds<NG>(st + F::CODES + gr * NG * 4, kp[0]);
      kv_lds<NG>(st + F::CODES + (gr + 8) * NG * 4, kp[1]);
      constexpr int KSG = KS / NG;              // k steps of a group
      constexpr int KSW = BITS == 8 ? 1 : 32 / BITS / 4;   // k steps of a word
      uint32_t pa[2][2 * KSW];
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
        KvZero<BITS> z[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) z[r].set(__byte_perm(kp[r][k], 0, 0x3232));
#pragma unroll
        for (int j = 0; j < KSG; ++j) {
          const int ks = k * KSG + j, w = ks / KSW, in = ks % KSW;
          if (in == 0 || j == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (BITS == 8) {
                kv_e4m3x4(kw[r][w], pa[r][0], pa[r][1]);
              } else {
                kv_int_pairs<BITS>(kw[r][w], z[r], pa[r]);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 bq = *reinterpret_cast<const uint2*>(qfrag + ((nt * KS + ks) * 32 + lane) * 2);
            kv_mma(acc[nt], pa[0][2 * in], pa[1][2 * in], pa[0][2 * in + 1], pa[1][2 * in + 1], bq.x, bq.y);
          }
        }
        const float s0 = __half2float(u32_as_h2(kp[0][k]).x), s1 = __half2float(u32_as_h2(kp[1][k]).x);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] = fmaf(acc[nt][0], s0, s[nt][0]);
          s[nt][1] = fmaf(acc[nt][1], s0, s[nt][1]);
          s[nt][2] = fmaf(acc[nt][2], s1, s[nt][2]);
          s[nt][3] = fmaf(acc[nt][3], s1, s[nt][3]);
        }
      }
      // -- V's words; of a block that is not all there, tokens that are not are zeroed
      uint32_t vw[2][WORDS];
      kv_lane_words<F::LB, F::PIECE>(st + F::V_OFFSET, lane, 0, vw[0]);
      kv_lane_words<F::LB, F::PIECE>(st + F::V_OFFSET, lane, 1, vw[1]);
      uint32_t vp[2][NG], vz[2][NG];            // (s, z) of tokens gr, gr + 8; zeros of 2 tq, 2 tq + 1 (+ 8)
      const uint32_t vpairs = st + F::V_OFFSET + F::CODES;
      kv_lds<NG>(vpairs + gr * NG * 4, vp[0]);
      kv_lds<NG>(vpairs + (gr + 8) * NG * 4, vp[1]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t e0[NG], e1[NG];
        kv_lds<NG>(vpairs + (2 * tq + 8 * r) * NG * 4, e0);
        kv_lds<NG>(vpairs + (2 * tq + 1 + 8 * r) * NG * 4, e1);
#pragma unroll
        for (int k = 0; k < NG; ++k) vz[r][k] = __byte_perm(e0[k], e1[k], 0x7632);
      }
      const int there = MASKED ? (gone ? 0 : seg.kv - blk * 16) : 16;   // tokens of the block
      if constexpr (MASKED) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t0 = 2 * tq + 8 * r;
          const uint32_t keep = (t0 < there ? 0xFFFFu : 0u) | (t0 + 1 < there ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int w = 0; w < WORDS; ++w) vw[r][w] &= keep;
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            vz[r][k] &= keep;
            if (gr + 8 * r >= there) vp[r][k] = 0;
          }
        }
      }
      // -- the largest finite scale's exponent, over all of the block's V
      {
        uint32_t sb = 0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const uint32_t bits = vp[r][k] & 0x7FFFu;
            sb = max(sb, bits < 0x7C00u ? bits : 0u);
          }
        const int e_new = static_cast<int>(__reduce_max_sync(0xffffffffu, sb) >> 10);
        if (e_new > e_run) {
          const float f = __uint_as_float(static_cast<uint32_t>(127 + e_run - e_new) << 23);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[mt][nt][i] *= f;
          e_run = e_new;
        }
      }
      // -- scores in powers of two, masks
      bool higher = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float f0 = q_factor[8 * nt + 2 * tq], f1 = q_factor[8 * nt + 2 * tq + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float t = s[nt][i] * ((i & 1) ? f1 : f0);
          if (a.cap > 0.f)    // cap tanh(t) = cap (1 - 2 / (1 + e^{2 t}))
            t = a.cap * kKvLog2e * (1.f - 2.f * kv_rcp(1.f + kv_exp2(t * (2.f * kKvLog2e))));
          if constexpr (MASKED) {
            const int j = (i & 2) ? gr + 8 : gr, p = blk * 16 + j, row = 8 * nt + 2 * tq + (i & 1);
            bool see = j < there;
            if (see && p >= old) {
              see = (row_mask[row] >> (p - old)) & 1ull;
              if (a.window > 0) see = see && row_pos[row] - new_pos[p - old] < a.window;
            } else if (see && a.window > 0) {
              see = row_pos[row] - p < a.window;
            }
            t = see ? t : -INFINITY;
          }
          s[nt][i] = t;
          higher |= t > m[nt][i & 1] + kKvSlack;
        }
      }
      // -- the running maximum moves only when a score is well above it
      if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(s[nt][c], s[nt][c + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(m[nt][c], mx);
            const float f = kv_exp2(m[nt][c] - m_new);
            m[nt][c] = m_new;
            l[nt][c] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][nt][c] *= f;
              o[mt][nt][c + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[nt][i] = kv_exp2(s[nt][i] - m[nt][i & 1]);
          l[nt][i & 1] += s[nt][i];
        }
      // -- p s_V 2^-E as the B operand, and the second product
      const float vf = __uint_as_float(static_cast<uint32_t>(127 + 14 - e_run) << 23);   // s 2^(14 - e) < 1
      constexpr int MTG = MT / NG;              // m tiles of a group
      constexpr int MTW = BITS == 8 ? 1 : 16 / BITS / 2;   // m tiles of a word
      uint32_t pv[2][BITS == 8 ? 2 : 16 / BITS];
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const float s0 = __half2float(u32_as_h2(vp[0][k]).x) * vf, s1 = __half2float(u32_as_h2(vp[1][k]).x) * vf;
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w0 = s[nt][0] * s0, w1 = s[nt][1] * s0, w2 = s[nt][2] * s1, w3 = s[nt][3] * s1;
          if constexpr (MASKED) {               // a NaN scale reaches only those that see its token
            w0 = s[nt][0] == 0.f ? 0.f : w0;
            w1 = s[nt][1] == 0.f ? 0.f : w1;
            w2 = s[nt][2] == 0.f ? 0.f : w2;
            w3 = s[nt][3] == 0.f ? 0.f : w3;
          }
          b[nt][0] = kv_transpose(h2_as_u32(__floats2half2_rn(w0, w1)));
          b[nt][1] = kv_transpose(h2_as_u32(__floats2half2_rn(w2, w3)));
        }
        KvZero<BITS> z[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) z[r].set(vz[r][k]);
#pragma unroll
        for (int j = 0; j < MTG; ++j) {
          const int mt = k * MTG + j, w = mt / MTW, in = mt % MTW;
          if (in == 0 || j == 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (BITS == 8) {        // bytes: even token's two channels, then the odd one's
                kv_e4m3x4(__byte_perm(vw[r][w], 0, 0x3120), pv[r][0], pv[r][1]);
              } else {
                kv_int_pairs<BITS>(vw[r][w], z[r], pv[r]);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            kv_mma(o[mt][nt], pv[0][2 * in], pv[0][2 * in + 1], pv[1][2 * in], pv[1][2 * in + 1], b[nt][0], b[nt][1]);
        }
      }
    };

    int done = 0;
    for (; done < mine; ++done) {
      const int i = done, s = i % STAGES;
      if (!mbar_wait(&bars[warp * STAGES + s], (phases >> s) & 1u, &abort_flag)) {
        ok = false;
        break;
      }
      phases ^= 1u << s;
      const int blk = block_of(i);
      const bool gone = absent[warp * STAGES + s] != 0;
      const uint32_t st = smem_addr(ring + s * F::BLOCK);
      // masks matter in blocks that reach the new tokens, or that the window
      // of the last new token does not cover
      const bool masked = gone || blk * 16 + 16 > old ||
                          (a.window > 0 && blk * 16 <= static_cast<int64_t>(seg.kv) - 1 - a.window);
      if (masked) process(std::true_type{}, st, blk, gone);
      else process(std::false_type{}, st, blk, false);
      __syncwarp();
      if (issued < mine) {
        if ((issued & 31) == 0) load_pages(issued);
        issue(issued);
        ++issued;
      }
    }
    if (!ok) {
      // a copy did not arrive in time: say so and wait, with the same limit,
      // for the copies still in flight
      if (lane == 0) {
        set_flag(g.status, TTQ_FLAG_TIMEOUT);
        abort_flag = 1;
        for (int i = done; i < issued; ++i) {
          int never = 0;
          mbar_wait(&bars[warp * STAGES + i % STAGES], (phases >> (i % STAGES)) & 1u, &never);
        }
      }
      __syncwarp();
    }

    // ---- merge the warps' states
    const float back = __uint_as_float(static_cast<uint32_t>(127 + e_run - 14) << 23);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[nt][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (gr == 0) {
          warp_m[warp][8 * nt + 2 * tq + c] = m[nt][c];
          warp_l[warp][8 * nt + 2 * tq + c] = v;
        }
      }
    __syncthreads();                            // every warp is done with the ring
    const bool failed = *static_cast<volatile int*>(&abort_flag) != 0;
    float* buf = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2) {
          // channels of this lane: 2 mt, 2 mt + 1, 2 mt + 2, 2 mt + 3 of its stream
          const int k = 2 * mt / (F::G / 8), j = 2 * mt % (F::G / 8);
          const int ch = k * F::G + gr * (F::G / 8) + j;
          *reinterpret_cast<float4*>(buf + (warp * ROWS + 8 * nt + 2 * tq + c) * A::LDO + ch) =
              make_float4(o[mt][nt][c] * back, o[mt][nt][c + 2] * back, o[mt + 1][nt][c] * back,
                          o[mt + 1][nt][c + 2] * back);
        }
    __syncthreads();
    // this run's slot of the workspace: the first if the segment began in an
    // earlier run
    float* slot = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (from > 0 ? 0 : 1)) * A::SLOT;
    for (int i = tid; i < ROWS * (HD / 4); i += W * 32) {
      const int r = i / (HD / 4), ch = (i % (HD / 4)) * 4;
      if (r0 + r >= R) continue;
      float mx = warp_m[0][r];
#pragma unroll
      for (int w = 1; w < W; ++w) mx = fmaxf(mx, warp_m[w][r]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = kv_exp2(warp_m[w][r] - mx);
        const float4 v = *reinterpret_cast<const float4*>(buf + (w * ROWS + r) * A::LDO + ch);
        sum = fmaf(warp_l[w][r], f, sum);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      if (whole) {
        kv_store_row<HD>(a, seg.row0, seg.h, r0 + r, ch, acc, sum);
      } else {
        *reinterpret_cast<float4*>(slot + r * HD + ch) = acc;
        if (ch == 0) {
          slot[ROWS * HD + r] = mx;
          slot[ROWS * HD + ROWS + r] = sum;
        }
      }
    }
    if (tid == 0 && from == 0 && !whole) {
      // the run that holds the segment's last block: the last i with i total / runs <= its place
      const int64_t last = x + left - 1;
      meta[0] = make_int4(static_cast<int>(((last + 1) * runs - 1) / total), seg.row0, seg.h, r0);
      meta[1] = make_int4(R, 0, 0, 0);
    }
    if (failed) return;      // the same for all threads: set before the barriers above
  }
}

// Merges the partial results of the segment that began in run blockIdx.x and
// went on into later runs: a block takes one row, its threads are the float4
// channels of the row times slices of the partial results, which are
// summed per slice and then over the slices, always in the same order.
constexpr int kKvJoinThreads = 256;
template <int HD, int ROWS>
__global__ void __launch_bounds__(kKvJoinThreads) kv_join_kernel(const KvAttentionArgs a) {
  constexpr int SLOT = ROWS * (HD + 2), LANES = HD / 4, SLICES = kKvJoinThreads / LANES;
  __shared__ float4 acc_s[SLICES][LANES];
  __shared__ float sum_s[SLICES];
  allow_dependents_launch();
  grid_dependency_wait();
  const int4 m0 = a.meta[2 * blockIdx.x];
  if (m0.x < 0) return;
  const int R = a.meta[2 * blockIdx.x + 1].x;
  const int first = blockIdx.x, last = m0.x, row0 = m0.y, h = m0.z, r0 = m0.w, r = blockIdx.y;
  if (r0 + r >= R) return;
  const int slice = threadIdx.x / LANES, ch = (threadIdx.x % LANES) * 4;
  // partial result k of the segment is in the first slot of run first + k, but for k = 0
  auto slot_of = [&](int k) { return a.part + (2 * static_cast<int64_t>(first + k) + (k == 0 ? 1 : 0)) * SLOT; };
  const int n = last - first + 1;
  float mx = kKvFloor;
  for (int k = threadIdx.x; k < n; k += kKvJoinThreads) mx = fmaxf(mx, slot_of(k)[ROWS * HD + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  __shared__ float max_s[kKvJoinThreads / 32];
  if (threadIdx.x % 32 == 0) max_s[threadIdx.x / 32] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kKvJoinThreads / 32; ++w) mx = fmaxf(mx, max_s[w]);
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = slice; k < n; k += SLICES) {
    const float* slot = slot_of(k);
    const float4 v = *reinterpret_cast<const float4*>(slot + r * HD + ch);
    const float f = kv_exp2(slot[ROWS * HD + r] - mx);
    sum = fmaf(slot[ROWS * HD + ROWS + r], f, sum);
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  acc_s[slice][threadIdx.x % LANES] = acc;
  if (ch == 0) sum_s[slice] = sum;
  __syncthreads();
  if (slice != 0) return;
#pragma unroll
  for (int w = 1; w < SLICES; ++w) {
    const float4 v = acc_s[w][threadIdx.x];
    sum += sum_s[w];
    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
  }
  kv_store_row<HD>(a, row0, h, r0 + r, ch, acc, sum);
}

// One head size's kernels (a source file each).
cudaError_t kv_attention_hd64(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
cudaError_t kv_attention_hd128(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
cudaError_t kv_attention_hd256(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p, cudaStream_t s);
// Blocks per SM of the same kernels; 0 if the format is not built.
int kv_attention_ctas_hd64(int bits, int group, int nt);
int kv_attention_ctas_hd128(int bits, int group, int nt);
int kv_attention_ctas_hd256(int bits, int group, int nt);

// Calls f(BITS, NG, NT) as constants for one head size; false if not built.
template <int HD, typename Fn>
bool kv_with_format(int bits, int group, int nt, Fn&& f) {
  auto tiles = [&](auto BITSc, auto NGc) {
    if (nt == 1) return f(BITSc, NGc, std::integral_constant<int, 1>{}), true;
    if (nt == 2) return f(BITSc, NGc, std::integral_constant<int, 2>{}), true;
    if constexpr (HD <= 128)
      if (nt == 4) return f(BITSc, NGc, std::integral_constant<int, 4>{}), true;
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
int kv_attention_ctas(int bits, int group, int nt) {
  int n = 0;
  kv_with_format<HD>(bits, group, nt, [&](auto B, auto G, auto N) {
    n = KvAttention<HD, decltype(B)::value, decltype(G)::value, decltype(N)::value>::CTAS;
  });
  return n;
}

template <int HD>
cudaError_t kv_attention_launch(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p,
                                cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  kv_with_format<HD>(bits, group, p.nt, [&](auto Bc, auto Gc, auto Nc) {
    constexpr int BITS = decltype(Bc)::value, NG = decltype(Gc)::value, NT = decltype(Nc)::value;
    using A = KvAttention<HD, BITS, NG, NT>;
    auto* kernel = kv_attention_kernel<HD, BITS, NG, NT>;
    const int smem = A::SMEM + 16 * a.g.batch;
    static std::atomic<uint64_t> set{0};   // devices (a bit each) whose limit was raised
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(set.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, A::SMEM + 16 * kKvMaxBatch);
      if (e != cudaSuccess) return;
      set.fetch_or(bit, std::memory_order_relaxed);
    }
    e = launch_kernel(kernel, dim3(p.grid), dim3(A::W * 32), smem, stream, true, a);
    if (e != cudaSuccess) return;
    e = launch_kernel(kv_join_kernel<HD, A::ROWS>, dim3(p.grid, A::ROWS), dim3(kKvJoinThreads), 0, stream, true, a);
  });
  return e;
}

}  // namespace ttq
