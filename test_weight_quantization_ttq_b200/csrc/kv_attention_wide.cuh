// Attention over the quantised cache for many rows of a key/value head
// (trees of drafted tokens of grouped heads): a tile of 256 rows, on tcgen05.
//
// kv_attention.cuh says what is computed, how the work is cut and how the
// parts are merged; this is one thread block's part of a segment.  There a
// tile of 8 to 32 rows costs a warp the unpacking of every block's codes;
// here a block of 16 tokens is unpacked once for 256 rows, and a thread has a
// row of its own, so that maxima and sums need no shuffles.  A step is 64
// tokens, which two kinds of warps pass on:
//   8 unpack the K or the V part of one of its four blocks into binary16
//     operands (c - z, exact) in shared memory, rows of 128 bytes with their
//     16-byte chunks swizzled: K [64 tokens][channels], V [channels][64
//     tokens] with the channels of a group in the order e 8 + a for channel
//     a g / 8 + e, in which the lanes' stores have no bank conflicts.  A
//     thread of the first of them issues S_k = Q K_k^T for each group k of
//     channels (2 x 128 x 64; K's scales alone are left for the scores) and
//     O_k += P_k V_k, all in tensor memory;
//   8 (a thread a row) take S_k from tensor memory, s_K and the group sum,
//     cap, masks and exponentials, and put P_k = p s_V as binary16 into
//     shared memory.  O moves with the rows' offsets there (rarely: see
//     kKvSlack).
// The operands are in two buffers, and S too where tensor memory holds it
// (one group), so that the next step's scores and unpacking overlap this
// one's softmax.
// Measured: trees of 64 over 16384 positions of E4M3, cap, 256 rows: 134 us
// (8 tiles of 32: 170); trees of 24, 192 rows: 75 us (84).  Bound by the
// latency of the softmax's steps, not by a pipe (tensor pipe 13 to 14% busy,
// instructions issued in 40 to 46% of the cycles; the longest wait, a third, is
// for loads from tensor and global memory).  Both 128-row halves move in step,
// through the same barriers.  When these two took 138 and 76 us, two threads a
// row (138 and 80), tiles of 128 rows (136 and 92) and warps that sleep while
// they wait (143 and 100) were not better.
#pragma once

#include "kv_device.cuh"
#include "ttq_kernels.h"

namespace ttq {

template <int HD, int BITS, int NG>
struct KvWide {
  using F = KvFormat<HD, BITS, NG>;
  static constexpr int W = 16;                      // 8 of softmax, 8 that unpack; the first of these issues
  static constexpr int ROWS = 256, STEP = 64, TILES = ROWS / 128;
  static constexpr int LDO = HD + 4;                // padded row of the results in shared memory
  static constexpr int CTAS = 1, STAGES = 1;
  static constexpr int SB = NG == 1 ? 2 : 1;        // buffers of S
  static constexpr int QB = 128 * HD * 2, KB = STEP * HD * 2, VB = HD * STEP * 2, PB = 128 * STEP * 2;
  static constexpr int K_AT = TILES * QB, V_AT = K_AT + 2 * KB, P_AT = V_AT + 2 * VB;
  static constexpr int REGION = P_AT + TILES * NG * PB;     // the operands; at the end of a part the results
  static constexpr int WARP_BYTES = REGION;
  static constexpr int TABLE = 2 * 2 * NG * STEP * 4 + 2 * 4 * 4;   // scales of K and V, absent blocks: two steps'
  static constexpr int QFRAG = 0, ROWINFO = ROWS * 16 + TABLE;
  static constexpr int SMEM = 1024 + REGION + ROWINFO;
  static constexpr int O_AT = TILES * SB * NG * STEP;   // in tensor memory: S [buffer][tile][group], O [tile]
  static constexpr int COLUMNS = O_AT + TILES * HD <= 256 ? 256 : 512;
  static_assert(O_AT + TILES * HD <= 512, "tensor memory");
  static constexpr int MOST = 13;                   // results merged at a time: there are 148 at most
  static_assert(ROWS * LDO * 4 <= REGION && (MOST * (2 * ROWS + 1) + ROWS) * 4 <= REGION, "what the region holds");
  static constexpr int SLOT = ROWS * (HD + 4);
  // what a segment costs besides its blocks, in blocks (16 / 32 / 64: trees of
  // 24 over 8 contexts of 4099 85 / 76 / 84 us, trees of 32 over 16 of up to
  // 2000 88 / 85 / 99), and the least a run has
  static constexpr int OVERHEAD = 32, LEAST = 12;
};

// The barriers of a thread block.
struct KvWideBars {
  uint64_t op_full[2], op_free[2], s_full[2], s_free[2], p_full, pv_done, drain;
};

__device__ __forceinline__ void tmem_store_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
         "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void kv_sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void kv_sts32(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}

// What the threads of a block share over its parts.
template <int HD, int BITS, int NG>
struct KvWidePart {
  using A = KvWide<HD, BITS, NG>;
  using F = typename A::F;
  const KvAttentionArgs& a;
  KvWideBars& bars;
  int* abort_flag;
  uint8_t* region;           // 1024-byte aligned
  uint64_t* row_mask;
  float* q_factor;
  int* row_pos;
  float *s_k, *s_v;          // [2][NG][64]
  int* gone;                 // [2][4]
  uint32_t tmem;
  // of the part
  int b, h, row0, n, kv, old, blk0, count, steps, here, r0, plain0, plain1;
  int turn0;                 // steps before it

  // Bounded waits: of one thread, and of a warp whose lanes all go on or none.
  __device__ __forceinline__ bool wait_one(uint64_t* bar, int parity) const {
    if (mbar_wait(bar, parity & 1, abort_flag)) return true;
    *static_cast<volatile int*>(abort_flag) = 1;
    set_flag(a.g.status, TTQ_FLAG_TIMEOUT);
    return false;
  }
  __device__ __forceinline__ bool wait(uint64_t* bar, int parity) const {
    return __all_sync(0xffffffffu, wait_one(bar, parity));
  }

  // The rows of Q as the A operand, scaled by powers of two; by all warps.
  __device__ __forceinline__ void rows(int tid, float factor) const {
    constexpr int E = HD / 32, N = 4;
    const int warp = tid >> 5, lane = tid & 31, R = n * a.per;
    if (tid < A::ROWS) {
      const int rr = min(r0 + tid, R - 1), i_new = rr / a.per;
      const uint64_t mask = kv_new_tokens(a, row0, n, i_new);
      row_mask[tid] = mask;
      row_pos[tid] = old + __popcll(mask & ~(1ull << i_new));
    }
    const bool wide = a.q_type == kRowF32;
    float dk[E];
#pragma unroll
    for (int e = 0; e < E; ++e) dk[e] = a.Dk != nullptr ? __ldg(a.Dk + h * HD + lane * E + e) : 1.f;
    const uint8_t* q = static_cast<const uint8_t*>(a.Q) + lane * (wide ? 4 * E : 2 * E);
#pragma unroll 1
    for (int r1 = warp; r1 < A::ROWS; r1 += N * A::W) {
      uint32_t raw[N][E];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int rr = min(r0 + r1 + k * A::W, R - 1), i_new = rr / a.per;
        const int64_t at = static_cast<int64_t>(row0 + i_new) * a.q_row + static_cast<int64_t>(h * a.per + rr - i_new * a.per) * a.q_head;
        if (wide) kv_load_words<E>(q + at * 4, raw[k]);
        else kv_load_words<E / 2>(q + at * 2, raw[k]);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int r = r1 + k * A::W;
        if (r >= A::ROWS) break;
        float v[E], big = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t w = raw[k][e / 2];
          const float bf = __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
          const float hf = __half2float(e & 1 ? u32_as_h2(w).y : u32_as_h2(w).x);
          const float x = wide ? __uint_as_float(raw[k][e]) : a.q_type == kRowBF16 ? bf : hf;
          v[e] = r < here ? x * dk[e] : 0.f;
          big = fmaxf(big, fabsf(v[e]));
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);   // 2^-(ex - 127)
        const int c = lane * E;                  // its first channel
        const uint32_t at = smem_addr(region) + r / 128 * A::QB + c / 64 * (128 * 128) + r % 128 * 128 + (((c % 64 / 8) ^ (r & 7)) << 4) + c % 8 * 2;
#pragma unroll
        for (int e = 0; e < E; e += 2) kv_sts32(at + 2 * e, h2_as_u32(__floats2half2_rn(v[e] * down, v[e + 1] * down)));
        if (lane == 0) q_factor[r] = kv_row_factor(factor, ex);
      }
    }
    fence_proxy_async_smem();
  }

  // The codes and pairs that a lane takes of a part (K or V) of a block.
  struct Raw {
    uint32_t w[2][F::LB / 4], pair[2][2][NG];
    bool gone;
  };
  // where block j of the part is; a page number that is not one is looked at
  // when its block is due
  __device__ __forceinline__ int page_of(int j) const {
    if (j >= count) return -1;
    return __ldg(a.g.table + b * a.g.table_stride + a.g.page_of(blk0 + j));
  }
  __device__ __forceinline__ void load(int j, int page, int which, Raw& x) const {
    const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
    x.gone = !(page >= 0 && page < a.g.num_pages) || j >= count;
    if (x.gone) {
#pragma unroll
      for (int i = 0; i < 2 * (F::LB / 4); ++i) x.w[i / (F::LB / 4)][i % (F::LB / 4)] = 0;
#pragma unroll
      for (int i = 0; i < 4 * NG; ++i) x.pair[i / (2 * NG)][i / NG % 2][i % NG] = 0;
      if (j < count && lane == 0) set_flag(a.g.status, TTQ_FLAG_BAD_INDEX);
      return;
    }
    const int blk = blk0 + j, pg = a.g.page_of(blk);
    const uint8_t* part = a.g.pages + page * a.g.page_bytes +
                          (static_cast<int64_t>(h) * a.g.page_blocks + (blk - pg * a.g.page_blocks)) * F::BLOCK + which * F::V_OFFSET;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      kv_load_codes<F>(part, lane, r, x.w[r]);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const int tok = which == 0 ? gr + 8 * r : 2 * tq + p + 8 * r;
          x.pair[r][p][i] = *reinterpret_cast<const uint32_t*>(part + F::CODES + (tok * NG + i) * 4);
        }
    }
  }

  // Warp u of those that unpack: block u / 2 of every step, its K or V.
  __device__ __forceinline__ void unpack(int u) const {
    constexpr int G = F::G, WORDS = F::LB / 4;
    const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3, j0 = u >> 1, which = u & 1;
    const KvMagic<BITS> magic;
    Raw next;
    int page = page_of(j0);
    load(j0, page, which, next);
    page = page_of(j0 + 4);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int T = turn0 + i, s = T & 1, j = 4 * i + j0;
      Raw x = next;
      if (i + 1 < steps) {
        load(j + 4, page, which, next);
        page = page_of(j + 8);
      }
      if (T >= 2 && !wait(&bars.op_free[s], (T >> 1) - 1)) return;
      if (which == 0) {
        if (lane == 0) gone[s * 4 + j0] = x.gone;
        const uint32_t to = smem_addr(region) + A::K_AT + s * A::KB;
        constexpr int C = G / 4, FW = BITS == 8 ? 4 : 32 / BITS;   // a lane's codes of a group, codes of a word
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const int tok = j0 * 16 + gr + 8 * r;
            if (tq == 0) s_k[(s * NG + k) * A::STEP + tok] = __half2float(u32_as_h2(x.pair[r][0][k]).x);
            KvZero<BITS> z;
            z.set(__byte_perm(x.pair[r][0][k], 0, 0x3232));
            uint32_t v[C / 2];
#pragma unroll
            for (int e0 = k * C / FW * FW; e0 < (k + 1) * C; e0 += FW) {
              uint32_t p[FW / 2];
              if constexpr (BITS == 8) kv_e4m3x4(x.w[r][e0 / FW], p[0], p[1]);
              else kv_int_pairs<BITS>(x.w[r][e0 / FW], z, magic, p);
#pragma unroll
              for (int e = e0; e < e0 + FW; e += 2)
                if (e >= k * C && e < (k + 1) * C) v[(e - k * C) / 2] = p[(e - e0) / 2];
            }
#pragma unroll
            for (int m = 0; m < C / 8; ++m) {
              const int c = k * G + tq * C + 8 * m;
              kv_sts128(to + c / 64 * (A::STEP * 128) + tok * 128 + (((c % 64 / 8) ^ gr) << 4), v[4 * m], v[4 * m + 1],
                        v[4 * m + 2], v[4 * m + 3]);
            }
          }
      } else {
        const int there = x.gone ? 0 : min(kv - (blk0 + j) * 16, 16);
        const uint32_t to = smem_addr(region) + A::V_AT + s * A::VB;
        constexpr int C = G / 8, U = 16 / BITS;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t0 = 2 * tq + 8 * r;
          if (there < 16) {                      // tokens that are not there count for nothing, whatever their bytes are
            const uint32_t keep = (t0 < there ? 0xFFFFu : 0u) | (t0 + 1 < there ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) x.w[r][i] &= keep;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int k = 0; k < NG; ++k)
                if (t0 + p >= there) x.pair[r][p][k] = 0;
          }
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            if (gr == 0)
              *reinterpret_cast<float2*>(s_v + (s * NG + k) * A::STEP + j0 * 16 + t0) =
                  make_float2(__half2float(u32_as_h2(x.pair[r][0][k]).x), __half2float(u32_as_h2(x.pair[r][1][k]).x));
            KvZero<BITS> z;
            z.set(__byte_perm(x.pair[r][0][k], x.pair[r][1][k], 0x7632));
            const uint32_t at = to + (k * G + gr) * 128 + (((j0 * 2 + r) ^ gr) << 4) + 4 * tq;
#pragma unroll
            for (int e0 = k * C / U * U; e0 < (k + 1) * C; e0 += U) {
              uint32_t p[U];
              if constexpr (BITS == 8) kv_e4m3x4(__byte_perm(x.w[r][e0 / U], 0, 0x3120), p[0], p[1]);
              else kv_int_pairs<BITS>(x.w[r][e0 / U], z, magic, p);
#pragma unroll
              for (int e = e0; e < e0 + U; ++e)
                if (e >= k * C && e < (k + 1) * C) kv_sts32(at + (e - k * C) * 1024, p[e - e0]);
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.op_full[s]);
      // (this warp's next unpacking waits for the product before this step's anyway)
      if (u == 0 && __any_sync(0xffffffffu, lane == 0 && !(first(i) && (i == 0 || second(i - 1))))) return;
    }
    if (u == 0 && lane == 0) second(steps - 1);
  }

  // The products, by one thread: step i's S, and step i's P V.
  __device__ __forceinline__ bool first(int i) const {
    constexpr uint32_t DESC = idesc_f16kind(kFmtF16, 128, A::STEP);
    const uint32_t base = smem_addr(region);
    const int T = turn0 + i, s = T & 1, sb = T % A::SB;
    if (!wait_one(&bars.op_full[s], T >> 1) || (T >= A::SB && !wait_one(&bars.s_free[sb], T / A::SB - 1))) return false;
    tc_fence_after_sync();
#pragma unroll
    for (int tile = 0; tile < A::TILES; ++tile)
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int j = 0; j < F::G / 16; ++j) {
          const int c = k * F::G + 16 * j;       // channels
          mma_f16kind_ss(tmem + ((sb * A::TILES + tile) * NG + k) * A::STEP,
                         smem_desc_sw128(base + tile * A::QB + c / 64 * (128 * 128)) + c % 64 / 8,
                         smem_desc_sw128(base + A::K_AT + s * A::KB + c / 64 * (A::STEP * 128)) + c % 64 / 8, DESC, j > 0);
        }
    mma_commit(&bars.s_full[sb]);
    return true;
  }
  __device__ __forceinline__ bool second(int i) const {
    constexpr uint32_t DESC = idesc_f16kind(kFmtF16, 128, F::G);
    const uint32_t base = smem_addr(region), o = tmem + A::O_AT;
    const int T = turn0 + i, s = T & 1;
    if (!wait_one(&bars.p_full, T)) return false;
    tc_fence_after_sync();
#pragma unroll
    for (int tile = 0; tile < A::TILES; ++tile)
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int j = 0; j < A::STEP / 16; ++j)
          mma_f16kind_ss(o + tile * HD + k * F::G, smem_desc_sw128(base + A::P_AT + (tile * NG + k) * A::PB) + 2 * j,
                         smem_desc_sw128(base + A::V_AT + s * A::VB + k * F::G * 128) + 2 * j, DESC, i > 0 || j > 0);
    mma_commit(&bars.op_free[s]);
    mma_commit(&bars.pv_done);
    return true;
  }

  // The softmax of row r, by its thread.  Leaves the part's results in the
  // region (its rows of LDO floats), *m_out and *l_out.
  __device__ __forceinline__ void softmax(int r, float* m_out, float* l_out) const {
    constexpr int G = F::G, N = A::STEP;
    const int lane = threadIdx.x & 31, tile = r >> 7, r7 = r & 127;
    const uint32_t lanes = static_cast<uint32_t>(r7 & ~31) << 16;
    const uint32_t o = tmem + lanes + A::O_AT + tile * HD;
    const float f = q_factor[r];
    float off = 0.f, l = 0.f;                   // the row's offset and sum as kv_attention.cuh has them
    bool seen = false;                          // whether the offset is a token's
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      const int T = turn0 + i, s = T & 1, sb = T % A::SB;
      if (!wait(&bars.op_full[s], T >> 1) || !wait(&bars.s_full[sb], T / A::SB)) return;
      tc_fence_after_sync();
      float t[N];
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          uint32_t x[16];
          tmem_load_16(tmem + lanes + ((sb * A::TILES + tile) * NG + k) * A::STEP + c, x);
          tmem_load_wait(x);
          const float4* sk = reinterpret_cast<const float4*>(s_k + (s * NG + k) * A::STEP + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = sk[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = __uint_as_float(x[4 * j + e]), sc = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
              t[c + 4 * j + e] = k == 0 ? y * sc : fmaf(y, sc, t[c + 4 * j + e]);
            }
          }
        }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_free[sb]);
      // -- scores
      if (a.cap > kKvFineCap) {
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = kv_cap(t[j] * f, a.cap, true) - off;
      } else if (a.cap > 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = kv_cap(t[j] * f, a.cap, false) - off;
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = fmaf(t[j], f, -off);
      }
      // -- masks: the tokens that this row sees
      const int j0 = 4 * i;
      const int4 away = *reinterpret_cast<const int4*>(gone + s * 4);
      const bool masked = j0 < plain0 || j0 + 4 > plain1 || j0 + 4 > count || (away.x | away.y | away.z | away.w) != 0;
      if (masked) {
        uint64_t vis = 0;
#pragma unroll 1
        for (int j = 0; j < 4 && j0 + j < count; ++j)
          if (!gone[s * 4 + j])
            vis |= static_cast<uint64_t>(kv_visible(a, row0, old, kv, blk0 + j0 + j, row_mask[r], row_pos[r])) << (16 * j);
        const uint32_t half[2] = {static_cast<uint32_t>(vis), static_cast<uint32_t>(vis >> 32)};
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (!(half[j / 32] >> (j % 32) & 1u)) t[j] = -INFINITY;
      }
      // -- the offset moves only when a t + e is well above it (and to the
      // first); whether one may is asked of the largest score and scale (NaN
      // aside) first
      float most[4] = {t[0], t[1], t[2], t[3]}, top = kKvLeastScale;
#pragma unroll
      for (int j = 4; j < N; ++j) most[j % 4] = fmaxf(most[j % 4], t[j]);
      const float high = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
#pragma unroll
      for (int k = 0; k < NG; ++k)
        top = fmaxf(top, fmaxf(s_v[(s * NG + k) * A::STEP + lane], s_v[(s * NG + k) * A::STEP + 32 + lane]));
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      const bool move = !seen || high + kv_exponent(top) > kKvSlack;
      if (T > 0 && !wait(&bars.pv_done, T - 1)) return;   // O is at rest, P is free
      if (__any_sync(0xffffffffu, move)) {
        float up = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float sc = kKvLeastScale;
#pragma unroll
          for (int k = 0; k < NG; ++k) sc = fmaxf(sc, s_v[(s * NG + k) * A::STEP + j]);
          up = fmaxf(up, t[j] + kv_exponent(sc));
        }
        if (!(up > -INFINITY) || (seen && up <= kKvSlack)) up = 0.f;   // (a row by its own tokens)
        const float g = seen ? kv_exp2(-up) : 1.f;   // (before the first token l and O are zero, or NaN)
        seen = seen || high > -INFINITY;
        off += up;
        l *= g;
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] -= up;
        if (i > 0) {
          tc_fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            uint32_t x[16];
            tmem_load_16(o + c, x);
            tmem_load_wait(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * g);
            tmem_store_16(o + c, x);
          }
          tmem_store_wait();
        }
      }
      float sum[4] = {};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        t[j] = kv_exp2(t[j]);
        sum[j % 4] += t[j];
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // -- P
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int c = 0; c < N / 8; ++c) {
          const float4* sv = reinterpret_cast<const float4*>(s_v + (s * NG + k) * A::STEP + 8 * c);
          const float4 v0 = sv[0], v1 = sv[1];
          float w[8] = {t[8 * c] * v0.x,     t[8 * c + 1] * v0.y, t[8 * c + 2] * v0.z, t[8 * c + 3] * v0.w,
                        t[8 * c + 4] * v1.x, t[8 * c + 5] * v1.y, t[8 * c + 6] * v1.z, t[8 * c + 7] * v1.w};
          if (masked) {                          // a NaN scale reaches only those that see its token
#pragma unroll
            for (int e = 0; e < 8; ++e) kv_zero_with(w[e], t[8 * c + e]);
          }
          kv_sts128(smem_addr(region) + A::P_AT + (tile * NG + k) * A::PB + r7 * 128 + ((c ^ (r & 7)) << 4),
                    h2_as_u32(__floats2half2_rn(w[0], w[1])), h2_as_u32(__floats2half2_rn(w[2], w[3])),
                    h2_as_u32(__floats2half2_rn(w[4], w[5])), h2_as_u32(__floats2half2_rn(w[6], w[7])));
        }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full);
    }
    if (!wait(&bars.pv_done, turn0 + steps - 1)) return;   // all products of the part are done
    tc_fence_after_sync();
    *m_out = seen ? off : kKvFloor;
    *l_out = l;
    float* to = reinterpret_cast<float*>(region) + r * A::LDO;
#pragma unroll
    for (int c = 0; c < HD; c += 16) {
      uint32_t x[16];
      tmem_load_16(o + c, x);
      tmem_load_wait(x);
#pragma unroll
      for (int e = 0; e < 8; ++e)                // column k g + 8 j + e is channel k g + e g / 8 + j
        *reinterpret_cast<float2*>(to + c / G * G + e * (G / 8) + c % G / 8) =
            make_float2(__uint_as_float(x[e]), __uint_as_float(x[8 + e]));
    }
    tc_fence_before_sync();
  }
};

}  // namespace ttq
