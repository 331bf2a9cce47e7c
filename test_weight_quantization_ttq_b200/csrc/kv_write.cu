// Rows of keys and values into the paged cache (ttq_kv_write): kv_rows.cuh.
#include "kv_rows.cuh"

namespace ttq {
namespace {

// A group's scale and zero from its range; flags gets what it shows.
struct KvGroup {
  float inv;
  uint32_t pair;       // (scale, zero) as two binary16
  int z;
  bool bad;            // nothing stands for it: a NaN scale says so
};
template <int BITS, bool SYM>
__device__ __forceinline__ KvGroup group_of(float mn, float mx, uint32_t& flags) {
  constexpr int QMAX = (1 << BITS) - 1;
  KvGroup k;
  // the range; of the symmetric schemes the largest magnitude (mn is 0)
  const float range = __fsub_rn(mx, mn);
  float s32;
  if constexpr (BITS == 8) s32 = div_by_const<448>(range);
  else s32 = div_by_const<SYM ? (1 << (BITS - 1)) - 1 : QMAX>(range);
  if (!(s32 >= 6.103515625e-05f)) s32 = 6.103515625e-05f;   // 2^-14
  const __half s16 = __float2half_ru(s32);
  const float s = __half2float(s16);
  const bool nan = !(range <= 3.402823466e38f), ovf = !(s <= 65504.f);
  k.bad = nan || ovf;
  if (k.bad) flags |= TTQ_FLAG_NONFINITE | (ovf && !nan ? TTQ_FLAG_SCALE_OVERFLOW : 0u);
  k.inv = __frcp_rn(s);
  // rint of the exact product: a fused multiply-add with 1.5 * 2^23 rounds
  // it to an integer, ties to even, read from the low fraction bits
  k.z = 0;
  if constexpr (BITS != 8)
    k.z = SYM ? 1 << (BITS - 1) : min(max(__float_as_int(__fmaf_rn(-mn, k.inv, 12582912.0f)) - 0x4B400000, 0), QMAX);
  k.pair = static_cast<uint32_t>(__half_as_ushort(s16)) |
           static_cast<uint32_t>(__half_as_ushort(__int2half_rn(k.z))) << 16;
  if (k.bad) k.pair = 0x7FFFu, k.z = 0;
  return k;
}

// Three-input minimum and maximum that keep a NaN.
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A lane's values of one token, as pairs of adjacent channels, times h; and
// the range of N pairs of them, joined over the lanes whose numbers differ
// in the bits of LANES.
template <int N>
__device__ __forceinline__ void scale_values(float2 (&x)[N], const float* h) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 f = *reinterpret_cast<const float4*>(h + 2 * i);
    x[i] = __fmul2_rn(x[i], make_float2(f.x, f.y));
    x[i + 1] = __fmul2_rn(x[i + 1], make_float2(f.z, f.w));
  }
}
template <bool ABS, int N, int LANES>
__device__ __forceinline__ void range_of(const float2* x, float& mn, float& mx) {
  mn = mx = 0.f;                                 // ABS: the largest magnitude alone, in mx
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (ABS) {
      mx = max3_nan(mx, fabsf(x[i].x), fabsf(x[i].y));
    } else {
      mn = min3_nan(mn, x[i].x, x[i].y);
      mx = max3_nan(mx, x[i].x, x[i].y);
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (!(LANES & o)) continue;
    if constexpr (!ABS) mn = kv_min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = kv_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
}

// The groups of N ranges that all of 2^k lanes know (lane number `me` among
// them, LANES apart in the warp): each lane forms one (or N / 2^k), and they
// tell each other.  store(n, pair) keeps the pair of group n.
template <int BITS, bool SYM, int N, int COUNT, int APART, typename Store>
__device__ __forceinline__ void share_groups(const float (&mn)[N], const float (&mx)[N], int me, KvGroup (&q)[N],
                                             uint32_t& flags, Store&& store) {
  const int lane = threadIdx.x & 31, first = lane - me * APART;
#pragma unroll
  for (int n0 = 0; n0 < N; n0 += COUNT) {
    float a = mn[n0], b = mx[n0];
#pragma unroll
    for (int n = 1; n < COUNT && n0 + n < N; ++n)
      if (me % (N < COUNT ? N : COUNT) == n) a = mn[n0 + n], b = mx[n0 + n];
    const int own = n0 + me % (N < COUNT ? N : COUNT);
    uint32_t f = 0;
    const KvGroup k = group_of<BITS, SYM>(a, b, f);
    if (me < N && store(own, k.pair)) flags |= f;
#pragma unroll
    for (int n = 0; n < COUNT && n0 + n < N; ++n) {
      const int from = first + n * APART;
      q[n0 + n].inv = __shfl_sync(0xffffffffu, k.inv, from);
      const int zb = __shfl_sync(0xffffffffu, k.bad ? -1 : k.z, from);
      q[n0 + n].bad = zb < 0;
      q[n0 + n].z = max(zb, 0);
    }
  }
}

// rint of the exact products of a pair with inv, in the low fraction bits.
__device__ __forceinline__ float2 rint_pair(float2 x, float inv) {
  return __ffma2_rn(x, make_float2(inv, inv), make_float2(12582912.0f, 12582912.0f));   // 1.5 * 2^23
}
// The codes of two rounded values (their zeros in the halves of z), in the
// halves of a word: rint(x inv) + z is never below 0 for a finite group, so
// the top alone is clamped.
template <int BITS>
__device__ __forceinline__ uint32_t int_codes(float a, float b, uint32_t z) {
  constexpr uint32_t QQ = ((1u << BITS) - 1) * 0x00010001u;
  return __viaddmin_s16x2(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410), z, QQ);
}
// Two E4M3 codes, of a pair times inv.
__device__ __forceinline__ uint32_t e4m3_codes(float2 x, float inv) {
  return __nv_cvt_float2_to_fp8x2(__fmul2_rn(x, make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
}

// N words of a lane's half to their pieces.
template <typename F, int N>
__device__ __forceinline__ void store_words(uint8_t* part, int lane, int half, const uint32_t (&w)[N]) {
  constexpr int PW = F::PIECE / 4;
#pragma unroll
  for (int c = 0; c < N / PW; ++c) {
    uint8_t* p = part + (c * 2 + half) * 32 * F::PIECE + lane * F::PIECE;
    if constexpr (PW == 1) *reinterpret_cast<uint32_t*>(p) = w[c];
    else if constexpr (PW == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[2 * c], w[2 * c + 1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}
// N pairs of consecutive values of a row in shared memory.
template <int TYPE, int N>
__device__ __forceinline__ void load_values(const uint8_t* p, float2* x) {
  if constexpr (TYPE == kRowF32) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 v = reinterpret_cast<const float4*>(p)[i / 2];
      x[i] = make_float2(v.x, v.y);
      x[i + 1] = make_float2(v.z, v.w);
    }
  } else {
    uint32_t w[N];
    if constexpr (N == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      x[i] = TYPE == kRowBF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                              : __half22float2(u32_as_h2(w[i]));
  }
}

// A warp's shared memory: tiles of 16 rows (two up to 256 bytes a row: the
// next part's rows are on their way while this one's are quantised), and
// sqrt(D) of its head.  Rows of 512 bytes take one tile and three blocks an SM;
// at 80 registers heads of 256 spill, and of 6000 rows of 8 such heads two
// blocks were faster (INT4 g64 27.6 us, 19.9 with two; E4M3 24.9 and 20.0), as
// were two tiles in one block (20.6, 20.2): the choice for them is open.
template <int HD, int TYPE>
struct WriteTile {
  static constexpr int ROW_BYTES = HD * (TYPE == kRowF32 ? 4 : 2), ROW = ROW_BYTES + 16;   // padded
  static constexpr int TILES = ROW_BYTES <= 256 ? 2 : 1;
  static constexpr int TILE = 16 * ROW, WARP = TILES * TILE + HD * 4;
  // thread blocks per SM by shared memory
  static constexpr int CTAS = 222 * 1024 / (kWarps * WARP) >= 3 ? 3 : 222 * 1024 / (kWarps * WARP) >= 2 ? 2 : 1;
};

template <int HD, int BITS, int NG, bool SYM, int TYPE>
__global__ void __launch_bounds__(kThreads, WriteTile<HD, TYPE>::CTAS) kv_write_kernel(const KvWriteArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  using S = WriteTile<HD, TYPE>;
  constexpr int G = F::G, WORDS = F::LB / 4;
  extern __shared__ __align__(128) uint8_t smem[];
  allow_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, tq = lane & 3;
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  uint8_t* tiles = smem + warp * S::WARP;
  int4* seqs = reinterpret_cast<int4*>(smem + kWarps * S::WARP);
  const int64_t total = static_cast<int64_t>(schedule(g, seqs)) * g.kv_heads * 2;
  // sqrt(D) of the head that this warp is at, as the lanes take it: a warp
  // keeps its head where the grid allows (see the launch)
  float* h_tab = reinterpret_cast<float*>(tiles + S::TILES * S::TILE);
  int h_of = -1;
  uint32_t flags = 0;
  // the rows of a part into tile s; tokens that have none are zero.  (Bulk
  // copies, one a row, were slower: each is issued for one lane at a time, and
  // 16 of them took some 300 instructions of 1100.)
  auto fetch = [&](const KvTask& k, int s) {
    constexpr int LANES = S::ROW_BYTES / 16, STEP = LANES < 32 ? 32 / LANES : 1;   // tokens of a pass
    const int64_t stride = a.row[k.which] * (S::ROW_BYTES / HD);
    const uint32_t rows = (1u << k.hi) - (1u << k.lo);
#pragma unroll
    for (int c = 0; c < (LANES > 32 ? LANES / 32 : 1); ++c) {
      const int tok0 = lane / LANES, at = (c * 32 + lane) % LANES * 16;
      const uint32_t dst = smem_addr(tiles + s * S::TILE + tok0 * S::ROW + at);
      const uint8_t* x = static_cast<const uint8_t*>(a.x[k.which]) + k.h * a.head[k.which] * (S::ROW_BYTES / HD) +
                         (k.row + tok0) * stride + at;
#pragma unroll
      for (int i = 0; i < 16; i += STEP) {
        kv_copy16(dst + i * S::ROW, x, rows >> (tok0 + i) & 1);
        x += STEP * stride;
      }
    }
    kv_copy_commit();
  };
  KvWalk walk(g, total);
  KvTask next = {};
  if (walk.more()) {
    next = walk.task(g, seqs);
    if (S::TILES == 2) fetch(next, 0);
  }
#pragma unroll 1
  for (int turn = 0; walk.more(); ++turn) {
    const KvTask k = next;
    const int s = turn % S::TILES;
    __syncwarp();                                // everyone is done with the tile that is filled next
    if (S::TILES == 1) fetch(k, 0);
    walk.next();
    if (walk.more()) {
      next = walk.task(g, seqs);
      if (S::TILES == 2) fetch(next, (turn + 1) & 1);
    } else if (S::TILES == 2) {
      kv_copy_commit();                          // (an empty group: one is always behind the one waited for)
    }
    kv_copy_wait<S::TILES - 1>();
    __syncwarp();
    uint8_t* const part = part_of<F>(g, k);
    if (part == nullptr) continue;
    const uint8_t* tile = tiles + s * S::TILE;
    const bool scaled = a.D[k.which] != nullptr;
    if (scaled && h_of != 2 * k.h + k.which) {
      h_of = 2 * k.h + k.which;
      const float* D = a.D[k.which] + k.h * HD;
#pragma unroll
      for (int c = lane; c < HD; c += 32) {
        // K: the four quarters one after another, each with its part of all
        // groups; V: the eighths
        const int i = c / G, j = c % G, C = k.which == 0 ? G / 4 : G / 8;
        h_tab[j / C * (k.which == 0 ? HD / 4 : HD / 8) + i * C + j % C] = __fsqrt_rn(__ldg(D + c));
      }
      __syncwarp();
    }
    if (k.which == 0) {
      // K: this lane's quarter of every group of tokens gr and gr + 8
      constexpr int C = G / 8;                   // pairs of a group
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = gr + 8 * r;
        const bool is = tok >= k.lo && tok < k.hi;
        float2 x[NG * C];
#pragma unroll
        for (int i = 0; i < NG; ++i)
          load_values<TYPE, C>(tile + tok * S::ROW + (i * G + tq * 2 * C) * (S::ROW_BYTES / HD), x + i * C);
        if (scaled) scale_values(x, h_tab + tq * (HD / 4));
        uint32_t w[WORDS] = {};
        float mn[NG], mx[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) range_of<SYM || BITS == 8, C, 3>(x + i * C, mn[i], mx[i]);
        KvGroup qs[NG];
        share_groups<BITS, SYM, NG, 4, 1>(mn, mx, tq, qs, flags, [&](int n, uint32_t pair) {
          if (is) *reinterpret_cast<uint32_t*>(part + F::CODES + (tok * NG + n) * 4) = pair;
          return is;
        });
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const KvGroup q = qs[i];
          [[maybe_unused]] const uint32_t z = static_cast<uint32_t>(q.z) * 0x00010001u;
          if (q.bad) {                           // codes of zero
#pragma unroll
            for (int j = 0; j < C; ++j) x[i * C + j] = make_float2(0.f, 0.f);
          }
#pragma unroll
          for (int j = 0; j < C; ++j) {
            // a pair of channels is field j of a word's low and high half; E4M3: two bytes
            const int e = i * C + j;
            if constexpr (BITS == 8) {
              w[e / 2] += e4m3_codes(x[e], q.inv) << (e % 2 * 16);
            } else {
              constexpr int FW = 16 / BITS;
              const float2 n = rint_pair(x[e], q.inv);
              w[e / FW] += int_codes<BITS>(n.x, n.y, z) << (e % FW * BITS);
            }
          }
        }
        if (is) store_words<F, WORDS>(part, lane, r, w);
      }
    } else {
      // V: this lane's eighth of every group of tokens 2 tq, 2 tq + 1 (+ 8)
      constexpr int C = G / 16, U = 16 / BITS;   // pairs of a group; channels of a 16-bit unit
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = 2 * tq + 8 * r;
        const bool is[2] = {tok >= k.lo && tok < k.hi, tok + 1 >= k.lo && tok + 1 < k.hi};
        uint32_t w[WORDS] = {};
        float2 x[2][NG * C];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int i = 0; i < NG; ++i)
            load_values<TYPE, C>(tile + (tok + p) * S::ROW + (i * G + gr * 2 * C) * (S::ROW_BYTES / HD), x[p] + i * C);
          if (scaled) scale_values(x[p], h_tab + gr * (HD / 8));
        }
        float mn[2 * NG], mx[2 * NG];            // of token p, group i at 2 i + p
#pragma unroll
        for (int n = 0; n < 2 * NG; ++n) range_of<SYM || BITS == 8, C, 28>(x[n % 2] + n / 2 * C, mn[n], mx[n]);
        KvGroup qs[2 * NG];
        share_groups<BITS, SYM, 2 * NG, 8, 4>(mn, mx, gr, qs, flags, [&](int n, uint32_t pair) {
          const bool has = is[n % 2];
          if (has) *reinterpret_cast<uint32_t*>(part + F::CODES + ((tok + n % 2) * NG + n / 2) * 4) = pair;
          return has;
        });
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const KvGroup q[2] = {qs[2 * i], qs[2 * i + 1]};
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (q[p].bad) {                      // codes of zero
#pragma unroll
              for (int j = 0; j < C; ++j) x[p][i * C + j] = make_float2(0.f, 0.f);
            }
          [[maybe_unused]] const uint32_t z = static_cast<uint32_t>(q[0].z) | static_cast<uint32_t>(q[1].z) << 16;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            // both tokens' codes of a channel: the same field of the word's halves
            const int e = i * C + j;             // a pair of channels
            if constexpr (BITS == 8) {
              w[e] = __byte_perm(e4m3_codes(x[0][e], q[0].inv), e4m3_codes(x[1][e], q[1].inv), 0x5410);
            } else {
              const float2 n0 = rint_pair(x[0][e], q[0].inv), n1 = rint_pair(x[1][e], q[1].inv);
              const int f0 = 2 * e % U * BITS;
              w[2 * e / U] += int_codes<BITS>(n0.x, n1.x, z) << f0;
              w[2 * e / U] += int_codes<BITS>(n0.y, n1.y, z) << (f0 + BITS);
            }
          }
        }
        if (is[0] && is[1]) {
          store_words<F, WORDS>(part, lane, r, w);
        } else if (is[0] || is[1]) {
          // one token of the pair: its halves of the words, the other's stay
          const int p = is[1];
#pragma unroll
          for (int i = 0; i < WORDS; ++i)
            *reinterpret_cast<uint16_t*>(part + F::place(lane, r, i * 4 + 2 * p)) =
                static_cast<uint16_t>(p ? w[i] >> 16 : w[i]);
        }
      }
    }
  }
  if (flags) set_flag(g.status, flags);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, int hd, int bits, int group, bool symmetric,
                            int dtype, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto go = [&](auto SYMc, auto TYPEc) {
      constexpr bool SYM = decltype(SYMc)::value;
      constexpr int TYPE = decltype(TYPEc)::value;
      using S = WriteTile<HD, TYPE>;
      constexpr int bytes = kWarps * S::WARP;
      auto* k = kv_write_kernel<HD, BITS, NG, SYM, TYPE>;
      static std::atomic<uint64_t> set{0};
      if ((e = kv_allow_smem(reinterpret_cast<const void*>(k), bytes + 16 * kKvMaxBatch, set)) != cudaSuccess) return;
      const dim3 grid(part_grid(a.g, num_sms, S::CTAS));
      e = launch_kernel(k, grid, dim3(kThreads), bytes + 16 * a.g.batch, stream, true, a);
    };
    auto of_type = [&](auto SYMc) {
      if (dtype == kRowF32) go(SYMc, std::integral_constant<int, kRowF32>{});
      else if (dtype == kRowBF16) go(SYMc, std::integral_constant<int, kRowBF16>{});
      else go(SYMc, std::integral_constant<int, kRowF16>{});
    };
    if constexpr (BITS == 8) of_type(std::false_type{});
    else if (symmetric) of_type(std::true_type{});
    else of_type(std::false_type{});
  });
  return e;
}

}  // namespace ttq
