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
  const float range = __fsub_rn(mx, mn);
  const float span = (BITS == 8 || SYM) ? kv_max_nan(mx, -mn) : range;
  float s32;
  if constexpr (BITS == 8) s32 = div_by_const<448>(span);
  else s32 = div_by_const<SYM ? (1 << (BITS - 1)) - 1 : QMAX>(span);
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
template <int N, int LANES>
__device__ __forceinline__ void range_of(const float2* x, float& mn, float& mx) {
  mn = mx = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mn = min3_nan(mn, x[i].x, x[i].y);
    mx = max3_nan(mx, x[i].x, x[i].y);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (!(LANES & o)) continue;
    mn = kv_min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = kv_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
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
// N pairs of consecutive values of a row.
template <int TYPE, int N>
__device__ __forceinline__ void load_values(const void* p, int64_t at, float2* x) {
  if constexpr (TYPE == kRowF32) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 2 * i));
      x[i] = make_float2(v.x, v.y);
      x[i + 1] = make_float2(v.z, v.w);
    }
  } else {
    uint32_t w[N];
    const uint16_t* s = static_cast<const uint16_t*>(p) + at;
    if constexpr (N == 2) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(s));
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(s + 2 * i));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      x[i] = TYPE == kRowBF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                              : __half22float2(u32_as_h2(w[i]));
  }
}

template <int HD, int BITS, int NG, bool SYM, int TYPE>
__global__ void __launch_bounds__(kThreads, HD == 256 ? 2 : 3) kv_write_kernel(const KvWriteArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  constexpr int G = F::G, WORDS = F::LB / 4;
  extern __shared__ int4 seqs[];
  allow_dependents_launch();
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
  const int64_t total = static_cast<int64_t>(schedule(g, seqs)) * g.kv_heads * 2;
  // sqrt(D) of the head that this warp is at, as the lanes take it: a warp
  // keeps its head where the grid allows (see the launch)
  float* h_tab = reinterpret_cast<float*>(seqs + g.batch) + (threadIdx.x >> 5) * HD;
  int h_of = -1;
  uint32_t flags = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < total;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const KvTask k = task_of<F>(g, seqs, t);
    if (k.part == nullptr) continue;
    const bool scaled = a.D[k.which] != nullptr;
    if (scaled && h_of != 2 * k.h + k.which) {
      h_of = 2 * k.h + k.which;
      const float* D = a.D[k.which] + k.h * HD;
      __syncwarp();
#pragma unroll
      for (int c = lane; c < HD; c += 32) {
        // K: the four quarters one after another, each with its part of all
        // groups; V: the eighths
        const int i = c / G, j = c % G, C = k.which == 0 ? G / 4 : G / 8;
        h_tab[j / C * (k.which == 0 ? HD / 4 : HD / 8) + i * C + j % C] = __fsqrt_rn(__ldg(D + c));
      }
      __syncwarp();
    }
    const int64_t base = k.h * a.head[k.which];
    if (k.which == 0) {
      // K: this lane's quarter of every group of tokens gr and gr + 8
      constexpr int C = G / 8;                   // pairs of a group
      float2 x[2][NG * C];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = gr + 8 * r;
        if (tok >= k.lo && tok < k.hi) {
          const int64_t at = (k.row + tok) * a.row[0] + base + tq * 2 * C;
#pragma unroll
          for (int i = 0; i < NG; ++i) load_values<TYPE, C>(a.x[0], at + i * G, x[r] + i * C);
        } else {
#pragma unroll
          for (int j = 0; j < NG * C; ++j) x[r][j] = make_float2(0.f, 0.f);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = gr + 8 * r;
        const bool is = tok >= k.lo && tok < k.hi;
        if (scaled) scale_values(x[r], h_tab + tq * (HD / 4));
        uint32_t w[WORDS] = {}, f = 0;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          float mn, mx;
          range_of<C, 3>(x[r] + i * C, mn, mx);
          const KvGroup q = group_of<BITS, SYM>(mn, mx, f);
          if (is && tq == 0) *reinterpret_cast<uint32_t*>(k.part + F::CODES + (tok * NG + i) * 4) = q.pair;
          const uint32_t z = static_cast<uint32_t>(q.z) * 0x00010001u;
          if (q.bad) {                           // codes of zero
#pragma unroll
            for (int j = 0; j < C; ++j) x[r][i * C + j] = make_float2(0.f, 0.f);
          }
#pragma unroll
          for (int j = 0; j < C; ++j) {
            // a pair of channels is field j of a word's low and high half; E4M3: two bytes
            const int e = i * C + j;
            if constexpr (BITS == 8) {
              w[e / 2] |= e4m3_codes(x[r][e], q.inv) << (e % 2 * 16);
            } else {
              constexpr int FW = 16 / BITS;
              const float2 n = rint_pair(x[r][e], q.inv);
              w[e / FW] |= int_codes<BITS>(n.x, n.y, z) << (e % FW * BITS);
            }
          }
        }
        if (is) {
          store_words<F, WORDS>(k.part, lane, r, w);
          flags |= f;
        }
      }
    } else {
      // V: this lane's eighth of every group of tokens 2 tq, 2 tq + 1 (+ 8)
      constexpr int C = G / 16, U = 16 / BITS;   // pairs of a group; channels of a 16-bit unit
      float2 x[2][2][NG * C];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int tok = 2 * tq + p + 8 * r;
          if (tok >= k.lo && tok < k.hi) {
            const int64_t at = (k.row + tok) * a.row[1] + base + gr * 2 * C;
#pragma unroll
            for (int i = 0; i < NG; ++i) load_values<TYPE, C>(a.x[1], at + i * G, x[r][p] + i * C);
          } else {
#pragma unroll
            for (int j = 0; j < NG * C; ++j) x[r][p][j] = make_float2(0.f, 0.f);
          }
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = 2 * tq + 8 * r;
        const bool is[2] = {tok >= k.lo && tok < k.hi, tok + 1 >= k.lo && tok + 1 < k.hi};
        uint32_t w[WORDS] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (scaled) scale_values(x[r][p], h_tab + gr * (HD / 8));
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          KvGroup q[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            float mn, mx;
            uint32_t f = 0;
            range_of<C, 28>(x[r][p] + i * C, mn, mx);
            q[p] = group_of<BITS, SYM>(mn, mx, f);
            if (q[p].bad) {                      // codes of zero
#pragma unroll
              for (int j = 0; j < C; ++j) x[r][p][i * C + j] = make_float2(0.f, 0.f);
            }
            if (is[p]) {
              flags |= f;
              if (gr == 0) *reinterpret_cast<uint32_t*>(k.part + F::CODES + ((tok + p) * NG + i) * 4) = q[p].pair;
            }
          }
          const uint32_t z = static_cast<uint32_t>(q[0].z) | static_cast<uint32_t>(q[1].z) << 16;
#pragma unroll
          for (int j = 0; j < C; ++j) {
            // both tokens' codes of a channel: the same field of the word's halves
            const int e = i * C + j;             // a pair of channels
            if constexpr (BITS == 8) {
              w[e] = __byte_perm(e4m3_codes(x[r][0][e], q[0].inv), e4m3_codes(x[r][1][e], q[1].inv), 0x5410);
            } else {
              const float2 n0 = rint_pair(x[r][0][e], q[0].inv), n1 = rint_pair(x[r][1][e], q[1].inv);
              const int f0 = 2 * e % U * BITS;
              w[2 * e / U] |= int_codes<BITS>(n0.x, n1.x, z) << f0 | int_codes<BITS>(n0.y, n1.y, z) << (f0 + BITS);
            }
          }
        }
        if (is[0] && is[1]) {
          store_words<F, WORDS>(k.part, lane, r, w);
        } else if (is[0] || is[1]) {
          // one token of the pair: its halves of the words, the other's stay
          const int p = is[1];
#pragma unroll
          for (int i = 0; i < WORDS; ++i)
            *reinterpret_cast<uint16_t*>(k.part + F::place(lane, r, i * 4 + 2 * p)) =
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
  const dim3 grid(part_grid(a.g, num_sms, hd == 256 ? 2 : 3));
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto go = [&](auto SYMc) {
      constexpr bool SYM = decltype(SYMc)::value;
      auto* k = dtype == kRowF32    ? kv_write_kernel<HD, BITS, NG, SYM, kRowF32>
                : dtype == kRowBF16 ? kv_write_kernel<HD, BITS, NG, SYM, kRowBF16>
                                    : kv_write_kernel<HD, BITS, NG, SYM, kRowF16>;
      e = launch_kernel(k, grid, dim3(kThreads), 16 * a.g.batch + kWarps * HD * 4, stream, true, a);
    };
    if constexpr (BITS == 8) go(std::false_type{});
    else if (symmetric) go(std::true_type{});
    else go(std::false_type{});
  });
  return e;
}

}  // namespace ttq
