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

// The codes of two values, in the low and the high half of a word.
template <int BITS>
__device__ __forceinline__ uint32_t codes_of(float a, const KvGroup& ga, float b, const KvGroup& gb) {
  if constexpr (BITS == 8) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a, ga.inv), __fmul_rn(b, gb.inv)), __NV_SATFINITE, __NV_E4M3);
    return (ga.bad ? 0u : c & 0xFFu) | (gb.bad ? 0u : (c & 0xFF00u) << 8);
  } else {
    constexpr uint32_t QQ = ((1u << BITS) - 1) * 0x00010001u;
    const uint32_t n = __byte_perm(__float_as_uint(__fmaf_rn(a, ga.inv, 12582912.0f)),
                                   __float_as_uint(__fmaf_rn(b, gb.inv, 12582912.0f)), 0x5410);
    // rint(x inv) + z is never below 0 for a finite group: the top alone is clamped
    const uint32_t c = __viaddmin_s16x2(n, static_cast<uint32_t>(ga.z) | static_cast<uint32_t>(gb.z) << 16, QQ);
    return (ga.bad ? 0u : c & 0xFFFFu) | (gb.bad ? 0u : c & 0xFFFF0000u);
  }
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
// N consecutive values of a row (4 N of it at a time where they are 8 or more).
template <int TYPE, int N>
__device__ __forceinline__ void load_values(const void* p, int64_t at, float* x) {
  if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      float v[8];
      kv_load8<TYPE>(p, at + i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i + j] = v[j];
    }
  } else {
    static_assert(N == 4, "4 or a multiple of 8");
    if constexpr (TYPE == kRowF32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 h = __half22float2(u32_as_h2(w[i]));
        x[2 * i] = TYPE == kRowBF16 ? __uint_as_float(w[i] << 16) : h.x;
        x[2 * i + 1] = TYPE == kRowBF16 ? __uint_as_float(w[i] & 0xFFFF0000u) : h.y;
      }
    }
  }
}

template <int HD, int BITS, int NG, bool SYM, int TYPE>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  constexpr int G = F::G, WORDS = F::LB / 4;
  extern __shared__ int4 seqs[];
  allow_dependents_launch();
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
  const int64_t total = static_cast<int64_t>(schedule(g, seqs)) * g.kv_heads * 2;
  uint32_t flags = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < total;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    const KvTask k = task_of<F>(g, seqs, t);
    if (k.part == nullptr) continue;
    const float* D = a.D[k.which] != nullptr ? a.D[k.which] + k.h * HD : nullptr;
    const void* rows = a.x[k.which];
    const int64_t base = k.h * a.head[k.which];
    if (k.which == 0) {
      // K: this lane's quarter of every group of tokens gr and gr + 8
      constexpr int C = G / 4;
      float x[2][NG * C];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = gr + 8 * r;
        const bool is = tok >= k.lo && tok < k.hi;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (is) {
            load_values<TYPE, C>(rows, (k.row + tok) * a.row[0] + base + i * G + tq * C, x[r] + i * C);
          } else {
#pragma unroll
            for (int j = 0; j < C; ++j) x[r][i * C + j] = 0.f;
          }
        }
      }
      if (D != nullptr) {
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const float h = __fsqrt_rn(__ldg(D + i * G + tq * C + j));
            x[0][i * C + j] = __fmul_rn(x[0][i * C + j], h);
            x[1][i * C + j] = __fmul_rn(x[1][i * C + j], h);
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = gr + 8 * r;
        const bool is = tok >= k.lo && tok < k.hi;
        uint32_t w[WORDS] = {}, f = 0;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          float mn = 0.f, mx = 0.f;
#pragma unroll
          for (int j = 0; j < C; ++j) mn = kv_min_nan(mn, x[r][i * C + j]), mx = kv_max_nan(mx, x[r][i * C + j]);
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            mn = kv_min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = kv_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          }
          const KvGroup q = group_of<BITS, SYM>(mn, mx, f);
          if (is && tq == 0) *reinterpret_cast<uint32_t*>(k.part + F::CODES + (tok * NG + i) * 4) = q.pair;
#pragma unroll
          for (int j = 0; j < C; j += 2) {
            // a pair is a word's fields i of the low and of the high half; E4M3: two bytes
            const uint32_t c = codes_of<BITS>(x[r][i * C + j], q, x[r][i * C + j + 1], q);
            const int e = i * C + j;
            if constexpr (BITS == 8) w[e / 4] |= __byte_perm(c, 0, 0x4420) << (e % 4 * 8);
            else w[e / (32 / BITS)] |= c << (e % (32 / BITS) / 2 * BITS);
          }
        }
        if (is) {
          store_words<F, WORDS>(k.part, lane, r, w);
          flags |= f;
        }
      }
    } else {
      // V: this lane's eighth of every group of tokens 2 tq, 2 tq + 1 (+ 8)
      constexpr int C = G / 8, U = 16 / BITS;   // channels of a group; of a 16-bit unit
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = 2 * tq + 8 * r;
        const bool is[2] = {tok >= k.lo && tok < k.hi, tok + 1 >= k.lo && tok + 1 < k.hi};
        float x[2][NG * C];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            if (is[p]) {
              load_values<TYPE, C>(rows, (k.row + tok + p) * a.row[1] + base + i * G + gr * C, x[p] + i * C);
            } else {
#pragma unroll
              for (int j = 0; j < C; ++j) x[p][i * C + j] = 0.f;
            }
          }
        if (D != nullptr) {
#pragma unroll
          for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int j = 0; j < C; ++j) {
              const float h = __fsqrt_rn(__ldg(D + i * G + gr * C + j));
              x[0][i * C + j] = __fmul_rn(x[0][i * C + j], h);
              x[1][i * C + j] = __fmul_rn(x[1][i * C + j], h);
            }
        }
        uint32_t w[WORDS] = {};
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          KvGroup q[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            float mn = 0.f, mx = 0.f;
            uint32_t f = 0;
#pragma unroll
            for (int j = 0; j < C; ++j) mn = kv_min_nan(mn, x[p][i * C + j]), mx = kv_max_nan(mx, x[p][i * C + j]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mn = kv_min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
              mx = kv_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            q[p] = group_of<BITS, SYM>(mn, mx, f);
            if (is[p]) {
              flags |= f;
              if (gr == 0) *reinterpret_cast<uint32_t*>(k.part + F::CODES + ((tok + p) * NG + i) * 4) = q[p].pair;
            }
          }
#pragma unroll
          for (int j = 0; j < C; ++j) {
            // both tokens' codes of a channel: the same field of the word's halves
            const int e = i * C + j;
            w[e / U] |= codes_of<BITS>(x[0][e], q[0], x[1][e], q[1]) << (e % U * BITS);
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
  const dim3 grid(part_grid(a.g, num_sms, 4));
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto go = [&](auto SYMc) {
      constexpr bool SYM = decltype(SYMc)::value;
      auto* k = dtype == kRowF32    ? kv_write_kernel<HD, BITS, NG, SYM, kRowF32>
                : dtype == kRowBF16 ? kv_write_kernel<HD, BITS, NG, SYM, kRowBF16>
                                    : kv_write_kernel<HD, BITS, NG, SYM, kRowF16>;
      e = launch_kernel(k, grid, dim3(kThreads), 16 * a.g.batch, stream, true, a);
    };
    if constexpr (BITS == 8) go(std::false_type{});
    else if (symmetric) go(std::true_type{});
    else go(std::false_type{});
  });
  return e;
}

}  // namespace ttq
