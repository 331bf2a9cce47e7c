// Writing rows of keys and values into the paged cache as group-wise codes,
// and reading them back (ttq_kv_write, ttq_kv_read).
//
// The quantiser is the layer's own, in the same binary32 order (bit-exact
// with ttq_quantize_weight_ex of the row as one row of a weight):
//   x = k sqrt(D); m = min(0, min x); M = max(0, max x) over the group;
//   s32 = (M - m) / (2^b - 1), at least 2^-14; s = binary16 round-up(s32);
//   inv = 1 / s; z = clamp(rint(-m inv)); q = clamp(rint(x inv) + z),
// rint of the exact product.  Symmetric and E4M3 codes likewise.
//
// Both kernels are bound by memory: a position of one head is 4 hd bytes of
// bf16 rows against 2 (hd b / 8 + 4 hd / g) bytes of cache.  A lane owns 8
// consecutive channels of one row of one head (16 bytes of a bf16 row); the
// g / 8 lanes of a group find its range by shuffles.
#include <type_traits>

#include "kv_device.cuh"
#include "ttq_kernels.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;

// The 8 codes of channels 8 i .. 8 i + 7 of a row, as bytes of the K and V
// parts.  idx: the first channel's group and its place there.
template <int HD, int BITS, int NG>
struct KvPlace {
  using F = KvFormat<HD, BITS, NG>;
  int k, r;   // group and channel within the group
  __device__ explicit KvPlace(int ch) : k(ch / F::G), r(ch % F::G) {}
  // K: lane and stream index of the first of the 8 codes (consecutive there)
  __device__ int k_lane(int tok) const { return 4 * (tok & 7) + r / (F::G / 4); }
  __device__ int k_index() const { return k * (F::G / 4) + r % (F::G / 4); }
  // V: the same for the quad of 4 channels r + 4 q
  __device__ int v_lane(int tok, int q) const { return 4 * ((r + 4 * q) / (F::G / 8)) + (tok & 7) / 2; }
  __device__ int v_index(int q) const { return k * (F::G / 8) + (r + 4 * q) % (F::G / 8); }
};

// Stores a row's 8 codes into its block.
template <int HD, int BITS, int NG>
__device__ __forceinline__ void store_codes(uint8_t* block, int which, int tok, int ch, const uint32_t (&q)[8]) {
  using F = KvFormat<HD, BITS, NG>;
  const KvPlace<HD, BITS, NG> at(ch);
  const int half = tok >> 3;
  if (which == 0) {
    const int lane = at.k_lane(tok), e = at.k_index();
    if constexpr (BITS == 8) {
      *reinterpret_cast<uint2*>(block + F::place(lane, half, e)) =
          make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
    } else if constexpr (BITS == 4) {
      *reinterpret_cast<uint32_t*>(block + F::place(lane, half, e / 2)) =
          q[0] | q[2] << 4 | q[4] << 8 | q[6] << 12 | q[1] << 16 | q[3] << 20 | q[5] << 24 | q[7] << 28;
    } else {
      // 8 of a word's 16 codes: the even channels in one byte of its low
      // half, the odd ones in the same byte of its high half
      uint8_t* w = block + F::place(lane, half, e / 16 * 4) + (e % 16) / 8;
      w[0] = static_cast<uint8_t>(q[0] | q[2] << 2 | q[4] << 4 | q[6] << 6);
      w[2] = static_cast<uint8_t>(q[1] | q[3] << 2 | q[5] << 4 | q[7] << 6);
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int lane = at.v_lane(tok, u), e = at.v_index(u);
    const uint32_t* c = q + 4 * u;
    const int odd = (tok & 1) * 2;
    if constexpr (BITS == 8) {
      *reinterpret_cast<uint16_t*>(block + F::place(lane, half, e * 2 + odd)) = static_cast<uint16_t>(c[0] | c[1] << 8);
      *reinterpret_cast<uint16_t*>(block + F::place(lane, half, e * 2 + 4 + odd)) = static_cast<uint16_t>(c[2] | c[3] << 8);
    } else if constexpr (BITS == 4) {
      *reinterpret_cast<uint16_t*>(block + F::place(lane, half, e + odd)) =
          static_cast<uint16_t>(c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12);
    } else {
      block[F::place(lane, half, e / 8 * 4 + odd + (e % 8) / 4)] =
          static_cast<uint8_t>(c[0] | c[1] << 2 | c[2] << 4 | c[3] << 6);
    }
  }
}

// A row's 8 codes as they stand in its block: one code per element.
template <int HD, int BITS, int NG>
__device__ __forceinline__ void load_codes(const uint8_t* block, int which, int tok, int ch, uint32_t (&q)[8]) {
  using F = KvFormat<HD, BITS, NG>;
  const KvPlace<HD, BITS, NG> at(ch);
  const int half = tok >> 3;
  if (which == 0) {
    const int lane = at.k_lane(tok), e = at.k_index();
    if constexpr (BITS == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(block + F::place(lane, half, e));
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = (w.x >> (8 * i)) & 255u, q[4 + i] = (w.y >> (8 * i)) & 255u;
    } else if constexpr (BITS == 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(block + F::place(lane, half, e / 2));
#pragma unroll
      for (int i = 0; i < 4; ++i) q[2 * i] = (w >> (4 * i)) & 15u, q[2 * i + 1] = (w >> (16 + 4 * i)) & 15u;
    } else {
      const uint8_t* w = block + F::place(lane, half, e / 16 * 4) + (e % 16) / 8;
      const uint32_t a = w[0], b = w[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[2 * i] = (a >> (2 * i)) & 3u, q[2 * i + 1] = (b >> (2 * i)) & 3u;
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int lane = at.v_lane(tok, u), e = at.v_index(u);
    uint32_t* c = q + 4 * u;
    const int odd = (tok & 1) * 2;
    if constexpr (BITS == 8) {
      const uint32_t a = *reinterpret_cast<const uint16_t*>(block + F::place(lane, half, e * 2 + odd));
      const uint32_t b = *reinterpret_cast<const uint16_t*>(block + F::place(lane, half, e * 2 + 4 + odd));
      c[0] = a & 255u, c[1] = a >> 8, c[2] = b & 255u, c[3] = b >> 8;
    } else if constexpr (BITS == 4) {
      const uint32_t a = *reinterpret_cast<const uint16_t*>(block + F::place(lane, half, e + odd));
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = (a >> (4 * i)) & 15u;
    } else {
      const uint32_t a = block[F::place(lane, half, e / 8 * 4 + odd + (e % 8) / 4)];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = (a >> (2 * i)) & 3u;
    }
  }
}

// Codes, scale and zero of the lane's 8 channels; the lanes of a group agree
// on its range.  flags gets what the group shows.
template <int BITS, int GL, bool SYM>   // GL: lanes of a group
__device__ __forceinline__ void quantise8(const float (&x)[8], uint32_t (&q)[8], uint32_t& pair, uint32_t& flags) {
  constexpr int QMAX = (1 << BITS) - 1;
  float mn = 0.f, mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) mn = kv_min_nan(mn, x[i]), mx = kv_max_nan(mx, x[i]);
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) {
    mn = kv_min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = kv_max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const float range = __fsub_rn(mx, mn);
  const float span = (BITS == 8 || SYM) ? kv_max_nan(mx, -mn) : range;
  float s32;
  if constexpr (BITS == 8) s32 = div_by_const<448>(span);
  else s32 = div_by_const<SYM ? (1 << (BITS - 1)) - 1 : QMAX>(span);
  if (!(s32 >= 6.103515625e-05f)) s32 = 6.103515625e-05f;
  const __half s16 = __float2half_ru(s32);
  const float s = __half2float(s16);
  const bool bad = !(range <= 3.402823466e38f), ovf = !(s <= 65504.f);
  if (bad || ovf) {
    // nothing of the group can be stood for: a NaN scale says so
    flags |= TTQ_FLAG_NONFINITE | (ovf && !bad ? TTQ_FLAG_SCALE_OVERFLOW : 0u);
    pair = 0x7FFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0;
    return;
  }
  const float inv = __frcp_rn(s);
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = __nv_cvt_float_to_fp8(__fmul_rn(x[i], inv), __NV_SATFINITE, __NV_E4M3);
    pair = __half_as_ushort(s16);
  } else {
    // rint of the exact product: a fused multiply-add with 1.5 * 2^23 rounds
    // it to an integer, ties to even, read from the low fraction bits
    const int zi = __float_as_int(__fmaf_rn(-mn, inv, 12582912.0f)) - 0x4B400000;
    const int z = SYM ? 1 << (BITS - 1) : min(max(zi, 0), QMAX);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = __float_as_int(__fmaf_rn(x[i], inv, 12582912.0f)) - 0x4B400000 + z;
      q[i] = static_cast<uint32_t>(min(max(n, 0), QMAX));
    }
    pair = static_cast<uint32_t>(__half_as_ushort(s16)) |
           (static_cast<uint32_t>(__half_as_ushort(__int2half_rn(z))) << 16);
  }
}

template <int HD, int BITS, int NG, bool SYM, int TYPE>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  constexpr int LANES = HD / 8;              // lanes of one row of one head
  allow_dependents_launch();
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  const int sub = threadIdx.x % LANES, ch = sub * 8;
  const int64_t tasks = g.rows * g.kv_heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / LANES);
  uint32_t flags = 0;
  // every lane of a warp takes part in the shuffles of every turn
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kThreads / LANES); t0 < tasks; t0 += step) {
    const int64_t t = t0 + threadIdx.x / LANES;
    const int64_t row = t / g.kv_heads;
    const int h = static_cast<int>(t - row * g.kv_heads);
    uint8_t* block = nullptr;
    int tok = 0;
    if (t < tasks) {
      const int b = kv_find_sequence(g, row);
      if (b >= 0) {
        KvSequence s;
        if (kv_sequence(g, b, s) && row >= s.row0 && row < s.row0 + s.n) {
          const int pos = s.kv - s.n + static_cast<int>(row - s.row0);
          block = kv_block(g, b, pos, h, F::BLOCK);
          tok = pos & 15;
        }
        if (block == nullptr) flags |= TTQ_FLAG_BAD_INDEX;
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[8] = {};
      if (block != nullptr) {
        kv_load8<TYPE>(a.x[which], row * a.row[which] + h * a.head[which] + ch, x);
        if (a.D[which] != nullptr) {
          const float* D = a.D[which] + h * HD + ch;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], __fsqrt_rn(__ldg(D + i)));
        }
      }
      uint32_t q[8], pair, f = 0;
      quantise8<BITS, F::G / 8, SYM>(x, q, pair, f);
      if (block != nullptr) {
        flags |= f;
        uint8_t* part = block + which * F::V_OFFSET;
        store_codes<HD, BITS, NG>(part, which, tok, ch, q);
        if (ch % F::G == 0)
          *reinterpret_cast<uint32_t*>(part + F::CODES + (tok * NG + ch / F::G) * 4) = pair;
      }
    }
  }
  if (flags) set_flag(g.status, flags);
}

template <int HD, int BITS, int NG, int TYPE>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  constexpr int LANES = HD / 8;
  allow_dependents_launch();
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  const int sub = threadIdx.x % LANES, ch = sub * 8;
  const int64_t tasks = g.rows * g.kv_heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / LANES);
  uint32_t flags = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES; t < tasks; t += step) {
    const int64_t row = t / g.kv_heads;
    const int h = static_cast<int>(t - row * g.kv_heads);
    const int b = kv_find_sequence(g, row);
    if (b < 0) continue;
    KvSequence s;
    if (!kv_sequence(g, b, s) || row < s.row0 || row >= s.row0 + s.n) {
      flags |= TTQ_FLAG_BAD_INDEX;
      continue;
    }
    const int pos = s.kv - s.n + static_cast<int>(row - s.row0), tok = pos & 15;
    const uint8_t* block = kv_block(g, b, pos, h, F::BLOCK);
    if (block == nullptr) flags |= TTQ_FLAG_BAD_INDEX;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (a.y[which] == nullptr) continue;
      float x[8] = {};
      if (block != nullptr) {
        const uint8_t* part = block + which * F::V_OFFSET;
        uint32_t q[8];
        load_codes<HD, BITS, NG>(part, which, tok, ch, q);
        const uint32_t pair = *reinterpret_cast<const uint32_t*>(part + F::CODES + (tok * NG + ch / F::G) * 4);
        const float2 sz = __half22float2(u32_as_h2(pair));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v;
          if constexpr (BITS == 8) v = __half2float(u32_as_h2(kv_e4m3x2(q[i])).x);
          else v = static_cast<float>(q[i]) - sz.y;
          x[i] = v * sz.x;     // exact: at most 8 bits times 11
          if (a.Dr[which] != nullptr) x[i] *= __ldg(a.Dr[which] + h * HD + ch + i);
        }
      }
      kv_store8<TYPE>(a.y[which], (row * g.kv_heads + h) * HD + ch, x);
    }
  }
  if (flags) set_flag(g.status, flags);
}

// Calls f with the format's constants; false if it is not built.
template <typename Fn>
bool with_format(int hd, int bits, int group, Fn&& f) {
  auto bits_of = [&](auto HDc, auto NGc) {
    if (bits == 2) return f(HDc, std::integral_constant<int, 2>{}, NGc), true;
    if (bits == 4) return f(HDc, std::integral_constant<int, 4>{}, NGc), true;
    if (bits == 8) return f(HDc, std::integral_constant<int, 8>{}, NGc), true;
    return false;
  };
  auto groups_of = [&](auto HDc) {
    const int ng = hd / group;
    if (ng == 1) return bits_of(HDc, std::integral_constant<int, 1>{});
    if (ng == 2) return bits_of(HDc, std::integral_constant<int, 2>{});
    if constexpr (decltype(HDc)::value >= 128)
      if (ng == 4) return bits_of(HDc, std::integral_constant<int, 4>{});
    return false;
  };
  if (hd == 64) return groups_of(std::integral_constant<int, 64>{});
  if (hd == 128) return groups_of(std::integral_constant<int, 128>{});
  if (hd == 256) return groups_of(std::integral_constant<int, 256>{});
  return false;
}

unsigned row_grid(int64_t tasks, int lanes, int num_sms) {
  const int64_t blocks = (tasks * lanes + kThreads - 1) / kThreads, most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, int hd, int bits, int group, bool symmetric,
                            int dtype, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  const dim3 grid(row_grid(a.g.rows * a.g.kv_heads, hd / 8, num_sms));
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto go = [&](auto SYMc) {
      constexpr bool SYM = decltype(SYMc)::value;
      auto* k = dtype == kRowF32    ? kv_write_kernel<HD, BITS, NG, SYM, kRowF32>
                : dtype == kRowBF16 ? kv_write_kernel<HD, BITS, NG, SYM, kRowBF16>
                                    : kv_write_kernel<HD, BITS, NG, SYM, kRowF16>;
      e = launch_kernel(k, grid, dim3(kThreads), 0, stream, true, a);
    };
    if constexpr (BITS == 8) go(std::false_type{});
    else if (symmetric) go(std::true_type{});
    else go(std::false_type{});
  });
  return e;
}

cudaError_t launch_kv_read(const KvReadArgs& a, int hd, int bits, int group, int dtype,
                           int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  const dim3 grid(row_grid(a.g.rows * a.g.kv_heads, hd / 8, num_sms));
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto* k = dtype == kRowF32    ? kv_read_kernel<HD, BITS, NG, kRowF32>
              : dtype == kRowBF16 ? kv_read_kernel<HD, BITS, NG, kRowBF16>
                                  : kv_read_kernel<HD, BITS, NG, kRowF16>;
    e = launch_kernel(k, grid, dim3(kThreads), 0, stream, true, a);
  });
  return e;
}

}  // namespace ttq
