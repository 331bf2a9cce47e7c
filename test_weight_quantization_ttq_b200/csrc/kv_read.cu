// Rows of keys and values back from the paged cache (ttq_kv_read): kv_rows.cuh.
#include "kv_rows.cuh"

namespace ttq {
namespace {

// Two codes' values less the zero, as float32: pair p of kv_int_pairs, or two E4M3.
__device__ __forceinline__ float2 floats_of(uint32_t p) { return __half22float2(u32_as_h2(p)); }

template <int HD, int BITS, int NG, int TYPE>
__global__ void __launch_bounds__(kThreads, HD == 256 || TYPE == kRowF32 ? 2 : 3) kv_read_kernel(const KvReadArgs a) {
  using F = KvFormat<HD, BITS, NG>;
  constexpr int G = F::G, WORDS = F::LB / 4, SIZE = TYPE == kRowF32 ? 4 : 2;
  constexpr int ROW = HD * SIZE + 16;            // padded row of a warp's tile
  extern __shared__ int4 seqs[];
  allow_dependents_launch();
  grid_dependency_wait();
  const KvGeometry& g = a.g;
  const int lane = threadIdx.x & 31, gr = lane >> 2, tq = lane & 3;
  const int64_t total = static_cast<int64_t>(schedule(g, seqs)) * g.kv_heads * 2;
  uint8_t* tile = reinterpret_cast<uint8_t*>(seqs + g.batch) + (threadIdx.x >> 5) * 16 * ROW;
  const KvMagic<BITS> magic;
  // C (4 or a multiple of 8) consecutive values of a token's row into the tile
  auto put = [&](int tok, int ch, auto& x) {
    constexpr int C = sizeof(x) / sizeof(x[0]);
    uint8_t* p = tile + tok * ROW + ch * SIZE;
    if constexpr (TYPE == kRowF32) {
#pragma unroll
      for (int i = 0; i < C; i += 4) *reinterpret_cast<float4*>(p + 4 * i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if constexpr (C == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(kv_pack2<TYPE>(x[0], x[1]), kv_pack2<TYPE>(x[2], x[3]));
    } else {
#pragma unroll
      for (int i = 0; i < C; i += 8)
        *reinterpret_cast<uint4*>(p + 2 * i) =
            make_uint4(kv_pack2<TYPE>(x[i], x[i + 1]), kv_pack2<TYPE>(x[i + 2], x[i + 3]),
                       kv_pack2<TYPE>(x[i + 4], x[i + 5]), kv_pack2<TYPE>(x[i + 6], x[i + 7]));
    }
  };
  KvWalk walk(g, total);
  KvTask next = {};
  if (walk.more()) next = walk.task(g, seqs);
#pragma unroll 1
  while (walk.more()) {
    const KvTask k = next;
    walk.next();
    if (walk.more()) next = walk.task(g, seqs);
    if (a.y[k.which] == nullptr) continue;
    const uint8_t* const part = part_of<F>(g, k);
    const float* Dr = a.Dr[k.which] != nullptr ? a.Dr[k.which] + k.h * HD : nullptr;
    __syncwarp();                                // the tile is free
    if (part != nullptr) {
      uint32_t w[2][WORDS], pair[2][2][NG];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        kv_load_codes<F>(part, lane, r, w[r]);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const int tok = k.which == 0 ? gr + 8 * r : 2 * tq + p + 8 * r;
            pair[r][p][i] = *reinterpret_cast<const uint32_t*>(part + F::CODES + (tok * NG + i) * 4);
          }
      }
      if (k.which == 0) {
        constexpr int C = G / 4, FW = BITS == 8 ? 4 : 32 / BITS;   // codes of a word
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float s = __half2float(u32_as_h2(pair[r][0][i]).x);
            KvZero<BITS> z;
            z.set(__byte_perm(pair[r][0][i], 0, 0x3232));
            float x[C];
#pragma unroll
            for (int e0 = i * C / FW * FW; e0 < (i + 1) * C; e0 += FW) {
              uint32_t p[FW / 2];
              if constexpr (BITS == 8) kv_e4m3x4(w[r][e0 / FW], p[0], p[1]);
              else kv_int_pairs<BITS>(w[r][e0 / FW], z, magic, p);
#pragma unroll
              for (int e = e0; e < e0 + FW; e += 2) {
                if (e < i * C || e >= (i + 1) * C) continue;   // (a word of two groups)
                // exact: 8 bits at most times 11
                const float2 v = __fmul2_rn(floats_of(p[(e - e0) / 2]), make_float2(s, s));
                x[e - i * C] = v.x;
                x[e - i * C + 1] = v.y;
              }
            }
            if (Dr != nullptr) {
#pragma unroll
              for (int j = 0; j < C; ++j) x[j] *= __ldg(Dr + i * G + tq * C + j);
            }
            put(gr + 8 * r, i * G + tq * C, x);
          }
      } else {
        constexpr int C = G / 8, U = 16 / BITS;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            const float s0 = __half2float(u32_as_h2(pair[r][0][i]).x), s1 = __half2float(u32_as_h2(pair[r][1][i]).x);
            KvZero<BITS> z;
            z.set(__byte_perm(pair[r][0][i], pair[r][1][i], 0x7632));
            float x[C], y[C];                    // of the even and of the odd token
#pragma unroll
            for (int e0 = i * C / U * U; e0 < (i + 1) * C; e0 += U) {
              uint32_t p[U];
              if constexpr (BITS == 8) kv_e4m3x4(__byte_perm(w[r][e0 / U], 0, 0x3120), p[0], p[1]);
              else kv_int_pairs<BITS>(w[r][e0 / U], z, magic, p);
#pragma unroll
              for (int e = e0; e < e0 + U; ++e) {
                if (e < i * C || e >= (i + 1) * C) continue;
                const float2 v = __fmul2_rn(floats_of(p[e - e0]), make_float2(s0, s1));
                x[e - i * C] = v.x;
                y[e - i * C] = v.y;
              }
            }
            if (Dr != nullptr) {
#pragma unroll
              for (int j = 0; j < C; ++j) {
                const float d = __ldg(Dr + i * G + gr * C + j);
                x[j] *= d;
                y[j] *= d;
              }
            }
            put(2 * tq + 8 * r, i * G + gr * C, x);
            put(2 * tq + 1 + 8 * r, i * G + gr * C, y);
          }
      }
    }
    __syncwarp();
    // the rows from the tile, 16 bytes a lane; of an absent page zeros
    constexpr int LANES = HD * SIZE / 16, STEP = LANES < 32 ? 32 / LANES : 1;   // tokens of a pass
    const int64_t stride = static_cast<int64_t>(g.kv_heads) * HD * SIZE;
#pragma unroll
    for (int c = 0; c < (LANES > 32 ? LANES / 32 : 1); ++c) {
      const int tok0 = lane / LANES, at = (c * 32 + lane) % LANES * 16;
      const uint8_t* from = tile + tok0 * ROW + at;
      uint8_t* y = static_cast<uint8_t*>(a.y[k.which]) + (k.row + tok0) * stride + k.h * HD * SIZE + at;
#pragma unroll
      for (int i = 0; i < 16; i += STEP) {
        const uint4 v = part != nullptr ? *reinterpret_cast<const uint4*>(from + i * ROW) : make_uint4(0, 0, 0, 0);
        if (tok0 + i >= k.lo && tok0 + i < k.hi) __stcs(reinterpret_cast<uint4*>(y), v);
        y += STEP * stride;
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_read(const KvReadArgs& a, int hd, int bits, int group, int dtype,
                           int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  const dim3 grid(part_grid(a.g, num_sms, hd == 256 || dtype == kRowF32 ? 2 : 3));
  with_format(hd, bits, group, [&](auto HDc, auto BITSc, auto NGc) {
    constexpr int HD = decltype(HDc)::value, BITS = decltype(BITSc)::value, NG = decltype(NGc)::value;
    auto go = [&](auto TYPEc) {
      constexpr int TYPE = decltype(TYPEc)::value;
      constexpr int bytes = kWarps * 16 * (HD * (TYPE == kRowF32 ? 4 : 2) + 16);
      auto* k = kv_read_kernel<HD, BITS, NG, TYPE>;
      // the leave is for the largest batch, whatever this call's is: another
      // thread may be between it and its launch
      static std::atomic<uint64_t> set{0};
      if ((e = kv_allow_smem(reinterpret_cast<const void*>(k), bytes + 16 * kKvMaxBatch, set)) != cudaSuccess) return;
      e = launch_kernel(k, grid, dim3(kThreads), bytes + 16 * a.g.batch, stream, true, a);
    };
    if (dtype == kRowF32) go(std::integral_constant<int, kRowF32>{});
    else if (dtype == kRowBF16) go(std::integral_constant<int, kRowBF16>{});
    else go(std::integral_constant<int, kRowF16>{});
  });
  return e;
}

}  // namespace ttq
