// Device-side helpers of the key/value cache's kernels: where a token's
// codes are in a block, and where a row of the batch is in the cache.
//
// A block holds 16 tokens of one head as K codes, K (scale, zero) pairs, V
// codes, V pairs.  The codes stand as the lanes of a warp take them for the
// A operand of m16n8k16: lane 4 a + c of a K block has, of tokens a and
// a + 8 (its two halves), the channels r in [c g / 4, (c + 1) g / 4) of
// every group of g; lane 4 a + c of a V block has, of the channels r in
// [a g / 8, (a + 1) g / 8) of every group, the tokens 2 c, 2 c + 1 and 2 c + 8,
// 2 c + 9.  A lane's bytes of one half are cut into pieces of at most 16 bytes,
// and a piece of all lanes is contiguous, so that a warp reads it without
// bank conflicts.
#pragma once

#include <cuda_fp8.h>

#include <cstring>

#include "kv_kernels.h"
#include "ttq_device.cuh"

namespace ttq {

template <int HD, int BITS, int NG>
struct KvFormat {
  static constexpr int G = HD / NG;                     // channels of a group
  static constexpr int LB = HD * BITS / 32;             // a lane's bytes of one half
  static constexpr int PIECE = LB < 16 ? LB : 16;
  static constexpr int CODES = kv_code_bytes(HD, BITS);
  static constexpr int PAIRS = kv_pair_bytes(HD, G);
  static constexpr int BLOCK = 2 * (CODES + PAIRS);
  static constexpr int V_OFFSET = CODES + PAIRS;        // the V part within the block
  static_assert(BLOCK % 16 == 0, "a block is one bulk copy");

  static __device__ __forceinline__ int place(int lane, int half, int byte) {
    return ((byte / PIECE) * 2 + half) * 32 * PIECE + lane * PIECE + byte % PIECE;
  }
};

// Where the rows of the batch are.  Sequence b is valid when its rows lie in
// [0, rows), are at most max_new and kv_len, and kv_len fits its table.
struct KvSequence {
  int row0, n, kv;
};
__device__ __forceinline__ bool kv_sequence(const KvGeometry& g, int b, KvSequence& s) {
  const int c0 = g.cu[b], c1 = g.cu[b + 1];
  const int kv = g.kv_len[b];
  s.row0 = c0;
  s.n = c1 - c0;
  s.kv = kv;
  return c0 >= 0 && c1 >= c0 && c1 <= g.rows && c1 - c0 <= g.max_new && kv >= c1 - c0 &&
         kv <= g.table_stride * g.page_blocks * 16;
}

__device__ __forceinline__ uint32_t h2_as_u32(__half2 v) {
  uint32_t u;
  memcpy(&u, &v, 4);
  return u;
}
__device__ __forceinline__ __half2 u32_as_h2(uint32_t u) {
  __half2 v;
  memcpy(&v, &u, 4);
  return v;
}

// The two binary16 pairs of a word of four E4M3 codes: exact.
__device__ __forceinline__ void kv_e4m3x4(uint32_t v, uint32_t& p0, uint32_t& p1) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}" : "=r"(p0), "=r"(p1) : "r"(v));
}

// (w & MASK) | magic in one instruction: a LOP3 takes one constant, so the
// other has to be in a register (left to the compiler it becomes two).
template <uint32_t MASK>
__device__ __forceinline__ __half2 kv_field(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(magic));
  return u32_as_h2(r);
}

// The exponents under which the fields of a word's halves count as integers:
// 1024, 64, 256 and 16 plus the code.
template <int BITS>
struct KvMagic {
  uint32_t v[4];
  __device__ __forceinline__ KvMagic() {
    // kept opaque, so that they stay in registers
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(v[0]));
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(v[1]));
    if constexpr (BITS == 2) {
      asm volatile("mov.b32 %0, 0x5C005C00;" : "=r"(v[2]));
      asm volatile("mov.b32 %0, 0x4C004C00;" : "=r"(v[3]));
    }
  }
};

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
// low and of the high half; both steps are exact in binary16.
template <int BITS>
__device__ __forceinline__ void kv_int_pairs(uint32_t w, const KvZero<BITS>& z, const KvMagic<BITS>& c, uint32_t* p) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = i ? w >> 8 : w;
    if constexpr (BITS == 4) {
      p[2 * i] = h2_as_u32(__hsub2(kv_field<0x000F000Fu>(u, c.v[0]), z.o[0]));
      p[2 * i + 1] = h2_as_u32(__hsub2(kv_field<0x00F000F0u>(u, c.v[1]), z.o[1]));
    } else {
      p[4 * i] = h2_as_u32(__hsub2(kv_field<0x00030003u>(u, c.v[0]), z.o[0]));
      p[4 * i + 1] = h2_as_u32(__hsub2(kv_field<0x000C000Cu>(u, c.v[2]), z.o[1]));
      p[4 * i + 2] = h2_as_u32(__hsub2(kv_field<0x00300030u>(u, c.v[1]), z.o[2]));
      p[4 * i + 3] = h2_as_u32(__hsub2(kv_field<0x00C000C0u>(u, c.v[3]), z.o[3]));
    }
  }
}

// NaN-keeping minimum and maximum.
__device__ __forceinline__ float kv_min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float kv_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// N words of a lane's half from their pieces.
template <typename F, int N>
__device__ __forceinline__ void kv_load_codes(const uint8_t* part, int lane, int half, uint32_t (&w)[N]) {
  constexpr int PW = F::PIECE / 4;
#pragma unroll
  for (int c = 0; c < N / PW; ++c) {
    const uint8_t* p = part + (c * 2 + half) * 32 * F::PIECE + lane * F::PIECE;
    if constexpr (PW == 1) {
      w[c] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (PW == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[2 * c] = u.x, w[2 * c + 1] = u.y;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[4 * c] = u.x, w[4 * c + 1] = u.y, w[4 * c + 2] = u.z, w[4 * c + 3] = u.w;
    }
  }
}

// 16 bytes global -> shared, asynchronously, past the L1 cache; zeros where
// `there` is false (src is not read then).  Copies since the last commit form
// a group; wait<N> returns when all but this thread's last N groups are done.
__device__ __forceinline__ void kv_copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void kv_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void kv_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two values in one word, rounded to nearest even.
template <int TYPE>
__device__ __forceinline__ uint32_t kv_pack2(float a, float b) {
  if constexpr (TYPE == kRowBF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    uint32_t u;
    memcpy(&u, &v, 4);
    return u;
  } else {
    return h2_as_u32(__floats2half2_rn(a, b));
  }
}
}  // namespace ttq
