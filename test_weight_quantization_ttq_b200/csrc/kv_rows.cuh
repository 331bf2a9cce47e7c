// Writing rows of keys and values into the paged cache as group-wise codes,
// and reading them back (ttq_kv_write, kv_write.cu; ttq_kv_read, kv_read.cu): what the
// two share.
//
// The quantiser is the layer's own, in the same binary32 order (bit-exact
// with ttq_quantize_weight_ex of the row as one row of a weight):
//   x = k sqrt(D); m = min(0, min x); M = max(0, max x) over the group;
//   s32 = (M - m) / (2^b - 1), at least 2^-14; s = binary16 round-up(s32);
//   inv = 1 / s; z = clamp(rint(-m inv)); q = clamp(rint(x inv) + z),
// rint of the exact product.  Symmetric and E4M3 codes likewise.
//
// Both kernels are bound by memory: a position of one head is 4 hd bytes of
// bf16 rows against 2 (hd b / 8 + 4 hd / g) bytes of cache.  A warp takes the
// K or the V part of one block (16 tokens of one head) and every lane the
// codes that the layout gives it, so that codes move in 16-byte pieces with
// all lanes contiguous, a group's range is found by 2 (K) or 3 (V) shuffles,
// and a row's place is looked up once per 16 rows.  (A thread per 8 channels
// of one row, with its own search, took 84 and 70 us where these take 47 and
// 35: the prompts of 5 requests, 12020 rows of 8 heads, written as INT4 codes
// and read back, and 32785 positions read.)
// Rows of the dense tensors are read 16 bytes a lane; they are written
// through shared memory, so that a store covers whole rows.
#pragma once

#include <type_traits>

#include "kv_device.cuh"
#include "ttq_kernels.h"

namespace ttq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// The work of a call: for each sequence the blocks that its rows lie in.
// seqs[b] = {end of its blocks in the sum over the sequences, kv, row0, n}.
__device__ __forceinline__ int schedule(const KvGeometry& g, int4* seqs) {
  __shared__ int total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < g.batch; b0 += 32) {
      const int b = b0 + lane;
      KvSequence s = {};
      int64_t v = 0;
      if (b < g.batch) {
        if (kv_sequence(g, b, s)) {
          if (s.n > 0) v = ((s.kv - 1) >> 4) - ((s.kv - s.n) >> 4) + 1;
        } else if (s.n != 0 && blockIdx.x == 0) {
          set_flag(g.status, TTQ_FLAG_BAD_INDEX);
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < g.batch) seqs[b] = make_int4(static_cast<int>(base + v), s.kv, s.row0, s.n);
      base += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) {
      // rows that several sequences claim can add up to more blocks than there
      // could be: then nothing is done
      const bool fits = base <= 0x7F000000;
      total = fits ? static_cast<int>(base) : 0;
      if (!fits && blockIdx.x == 0) set_flag(g.status, TTQ_FLAG_BAD_INDEX);
    }
  }
  __syncthreads();
  return total;
}

// A warp's part of the work: the block of a sequence, and what of it is there.
struct KvTask {
  int which, h;        // K or V, head
  int page, at;        // the block's page as the table gives it, and its place among the page's
  int row;             // row of the block's token 0 (may be below the sequence's first)
  int lo, hi;          // tokens [lo, hi) of the block have rows
};
// The codes of a task; null: the page is not one of the cache's.  (Apart from
// KvWalk::task, so that nothing waits for the table's entry before the task
// is due.)
template <typename F>
__device__ __forceinline__ uint8_t* part_of(const KvGeometry& g, const KvTask& k) {
  if (k.page >= 0 && k.page < g.num_pages)
    return g.pages + k.page * g.page_bytes +
           (static_cast<int64_t>(k.h) * g.page_blocks + k.at) * F::BLOCK + k.which * F::V_OFFSET;
  if ((threadIdx.x & 31) == 0) set_flag(g.status, TTQ_FLAG_BAD_INDEX);
  return nullptr;
}
// The parts that a warp takes, one after another: the sum over the sequences'
// blocks, then the heads, then K and V.
struct KvWalk {
  int ordinal, rest;   // block and part of it
  int step_ordinal, step_rest, parts;
  int b = 0;           // sequence of the last task
  int64_t left;        // parts of the call from here on
  __device__ __forceinline__ KvWalk(const KvGeometry& g, int64_t total) {
    parts = 2 * g.kv_heads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const uint32_t step = gridDim.x * kWarps;    // (both below 2^32: the grid is what is resident)
    ordinal = static_cast<uint32_t>(first) / parts;
    rest = static_cast<uint32_t>(first) % parts;
    step_ordinal = step / parts;
    step_rest = step % parts;
    left = total - first;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= gridDim.x * kWarps;
    ordinal += step_ordinal;
    rest += step_rest;
    if (rest >= parts) rest -= parts, ++ordinal;
  }
  __device__ __forceinline__ KvTask task(const KvGeometry& g, const int4* seqs) {
    if (seqs[b].x <= ordinal) {
      int lo = b + 1, hi = g.batch - 1;
      while (lo < hi) {                 // first with end > ordinal
        const int mid = (lo + hi) >> 1;
        if (seqs[mid].x > ordinal) hi = mid; else lo = mid + 1;
      }
      b = lo;
    }
    const int4 s = seqs[b];
    const int old = s.y - s.w, blk = (old >> 4) + ordinal - (b > 0 ? seqs[b - 1].x : 0);
    const int pg = g.page_of(blk);
    KvTask k;
    k.page = __ldg(g.table + b * g.table_stride + pg);
    k.at = blk - pg * g.page_blocks;
    k.which = rest & 1;
    k.h = rest >> 1;
    k.lo = max(old - blk * 16, 0);
    k.hi = min(s.y - blk * 16, 16);
    k.row = s.z + blk * 16 - old;
    return k;
  }
};

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

// Thread blocks for the most parts of blocks that the rows may lie in, up to
// `per_sm` a SM (what is resident, so that all end together).  Where there
// are more parts than warps the step of a warp, grid * kWarps parts, is made
// a multiple of the heads' parts, so that a warp stays at its head.
unsigned part_grid(const KvGeometry& g, int num_sms, int per_sm) {
  const int64_t blocks = (g.rows + 15) / 16 + 2 * static_cast<int64_t>(g.batch);
  const int64_t need = (blocks * g.kv_heads * 2 + kWarps - 1) / kWarps, most = static_cast<int64_t>(num_sms) * per_sm;
  if (need <= most) return static_cast<unsigned>(need);
  int64_t unit = g.kv_heads;                    // kv_heads / gcd(kv_heads, kWarps / 2)
  for (int w = kWarps / 2; w > 1 && unit % 2 == 0; w /= 2) unit /= 2;
  return static_cast<unsigned>(most >= unit ? most / unit * unit : most);
}

}  // namespace
}  // namespace ttq
