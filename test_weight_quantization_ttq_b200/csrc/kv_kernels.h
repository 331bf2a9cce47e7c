// Host-side launchers of the key/value cache's kernels (internal to
// libttq.so) and what they share.  Argument checking is done by the C ABI
// layer (kv_api.cu) before these are called.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace ttq {

constexpr int kKvMaxBatch = 1024;
constexpr int kKvMaxNew = 64;
constexpr int kKvPlanSMs = 148;   // fixed so that workspace sizes are device-independent

// Element types of the row tensors (the values of ttq_dtype).
constexpr int kRowF32 = 0;
constexpr int kRowBF16 = 1;
constexpr int kRowF16 = 2;

// Bytes of one part of a block of 16 tokens of one head.
constexpr int kv_code_bytes(int hd, int bits) { return 16 * hd * bits / 8; }
constexpr int kv_pair_bytes(int hd, int group) { return 16 * (hd / group) * 4; }
constexpr int kv_block_bytes(int hd, int bits, int group) {
  return 2 * (kv_code_bytes(hd, bits) + kv_pair_bytes(hd, group));
}

// Lets a kernel have `bytes` of dynamic shared memory on the current device;
// `set` remembers the devices (a bit each) that it was done for.
inline cudaError_t kv_allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (set.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The cache and the batch as the kernels take them.
struct KvGeometry {
  uint8_t* pages = nullptr;
  int64_t num_pages = 0, page_bytes = 0;
  int page_blocks = 1;          // blocks of 16 tokens in a page, 1 to 4096
  uint32_t page_magic = 1u << 27, page_shift = 0;   // of page_of
  int kv_heads = 1;
  const int32_t* table = nullptr;
  int64_t table_stride = 0;
  const int32_t* kv_len = nullptr;
  const int32_t* cu = nullptr;
  int batch = 0;
  int64_t rows = 0;
  int max_new = 0;
  uint32_t* status = nullptr;

  void set_page_blocks(int n) {
    page_blocks = n;
    page_shift = 0;
    while ((1 << page_shift) < n) ++page_shift;
    page_magic = static_cast<uint32_t>(((1ull << (27 + page_shift)) + n - 1) / n);
  }
  // blk / page_blocks for every block of 2^31 positions, 0 <= blk < 2^27: with
  // d = page_blocks <= 2^k, k = page_shift, the magic number is less than one
  // above 2^(27 + k) / d, so blk times it is less than 2^27 <= 2^(27 + k) / d
  // above 2^(27 + k) blk / d, too little to reach the next whole quotient.
  // (The magic number is at most 2^28, the shifted block below 2^32: a
  // multiplication's high word and a shift.)
  __host__ __device__ __forceinline__ int page_of(int blk) const {
    const uint32_t n = static_cast<uint32_t>(blk) << 5;
    return static_cast<int>(static_cast<uint32_t>(static_cast<uint64_t>(n) * page_magic >> 32) >> page_shift);
  }
};

struct KvWriteArgs {
  KvGeometry g;
  const void* x[2] = {};        // K, V rows
  int64_t row[2] = {}, head[2] = {};
  const float* D[2] = {};
};
cudaError_t launch_kv_write(const KvWriteArgs& a, int hd, int bits, int group, bool symmetric,
                            int dtype, int num_sms, cudaStream_t stream);

struct KvReadArgs {
  KvGeometry g;
  void* y[2] = {};              // K, V rows out (either may be null)
  const float* Dr[2] = {};
};
cudaError_t launch_kv_read(const KvReadArgs& a, int hd, int bits, int group, int dtype,
                           int num_sms, cudaStream_t stream);

struct KvAttentionArgs {
  KvGeometry g;
  const float* Dk = nullptr;    // D^{-1/2} of K and V, or null
  const float* Dv = nullptr;
  const void* Q = nullptr;
  int64_t q_row = 0, q_head = 0;
  int q_type = kRowBF16, y_type = kRowBF16;
  int heads = 1, per = 1;       // query heads; query heads of one key/value head
  float scale = 1.f, cap = 0.f;
  int64_t window = 0;
  const uint64_t* tree = nullptr;
  void* Y = nullptr;
  float* part = nullptr;        // two partial results per block of the grid
  uint32_t* tickets = nullptr;  // two per block of the grid, zero before and after
};
// How a launch is laid out: 8 nt query rows per tile in blocks of
// kKvAttentionWarps warps, or (nt = 16) 256 rows in blocks of 16 warps; `grid`
// blocks; q_parts binary16 numbers (1 or 2) that an element of Q is taken as;
// the floats of one partial result, and the bytes of all.
constexpr int kKvAttentionWarps = 4;
struct KvAttentionPlan {
  int nt, grid, q_parts;
  int64_t slot_floats, part_bytes;
};
// blocks: as many as the batch's sequences may have, of all heads.  grid 0: the
// format is not built.
KvAttentionPlan kv_attention_plan(int hd, int bits, int group, int64_t tile_rows, int64_t blocks, int q_parts);
cudaError_t launch_kv_attention(const KvAttentionArgs& a, int hd, int bits, int group,
                                const KvAttentionPlan& plan, cudaStream_t stream);

}  // namespace ttq
