// The C ABI of the quantised key/value cache (declared in include/ttq_kv.h):
// argument checks and launches.  Nothing here allocates device memory or
// synchronises.
#include <cmath>

#include "kv_attention.cuh"
#include "ttq_kv.h"

namespace ttq {
namespace {

constexpr size_t kStatusBytes = 4096;     // the least workspace an entry point takes
// The part of a workspace that ttq_workspace_init zeroes and every call leaves
// at zero: the status word, then the attention's tickets from byte 256.
constexpr size_t kKvHeader = 20480;
constexpr size_t kKvTickets = 256;
static_assert(kKvTickets + 2 * 4 * kKvPlanSMs * sizeof(uint32_t) <= kKvHeader,
              "two tickets a block, of at most 4 blocks per SM");

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool format_built(int hd, int bits, int group) {
  if (hd != 64 && hd != 128 && hd != 256) return false;
  if (bits != 2 && bits != 4 && bits != 8) return false;
  if (group != 32 && group != 64 && group != 128 && group != 256) return false;
  return group <= hd && hd / group <= 4;
}

size_t page_bytes(int page_size, int kv_heads, int hd, int bits, int group) {
  if (page_size < 16 || page_size > 65536 || page_size % 16 != 0 || kv_heads < 1 || kv_heads > 65535) return 0;
  if (!format_built(hd, bits, group)) return 0;
  return static_cast<size_t>(kv_heads) * (page_size / 16) * kv_block_bytes(hd, bits, group);
}

// The checks that the three entry points share, and the kernels' view.
ttq_status geometry(const ttq_kv_cache* c, const ttq_kv_batch* b, void* ws, size_t ws_bytes, KvGeometry* g) {
  if (c == nullptr || b == nullptr) return TTQ_ERR_INVALID_ARG;
  if (c->scheme != TTQ_QSCHEME_ASYMMETRIC && c->scheme != TTQ_QSCHEME_SYMMETRIC && c->scheme != TTQ_QSCHEME_FP8_E4M3)
    return TTQ_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0) return TTQ_ERR_INVALID_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->num_pages < 0 || c->num_pages > INT32_MAX) return TTQ_ERR_INVALID_ARG;
  if (!format_built(c->head_dim, c->bits, c->group)) return TTQ_ERR_UNSUPPORTED;
  if ((c->bits == 8) != (c->scheme == TTQ_QSCHEME_FP8_E4M3)) return TTQ_ERR_UNSUPPORTED;
  if (b->batch < 0 || b->rows < 0 || b->max_new < 0 || b->table_stride < 0) return TTQ_ERR_INVALID_ARG;
  if (b->rows > INT32_MAX || b->table_stride > INT32_MAX) return TTQ_ERR_INVALID_ARG;
  if (b->batch > kKvMaxBatch) return TTQ_ERR_UNSUPPORTED;
  if (b->batch > 0 && (b->kv_len == nullptr || b->cu_new == nullptr)) return TTQ_ERR_INVALID_ARG;
  if (b->batch > 0 && b->table_stride > 0 && b->page_table == nullptr) return TTQ_ERR_INVALID_ARG;
  if (c->num_pages > 0 && c->pages == nullptr) return TTQ_ERR_INVALID_ARG;
  if (!aligned(c->pages, 16) || !aligned(b->page_table, 4) || !aligned(b->kv_len, 4) || !aligned(b->cu_new, 4))
    return TTQ_ERR_INVALID_ARG;
  for (const float* d : {c->D_k, c->D_v, c->D_k_rsqrt, c->D_v_rsqrt})
    if (!aligned(d, 16)) return TTQ_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, 256)) return TTQ_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes) return TTQ_ERR_WORKSPACE;
  g->pages = static_cast<uint8_t*>(c->pages);
  g->num_pages = c->num_pages;
  g->page_bytes = static_cast<int64_t>(page_bytes(c->page_size, c->kv_heads, c->head_dim, c->bits, c->group));
  g->set_page_blocks(c->page_size / 16);
  g->kv_heads = c->kv_heads;
  g->table = b->page_table;
  g->table_stride = b->table_stride;
  g->kv_len = b->kv_len;
  g->cu = b->cu_new;
  g->batch = static_cast<int>(b->batch);
  g->rows = b->rows;
  g->max_new = static_cast<int>(b->max_new < INT32_MAX ? b->max_new : INT32_MAX);
  g->status = static_cast<uint32_t*>(ws);
  return TTQ_OK;
}

bool row_type(ttq_dtype t) { return t == TTQ_F32 || t == TTQ_BF16 || t == TTQ_F16; }

// Rows with the given strides: 16-byte loads of 8 channels.
bool strides_ok(const void* p, int64_t row, int64_t head) {
  return aligned(p, 16) && row >= 0 && head >= 0 && row % 8 == 0 && head % 8 == 0;
}

ttq_status status_of(cudaError_t e) { return e == cudaSuccess ? TTQ_OK : TTQ_ERR_CUDA; }

}  // namespace

// cap tanh(t / cap) is t but for (t / cap)^2 / 3 of it, and at most cap: with a
// cap of 2^64 all t to 2^52 are what they were, under 2^-64 all are zero beside 1.
// (Between them 1 / cap, 2 / cap and cap log2(e) are normal numbers.)
constexpr float kKvMostCap = 18446744073709551616.f, kKvLeastCap = 1.f / kKvMostCap;

// Tiles of 256 rows pay where there is work for them: the blocks that the
// batch's sequences may have, by the width of its page table (32 heads over 8,
// trees of 48: 4000 blocks 55 us, 42 in tiles of 32; 8000 blocks 71 and 68;
// trees of 64: 4000 blocks 61 and 51, 16448 blocks of E4M3 with a cap 135 and 170).
// The lengths themselves are on the device: a table much wider than they need
// takes these tiles where those of 32 were faster (a table 8 times as wide: trees
// of 24 over 8 contexts of 500 43 us against 37, of 64 over 2 of 2000 50 against 35).
constexpr int64_t kWideBlocks = 8192;

// 8, 16, 24 or 32 query rows per tile: the fewest that hold a sequence's rows
// of one key/value head, since rows of a tile that are not there cost as much
// as those that are, while every further tile reads and unpacks the codes
// again; of more rows than 32 tiles of 24 if that makes no more of them.  (24
// against 32: 16 sequences of 4000, 24 rows, 44.7 and 50.3 us; 16 of up to
// 2048, 48 rows of heads of 64, 24.7 and 28.2.  24 against 32 at 192 rows,
// which makes 8 tiles instead of 6: 94 and 83.  16 against 32 at 256: 188 and
// 165.)  Heads of 256 channels stop at 16 (their accumulators fill the
// registers).  The tiles of 256 rows of kv_attention_wide.cuh (nt = 16), of
// heads up to 128 in one or two groups, where each stands for 6 tiles of 32
// or more: trees of 24 with 192 rows 75 us (6 tiles 84), trees of 64 with
// 256 rows 134 (8 tiles 170); one of fewer rows costs as much, so that 5
// would be about even.  Q in two parts has no tiles of 24 and 256 rows (its
// second set of fragments does not fit beside the operands of 256).
KvAttentionPlan kv_attention_plan(int hd, int bits, int group, int64_t tile_rows, int64_t blocks, int q_parts) {
  KvAttentionPlan p = {};
  if (!format_built(hd, bits, group)) return p;
  const int64_t tiles32 = (tile_rows + 31) / 32, tiles256 = (tile_rows + 255) / 256;
  if (hd <= 128 && hd / group <= 2 && q_parts == 1 && tiles256 > 0 && tiles32 >= 6 * tiles256 && blocks >= kWideBlocks) p.nt = 16;
  else if (tile_rows <= 8) p.nt = 1;
  else if (tile_rows <= 16 || hd == 256) p.nt = 2;
  else p.nt = q_parts == 1 && (tile_rows + 23) / 24 == tiles32 ? 3 : 4;
  p.q_parts = q_parts;
  const int ctas = hd == 64    ? kv_attention_ctas_hd64(bits, group, p.nt, q_parts)
                   : hd == 128 ? kv_attention_ctas_hd128(bits, group, p.nt, q_parts)
                               : kv_attention_ctas_hd256(bits, group, p.nt, q_parts);
  p.grid = ctas * kKvPlanSMs;
  p.slot_floats = static_cast<int64_t>(p.nt == 16 ? 256 : 8 * p.nt) * (hd + 4);
  p.part_bytes = static_cast<int64_t>(p.grid) * 2 * p.slot_floats * 4;
  return p;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int hd, int bits, int group,
                                const KvAttentionPlan& plan, cudaStream_t stream) {
  if (hd == 64) return kv_attention_hd64(a, bits, group, plan, stream);
  if (hd == 128) return kv_attention_hd128(a, bits, group, plan, stream);
  return kv_attention_hd256(a, bits, group, plan, stream);
}

}  // namespace ttq

extern "C" {

using namespace ttq;

size_t ttq_kv_page_bytes(int page_size, int kv_heads, int head_dim, int bits, int group) {
  return page_bytes(page_size, kv_heads, head_dim, bits, group);
}

ttq_status ttq_kv_write(const ttq_kv_cache* cache, const ttq_kv_batch* batch, const void* K,
                        int64_t k_row, int64_t k_head, const void* V, int64_t v_row,
                        int64_t v_head, ttq_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
  KvWriteArgs a;
  const ttq_status st = geometry(cache, batch, ws, ws_bytes, &a.g);
  if (st != TTQ_OK) return st;
  if (!row_type(dtype)) return TTQ_ERR_INVALID_ARG;
  if (!strides_ok(K, k_row, k_head) || !strides_ok(V, v_row, v_head)) return TTQ_ERR_INVALID_ARG;
  if (batch->rows == 0 || batch->batch == 0) return TTQ_OK;
  if (K == nullptr || V == nullptr) return TTQ_ERR_INVALID_ARG;
  a.x[0] = K, a.x[1] = V;
  a.row[0] = k_row, a.row[1] = v_row;
  a.head[0] = k_head, a.head[1] = v_head;
  a.D[0] = cache->D_k, a.D[1] = cache->D_v;
  return status_of(launch_kv_write(a, cache->head_dim, cache->bits, cache->group,
                                   cache->scheme == TTQ_QSCHEME_SYMMETRIC, dtype, device_sms(),
                                   static_cast<cudaStream_t>(stream)));
}

ttq_status ttq_kv_read(const ttq_kv_cache* cache, const ttq_kv_batch* batch, void* K, void* V,
                       ttq_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
  KvReadArgs a;
  const ttq_status st = geometry(cache, batch, ws, ws_bytes, &a.g);
  if (st != TTQ_OK) return st;
  if (!row_type(dtype) || !aligned(K, 16) || !aligned(V, 16)) return TTQ_ERR_INVALID_ARG;
  if (batch->rows == 0 || batch->batch == 0 || (K == nullptr && V == nullptr)) return TTQ_OK;
  a.y[0] = K, a.y[1] = V;
  a.Dr[0] = cache->D_k_rsqrt, a.Dr[1] = cache->D_v_rsqrt;
  return status_of(launch_kv_read(a, cache->head_dim, cache->bits, cache->group, dtype, device_sms(),
                                  static_cast<cudaStream_t>(stream)));
}

size_t ttq_kv_attention_workspace_size(int head_dim, int bits, int group, int64_t heads,
                                       int64_t kv_heads, int64_t max_new) {
  if (kv_heads < 1 || heads < kv_heads || heads % kv_heads != 0 || heads > 65535) return 0;
  if (max_new < 0 || max_new > kKvMaxNew) return 0;
  // the most of what any types, context lengths and fewer rows take: the plans
  // of every width of tile up to the rows' own, for Q in one part and in two
  // (which has other tiles)
  const int64_t tile_rows = max_new * (heads / kv_heads);
  int64_t most = 0;
  for (const int q_parts : {1, 2})
    for (const int64_t rows : {8, 16, 24, 32, 256}) {
      const int64_t tile = tile_rows < rows ? tile_rows : rows;
      const KvAttentionPlan p = kv_attention_plan(head_dim, bits, group, tile, INT64_MAX, q_parts);
      if (p.grid == 0) return 0;
      if (p.part_bytes > most) most = p.part_bytes;
    }
  return kKvHeader + most;
}

ttq_status ttq_kv_attention(const ttq_kv_cache* cache, const ttq_kv_batch* batch, const void* Q,
                            int64_t q_row, int64_t q_head, ttq_dtype dtype, int64_t heads,
                            float scale, float softcap, int64_t window, const uint64_t* tree,
                            void* Y, ttq_dtype y_dtype, void* ws, size_t ws_bytes, void* stream) {
  KvAttentionArgs a;
  const ttq_status st = geometry(cache, batch, ws, ws_bytes, &a.g);
  if (st != TTQ_OK) return st;
  if (!row_type(dtype) || !row_type(y_dtype)) return TTQ_ERR_INVALID_ARG;
  if (heads < 1 || heads > 65535 || heads % cache->kv_heads != 0) return TTQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return TTQ_ERR_INVALID_ARG;
  if (!strides_ok(Q, q_row, q_head) || !aligned(Y, 16) || !aligned(tree, 8)) return TTQ_ERR_INVALID_ARG;
  if (batch->max_new > kKvMaxNew) return TTQ_ERR_UNSUPPORTED;
  const size_t need = ttq_kv_attention_workspace_size(cache->head_dim, cache->bits, cache->group, heads,
                                                      cache->kv_heads, batch->max_new);
  if (ws_bytes < need) return TTQ_ERR_WORKSPACE;
  if (batch->rows == 0 || batch->batch == 0 || batch->max_new == 0) return TTQ_OK;
  if (Q == nullptr || Y == nullptr) return TTQ_ERR_INVALID_ARG;
  const int per = static_cast<int>(heads / cache->kv_heads);
  const int64_t longest = batch->table_stride * a.g.page_blocks;   // blocks that a sequence may have (below 2^44)
  const int64_t blocks = batch->batch * cache->kv_heads * (longest < (1 << 27) ? longest : 1 << 27);
  // Q times D_k^{-1/2}, and float32 rows, do not fit binary16: an element is then
  // taken as two of them, so that scores are as exact as their fp32 sums, but for
  // outputs in bf16, whose own rounding is 8 times the one that a single binary16 costs.
  // (One alone put binary16 outputs 1.5 to 2.2 times as far off as their rounding
  // does.  The price, with D and outputs in binary16 against bf16: 64 sequences of up
  // to 8192 115 us against 90, window and cap 37 and 30, chains of 5 43 and 40, trees of
  // 24, in tiles of 32 rows then, 128 and 75.)
  const int q_parts = y_dtype != TTQ_BF16 && (dtype == TTQ_F32 || cache->D_k_rsqrt != nullptr) ? 2 : 1;
  const KvAttentionPlan p = kv_attention_plan(cache->head_dim, cache->bits, cache->group, batch->max_new * per, blocks,
                                              q_parts);
  if (ws_bytes < kKvHeader + static_cast<size_t>(p.part_bytes)) return TTQ_ERR_WORKSPACE;   // (need is the most of all plans)
  a.Dk = cache->D_k_rsqrt;
  a.Dv = cache->D_v_rsqrt;
  a.Q = Q;
  a.q_row = q_row;
  a.q_head = q_head;
  a.q_type = dtype;
  a.y_type = y_dtype;
  a.heads = static_cast<int>(heads);
  a.per = per;
  a.scale = scale;
  // beyond these a cap changes no score in fp32, and makes all the same
  a.cap = softcap >= kKvMostCap ? 0.f : softcap > 0.f && softcap < kKvLeastCap ? kKvLeastCap : softcap;
  a.window = window;
  a.tree = tree;
  a.Y = Y;
  a.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kKvTickets);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kKvHeader);
  return status_of(launch_kv_attention(a, cache->head_dim, cache->bits, cache->group, p,
                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
