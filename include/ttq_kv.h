/*
 * ttq_kv.h -- C ABI of the quantised key/value cache of libttq.so (sm_100a).
 *
 * The TTQ layer's quantiser (ttq.h: group-wise affine INT codes or E4M3
 * codes with binary16 scales formed on the fly, optionally after scaling
 * each channel by the square root of an activation statistic D) applied to
 * the rows of an attention layer's keys and values as they are produced,
 * and the attention that reads them.  The pages describe the quantiser and
 * name key/value-cache scales derived on the fly and speculative decoding as
 * topics beside the method (blog.lo0.es "Test-time quantization without
 * calibration dataset"); the cache's layout and these entry points are this
 * library's own.
 *
 * Conventions are those of ttq.h (device pointers, 16-byte alignment, a
 * caller-owned workspace with a status word, work enqueued on the caller's
 * stream, nothing allocated or synchronised, nothing thrown), and:
 *
 *  - The cache is paged.  A page holds page_size tokens (a multiple of 16)
 *    of all kv_heads heads, as [kv_heads][page_size / 16] blocks of 16
 *    tokens.  With b = bits, hd = head_dim, g = group, a block is
 *      K codes 16 hd b / 8 bytes | K pairs [16][hd / g] | V codes | V pairs,
 *    a pair being (scale, zero) as two binary16.  The codes stand in the
 *    order in which a warp takes them as the A operand of a 16 x 8 x 16
 *    matrix instruction (K: token rows x channels; V: channel rows x
 *    tokens).  With LB = hd b / 32, P = min(16, LB) and
 *      place(lane, half, byte) =
 *        ((byte / P) 2 + half) 32 P + lane P + byte % P,
 *    channel c = k g + r (group k) of token t of the block is in
 *      K: lane 4 (t % 8) + r / (g / 4), half t / 8, code e = k (g / 4) +
 *         r % (g / 4) of that lane: its 32-bit word e / (32 / b), there the
 *         field e' = e % (32 / b) for b = 8, and e' / 2 + (e' % 2) (16 / b)
 *         for b < 8 (bits [b f, b f + b) of the word hold field f);
 *      V: lane 4 (r / (g / 8)) + (t % 8) / 2, half t / 8, code e = k (g / 8)
 *         + r % (g / 8): 16-bit unit e / (16 / b) of the token, field
 *         e % (16 / b) of it, at byte 4 unit + 2 (t % 2).
 *    ttq_kv_write and ttq_kv_read convert; other programs need not know it.
 *  - Codes, scales and zeros of a row are those that ttq_quantize_weight_ex
 *    gives for the row as one row of a weight with the same D, bits, group
 *    and scheme (the binary32 order stated in ttq.h), and stand for
 *    scale * (code - zero) * D^{-1/2}.  One difference: a group that holds a
 *    NaN or an infinity, or whose scale exceeds binary16, is stored with a
 *    NaN scale and zero codes (flags NONFINITE, SCALE_OVERFLOW), so that
 *    reading it gives NaN and no other token is touched.
 *  - A call's rows belong to the sequences of a batch.  Sequence i has the
 *    rows cu_new[i] .. cu_new[i + 1] - 1 (n of them, possibly none), which
 *    stand for its last n positions: row cu_new[i] + k is position
 *    kv_len[i] - n + k.  Position p is token p % page_size of page
 *    page_table[i][p / page_size].  Rows in no sequence (padding behind the
 *    last) are neither read nor written.  Sequences may share pages that
 *    are only read; a page position that one ttq_kv_write call writes twice
 *    (a page listed twice in a row of the table, or owned by two sequences
 *    with rows there) holds a mixture of the rows afterwards.
 *  - Contents of page_table, kv_len and cu_new are checked on the device.  A
 *    sequence with cu_new decreasing or beyond `rows`, or with rows that are
 *    more than max_new or kv_len, or with kv_len beyond its table, is
 *    skipped, and a position whose page is not in [0, num_pages) is skipped (written
 *    nowhere, read as absent: zeros from ttq_kv_read, not attended to);
 *    both set TTQ_FLAG_BAD_INDEX.  Of a sequence without rows nothing else is
 *    looked at, and it sets no flag.
 */
#ifndef TTQ_KV_H_
#define TTQ_KV_H_

#include "ttq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache (a host struct; the pointers are device pointers).
 * page_size: a multiple of 16 in [16, 65536].  head_dim: 64, 128 or 256.
 * bits: 2 or 4 with the INT schemes, 8 with TTQ_QSCHEME_FP8_E4M3.
 * group: 32, 64, 128 or 256, dividing head_dim at most four times. */
typedef struct ttq_kv_cache {
  void* pages;         /* [num_pages][ttq_kv_page_bytes(...)] */
  int64_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t bits;
  int32_t group;
  int32_t scheme;      /* a ttq_qscheme */
  const float* D_k;    /* float32 [kv_heads][head_dim], as ttq_act_norm gives it for rows of */
  const float* D_v;    /* K or V, or NULL (D = I): read by ttq_kv_write */
  const float* D_k_rsqrt; /* their inverse square roots, or NULL: read by ttq_kv_read and */
  const float* D_v_rsqrt; /* ttq_kv_attention */
} ttq_kv_cache;

/* The rows of one call (a host struct; the pointers are device pointers). */
typedef struct ttq_kv_batch {
  const int32_t* page_table; /* [batch][table_stride] */
  int64_t table_stride;      /* pages that a sequence may have */
  const int32_t* kv_len;     /* [batch] positions, this call's rows included */
  const int32_t* cu_new;     /* [batch + 1] */
  int64_t batch;             /* 0 to 1024 sequences */
  int64_t rows;              /* rows of the row tensors (cu_new[batch] or more) */
  int64_t max_new;           /* no sequence has more rows than this in this call */
} ttq_kv_batch;

/* Bytes of one page; 0 if the format is not built. */
size_t ttq_kv_page_bytes(int page_size, int kv_heads, int head_dim, int bits, int group);

/* Quantises the rows of K and V and writes them into the cache.
 * K, V: [rows][kv_heads][head_dim] in dtype (TTQ_F32, TTQ_BF16 or TTQ_F16),
 * channels contiguous, row and head strides in elements (multiples of 8, so
 * that slices of a fused projection can be given).  Needs a workspace of at
 * least 4096 bytes (status word).  Flags NONFINITE, SCALE_OVERFLOW and
 * BAD_INDEX. */
ttq_status ttq_kv_write(const ttq_kv_cache* cache, const ttq_kv_batch* batch, const void* K,
                        int64_t k_row, int64_t k_head, const void* V, int64_t v_row,
                        int64_t v_head, ttq_dtype dtype, void* ws, size_t ws_bytes, void* stream);

/* Dequantises each sequence's last rows: K, V [rows][kv_heads][head_dim] in
 * dtype (TTQ_F32, TTQ_BF16 or TTQ_F16), contiguous; either may be NULL.
 * Without D the value scale * (code - zero) is rounded once; with D the
 * binary32 product with D^{-1/2} is rounded.  To read whole sequences give
 * cu_new the prefix sums of kv_len.  Needs a workspace of at least 4096
 * bytes.  Flags BAD_INDEX. */
ttq_status ttq_kv_read(const ttq_kv_cache* cache, const ttq_kv_batch* batch, void* K, void* V,
                       ttq_dtype dtype, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of ttq_kv_attention for these sizes; 0 if they are not
 * built.  The bytes do not depend on the context lengths. */
size_t ttq_kv_attention_workspace_size(int head_dim, int bits, int group, int64_t heads,
                                       int64_t kv_heads, int64_t max_new);

/* Attention of every sequence's rows (new tokens) over its cached positions.
 * Q [rows][heads][head_dim] in dtype (strides as for ttq_kv_write), Y
 * [rows][heads][head_dim] in y_dtype, contiguous; heads is a multiple of
 * kv_heads and query head i reads key/value head i / (heads / kv_heads).
 *   t_j = scale <q, K_j>;  t_j = softcap tanh(t_j / softcap) if softcap > 0
 *   y   = sum_j p_j V_j,  p = softmax of t over the positions that the row sees
 * and y = 0 for a row that sees none.  A row sees
 *   - of the positions before the sequence's new ones, all;
 *   - of the new ones, without `tree` itself and the earlier ones, with
 *     `tree` (uint64 [rows], one mask per row) new token k iff bit k of its
 *     mask is set (its own bit included; bits at and above the number of the
 *     sequence's rows stand for nothing);
 *   - with window > 0 only those less than `window` positions back, where a
 *     new token's position is the number of old ones plus the number of new
 *     ones that it sees besides itself (its depth in the tree).
 * The new tokens' own K and V are read from the cache: write them first.
 * max_new is at most 64: a longer piece of a prompt goes in pieces of 64,
 * each with the kv_len that ends at its last row.  With max_new 0 nothing is
 * done or checked on the device.
 *   heads, max_new and the room that the page table has (batch x table_stride
 * pages) choose how many query rows a thread block takes together, for all
 * sequences alike: a table wider than the contexts need, or one sequence with
 * many rows beside many with one, costs time (give the latter a call of their
 * own), and results of another choice differ in their last bits.
 *   The products run on the tensor cores with binary16 operands and fp32
 * accumulation: each row of Q (times D_k_rsqrt), scaled by a power of two,
 * is rounded to binary16 (bf16 and binary16 rows without D_k_rsqrt lose
 * nothing to it but elements under 2^-14 of the row's largest) or, where it
 * is float32 or times D_k_rsqrt and Y is not bf16, to the sum of two binary16
 * (22 bits; the products with K are done twice), the codes less their zeros
 * are exact, the probabilities times V's scales are rounded to binary16, in
 * units in which the largest product of a probability and a scale that the
 * row meets is near 1: products under 2^-14 of it are subnormal and keep
 * 2^-25 of it.  (The unit goes by each token's largest scale; a group of
 * channels whose scales lie 2^14 below another group's has only such
 * products.)  What a row does not see has no effect on it.  Scores, their
 * running maxima and sums are fp32; a capped score is off by 2^-22 of the cap
 * where that is at most 256, else by 2^-19 of itself, and a cap of 2^64 or
 * more, which changes no fp32 score, is left out.  Deterministic for given
 * inputs.  ws: ttq_kv_attention_workspace_size(...) bytes, initialised once
 * by ttq_workspace_init (every call leaves its counters at zero) and again
 * after TIMEOUT; calls that may run at the same time need one each.  Flags
 * BAD_INDEX and TIMEOUT. */
ttq_status ttq_kv_attention(const ttq_kv_cache* cache, const ttq_kv_batch* batch, const void* Q,
                            int64_t q_row, int64_t q_head, ttq_dtype dtype, int64_t heads,
                            float scale, float softcap, int64_t window, const uint64_t* tree,
                            void* Y, ttq_dtype y_dtype, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTQ_KV_H_ */
