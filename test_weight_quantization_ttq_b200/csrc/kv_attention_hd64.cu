// Attention over the quantised cache: head size 64 (kv_attention.cuh).
#include "kv_attention.cuh"

namespace ttq {

cudaError_t kv_attention_hd64(const KvAttentionArgs& a, int bits, int group, const KvAttentionPlan& p,
                              cudaStream_t stream) {
  return kv_attention_launch<64>(a, bits, group, p, stream);
}
int kv_attention_ctas_hd64(int bits, int group, int nt, int q_parts) {
  return kv_attention_ctas<64>(bits, group, nt, q_parts);
}

}  // namespace ttq
