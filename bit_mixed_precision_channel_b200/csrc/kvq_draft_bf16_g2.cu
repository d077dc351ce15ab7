// Decode-attention kernels with drafted tokens for bf16 caches, 2 rows (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(bf16_g2, __nv_bfloat16, 2)
}  // namespace kvq
