// Decode-attention kernels with drafted tokens for bf16 caches, 8 rows (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(bf16_g8, __nv_bfloat16, 8)
}  // namespace kvq
