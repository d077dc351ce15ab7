// Decode-attention kernels with drafted tokens for bf16 caches, 1 row (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(bf16_g1, __nv_bfloat16, 1)
}  // namespace kvq
