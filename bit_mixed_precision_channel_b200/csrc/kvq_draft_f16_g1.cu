// Decode-attention kernels with drafted tokens for fp16 caches, 1 row (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(f16_g1, __half, 1)
}  // namespace kvq
