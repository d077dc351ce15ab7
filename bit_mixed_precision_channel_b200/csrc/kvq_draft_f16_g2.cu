// Decode-attention kernels with drafted tokens for fp16 caches, 2 rows (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(f16_g2, __half, 2)
}  // namespace kvq
