// Decode-attention kernels with drafted tokens for fp16 caches, 8 rows (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(f16_g8, __half, 8)
}  // namespace kvq
