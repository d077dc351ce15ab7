// Decode-attention kernels with drafted tokens for fp16 caches, 4 rows (drafted token, query head) per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_DRAFT_INSTANCE(f16_g4, __half, 4)
}  // namespace kvq
