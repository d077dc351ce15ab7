// Decode-attention kernels over chosen pages for fp16 caches with 4 query heads per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_SPARSE_INSTANCE(f16_g4, __half, 4)
}  // namespace kvq
