// Decode-attention kernels over chosen pages for bf16 caches with 4 query heads per kv head.
#include "kvq_decode_impl.cuh"

namespace kvq {
KVQ_SPARSE_INSTANCE(bf16_g4, __nv_bfloat16, 4)
}  // namespace kvq
