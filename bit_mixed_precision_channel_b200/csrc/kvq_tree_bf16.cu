// Tree-attention kernels for bf16 caches.
#include "kvq_tree_impl.cuh"

namespace kvq {
cudaError_t tree_launch_bf16(const TreeParams& p, cudaStream_t stream) { return tree::launch<__nv_bfloat16>(p, stream); }
}  // namespace kvq
