// Tree-attention kernels for fp16 caches.
#include "kvq_tree_impl.cuh"

namespace kvq {
cudaError_t tree_launch_f16(const TreeParams& p, cudaStream_t stream) { return tree::launch<__half>(p, stream); }
}  // namespace kvq
