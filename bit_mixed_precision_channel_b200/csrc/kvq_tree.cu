// kvq_tree.cu — host side of tree attention: the launch per cache dtype (the kernels are in
// kvq_tree_impl.cuh).
#include "kvq_internal.cuh"

namespace kvq {

cudaError_t tree_launch_f16(const TreeParams& p, cudaStream_t stream);
cudaError_t tree_launch_bf16(const TreeParams& p, cudaStream_t stream);

cudaError_t launch_tree(const TreeParams& p, int dtype, cudaStream_t stream) {
  return dtype == KVQ_BF16 ? tree_launch_bf16(p, stream) : tree_launch_f16(p, stream);
}

}  // namespace kvq
