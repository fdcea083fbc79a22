// kvq_tree_inplace_d256.cu -- tree attention: KIVI records read in place, 256 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_inplace_d256(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<256, kInPlace>(a, N, stream); }
}  // namespace kvq
