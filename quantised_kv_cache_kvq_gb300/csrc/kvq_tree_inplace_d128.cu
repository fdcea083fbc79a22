// kvq_tree_inplace_d128.cu -- tree attention: KIVI records read in place, 128 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_inplace_d128(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<128, kInPlace>(a, N, stream); }
}  // namespace kvq
