// kvq_tree_kivi4_d256.cu -- tree attention: 4-bit KIVI, 256 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_kivi4_d256(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<256, kKivi4>(a, N, stream); }
}  // namespace kvq
