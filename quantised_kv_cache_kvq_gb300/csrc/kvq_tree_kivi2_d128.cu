// kvq_tree_kivi2_d128.cu -- tree attention: 2-bit KIVI, 128 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_kivi2_d128(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<128, kKivi2>(a, N, stream); }
}  // namespace kvq
