// kvq_tree_fp8_d64.cu -- tree attention: FP8, 64 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_fp8_d64(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<64, kFp8>(a, N, stream); }
}  // namespace kvq
