// kvq_tree_rows_d256.cu -- tree attention: INT8 and INT4 rows, 256 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_rows_d256(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<256, kRows>(a, N, stream); }
}  // namespace kvq
