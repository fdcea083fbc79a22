// kvq_tree_rows_d128.cu -- tree attention: INT8 and INT4 rows, 128 channels (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_rows_d128(TreeArgs& a, int N, cudaStream_t stream) { return launch_tree_kind<128, kRows>(a, N, stream); }
}  // namespace kvq
