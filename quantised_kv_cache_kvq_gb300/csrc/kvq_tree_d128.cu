// kvq_tree_d128.cu -- tree attention of 128-channel heads (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_d128(TreeArgs& a, int N, cudaStream_t stream) {
    switch (N) {
        case 16: return launch_tree_t<16, 128>(a, stream);
        case 32: return launch_tree_t<32, 128>(a, stream);
        case 64: return launch_tree_t<64, 128>(a, stream);
        case 128: return launch_tree_t<128, 128>(a, stream);
        default: return KVQ_ERR_UNSUPPORTED;
    }
}
}  // namespace kvq
