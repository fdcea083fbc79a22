// kvq_tree_d64.cu -- tree attention of 64-channel heads (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_d64(TreeArgs& a, int N, cudaStream_t stream) {
    switch (N) {
        case 16: return launch_tree_t<16, 64>(a, stream);
        case 32: return launch_tree_t<32, 64>(a, stream);
        case 64: return launch_tree_t<64, 64>(a, stream);
        case 128: return launch_tree_t<128, 64>(a, stream);
        default: return KVQ_ERR_UNSUPPORTED;
    }
}
}  // namespace kvq
