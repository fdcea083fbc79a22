// kvq_tree_d32.cu -- tree attention of 32-channel heads (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_d32(TreeArgs& a, int N, cudaStream_t stream) {
    switch (N) {
        case 16: return launch_tree_t<16, 32>(a, stream);
        case 32: return launch_tree_t<32, 32>(a, stream);
        case 64: return launch_tree_t<64, 32>(a, stream);
        case 128: return launch_tree_t<128, 32>(a, stream);
        default: return KVQ_ERR_UNSUPPORTED;
    }
}
}  // namespace kvq
