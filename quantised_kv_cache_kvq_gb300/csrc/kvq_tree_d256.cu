// kvq_tree_d256.cu -- tree attention of 256-channel heads (kernel: kvq_tree.cuh).
#include "kvq_tree_launch.cuh"

namespace kvq {
int launch_tree_d256(TreeArgs& a, int N, cudaStream_t stream) {
    switch (N) {
        case 16: return launch_tree_t<16, 256>(a, stream);
        case 32: return launch_tree_t<32, 256>(a, stream);
        case 64: return launch_tree_t<64, 256>(a, stream);
        default: return KVQ_ERR_UNSUPPORTED;
    }
}
}  // namespace kvq
