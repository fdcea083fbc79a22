// kvq_tree_launch.cuh -- launches one instantiation of the tree attention and of its merge.
#pragma once

#include "kvq_launch.h"
#include "kvq_tree.cuh"

namespace kvq {

template <int N, int D, int KIND>
int launch_tree_t(TreeArgs& a, cudaStream_t stream) {
    constexpr int NT = TreeShape<N, D>::kThreads;
    const int64_t smem = a.stage_at + (int64_t)a.stages * a.stage_bytes;
    int nb = 0;
    const int rc = decode_blocks(reinterpret_cast<const void*>(k_tree<N, D, KIND>), NT, smem, &nb);
    if (rc != KVQ_OK) return rc;
    // two blocks per SM where the plan left them room (the calculator counts one: it holds the
    // kernel's tensor memory against it, of which a block takes at most half); blocks do not wait
    // for each other, so one that is not resident at once costs time only
    if (a.blocks == 2 && TreeShape<N, D>::kBlocks == 2) nb *= 2;
    a.NB = nb < kMaxTreeBlocks ? nb : kMaxTreeBlocks;
    if (launch_dependent(k_tree<N, D, KIND>, dim3(a.NB), dim3(NT), static_cast<size_t>(smem), stream, a) != cudaSuccess)
        return KVQ_ERR_CUDA;
    const int64_t units = (int64_t)a.lo.B * a.lo.H * a.RT;
    return launch_dependent(k_tree_merge<N, D>, dim3(static_cast<unsigned>(units * (N / kMergeColumns))), dim3(kMergeThreads), 0, stream,
                            a) == cudaSuccess
               ? KVQ_OK
               : KVQ_ERR_CUDA;
}

// The kernels of one head size and kind, by their columns.
template <int D, int KIND>
int launch_tree_kind(TreeArgs& a, int N, cudaStream_t stream) {
    switch (N) {
        case 16: return launch_tree_t<16, D, KIND>(a, stream);
        case 32: return launch_tree_t<32, D, KIND>(a, stream);
        case 64: return launch_tree_t<64, D, KIND>(a, stream);
        case 128:
            if constexpr (D <= 128) return launch_tree_t<128, D, KIND>(a, stream);
            return KVQ_ERR_UNSUPPORTED;
        default: return KVQ_ERR_UNSUPPORTED;
    }
}

}  // namespace kvq
