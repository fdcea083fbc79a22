// kvq_tree.cu -- attention of drafted tokens over a cache and over the drafts that they see.
#include <cmath>
#include <cstdint>

#include "kvq_elements.cuh"
#include "kvq_internal.cuh"
#include "kvq_launch.h"
#include "kvq_rope_angle.cuh"

namespace kvq {
namespace {

constexpr int kTreeThreads = 256;

struct TreeArgs {
    Layout lo;
    const uint8_t* cache;
    int layer, nodes;
    const __nv_bfloat16 *q, *k, *v;
    const uint8_t* mask;
    const int32_t* n_nodes;
    float scale;
    __nv_bfloat16* out;
    uint8_t* ws;
    float rope_w[128];
};

// A block per (node, query head, sequence): its 8 warps take the tokens in turn, each with a
// running maximum and sum (one pass over the data), joined at the end.
__global__ void __launch_bounds__(kTreeThreads) k_tree(TreeArgs a) {
    __shared__ float so[8][256], sm[8], sl[8];
    const Layout& lo = a.lo;
    const int D = lo.D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, h = hq / lo.gqa;
    const int32_t* st = state_ptr(lo, a.cache, a.layer, b);
    const int n = st[0], qn = st[1];
    int nodes = a.n_nodes ? a.n_nodes[b] : a.nodes;
    nodes = nodes < 0 ? 0 : (nodes > a.nodes ? a.nodes : nodes);
    const int64_t row = (((int64_t)b * a.nodes + i) * lo.Hq + hq) * D;
    float m = -INFINITY, l = 0.0f, o[8] = {}, q[8];
    bool bad = false;
    for (int e = 0; e < D / 32; ++e) q[e] = __bfloat162float(a.q[row + lane + 32 * e]);
    if (i < nodes)
        for (int64_t t = warp; t < n + nodes; t += 8) {
            const int64_t j = t - n;
            if (j >= 0 && !(a.mask ? a.mask[((int64_t)b * a.nodes + i) * a.nodes + j] != 0 : j <= i)) continue;
            const int64_t drow = (((int64_t)b * a.nodes + j) * lo.H + h) * D;
            float s = 0.0f, v[8];
            for (int e = 0; e < D / 32; ++e) {
                const int c = lane + 32 * e;
                float k;
                if (j >= 0) {
                    k = __bfloat162float(a.k[drow + c]);
                    v[e] = __bfloat162float(a.v[drow + c]);
                } else {
                    k = cached_element(lo, a.cache, a.layer, b, h, qn, t, c, 0, &bad);
                    v[e] = cached_element(lo, a.cache, a.layer, b, h, qn, t, c, 1, &bad);
                    if (lo.rope_base > 0.0f) {
                        const int other = c < D / 2 ? c + D / 2 : c - D / 2;
                        const float y = cached_element(lo, a.cache, a.layer, b, h, qn, t, other, 0, &bad);
                        float sn, cs;
                        rope_sincos(__fmul_rn(static_cast<float>(t), a.rope_w[c % (D / 2)]), &sn, &cs);
                        k = c < D / 2 ? k * cs - y * sn : k * cs + y * sn;
                    }
                }
                s = fmaf(q[e], k, s);
            }
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            s *= a.scale;
            const float m2 = fmaxf(m, s), f = exp2f(m - m2), p = exp2f(s - m2);
            m = m2;
            l = l * f + p;
            for (int e = 0; e < D / 32; ++e) o[e] = fmaf(p, v[e], o[e] * f);
        }
    if (bad) atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_BAD_PAGE);
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int e = 0; e < D / 32; ++e) so[warp][lane + 32 * e] = o[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kTreeThreads) {
        float M = -INFINITY, L = 0.0f, O = 0.0f;
        for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
        for (int w = 0; w < 8; ++w) {
            if (sl[w] == 0.0f) continue;
            const float f = exp2f(sm[w] - M);
            L += sl[w] * f;
            O += so[w][c] * f;
        }
        a.out[row + c] = __float2bfloat16_rn(L != 0.0f ? O / L : 0.0f);
    }
}

int tree_plan(const kvq_config* cfg, int nodes, Layout* lo, int64_t* bytes) {
    const int rc = make_layout(cfg, cfg->max_tokens, lo);
    if (rc != KVQ_OK) return rc;
    if (nodes < 1 || nodes > KVQ_MAX_TREE_NODES) return KVQ_ERR_ARG;
    if (lo->dtype != KVQ_DTYPE_BF16) return KVQ_ERR_UNSUPPORTED;
    *bytes = 256;
    return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" {

int kvq_tree_workspace_bytes(const kvq_config* cfg, int32_t nodes, uint64_t* out_bytes) {
    if (!cfg || !out_bytes) return KVQ_ERR_ARG;
    kvq::Layout lo;
    int64_t bytes = 0;
    const int rc = kvq::tree_plan(cfg, nodes, &lo, &bytes);
    if (rc != KVQ_OK) return rc;
    *out_bytes = static_cast<uint64_t>(bytes);
    return KVQ_OK;
}

int kvq_tree_attention(const kvq_config* cfg, const void* cache, int32_t layer, int32_t nodes, const void* q,
                       const void* k_draft, const void* v_draft, const uint8_t* mask, const int32_t* n_nodes,
                       float softmax_scale, void* out, void* workspace, uint64_t workspace_bytes,
                       kvq_stream_t stream) {
    if (!cfg || !cache || !q || !k_draft || !v_draft || !out || !workspace) return KVQ_ERR_ARG;
    kvq::TreeArgs a;
    int64_t bytes = 0;
    const int rc = kvq::tree_plan(cfg, nodes, &a.lo, &bytes);
    if (rc != KVQ_OK) return rc;
    if (layer < 0 || layer >= a.lo.L) return KVQ_ERR_ARG;
    if (a.lo.PG > 0 && a.lo.NG > 0 && !a.lo.table) return KVQ_ERR_ARG;
    if (workspace_bytes < static_cast<uint64_t>(bytes)) return KVQ_ERR_WORKSPACE;
    auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(cache, 256) || off(workspace, 256) || off(q, 16) || off(k_draft, 16) || off(v_draft, 16) || off(out, 16) ||
        off(n_nodes, 4) || off(a.lo.table, 4))
        return KVQ_ERR_ALIGN;
    a.cache = static_cast<const uint8_t*>(cache);
    a.layer = layer;
    a.nodes = nodes;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k_draft);
    a.v = static_cast<const __nv_bfloat16*>(v_draft);
    a.mask = mask;
    a.n_nodes = n_nodes;
    a.scale = softmax_scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ws = static_cast<uint8_t*>(workspace);
    if (a.lo.rope_base > 0.0f)
        for (int i = 0; i < a.lo.D / 2; ++i)
            a.rope_w[i] = static_cast<float>(std::pow(static_cast<double>(a.lo.rope_base), -2.0 * i / a.lo.D));
    kvq::k_tree<<<dim3(nodes, a.lo.Hq, a.lo.B), kvq::kTreeThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
