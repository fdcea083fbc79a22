// kvq_tree.cu -- attention of drafted tokens over a cache and over the drafts that they see.
#include <cmath>
#include <cstdint>

#include "kvq_internal.cuh"
#include "kvq_launch.h"
#include "kvq_tree.cuh"

namespace kvq {

int launch_tree_rows_d32(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_fp8_d32(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi2_d64(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi4_d64(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi8_d64(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_rows_d64(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_fp8_d64(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi2_d128(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi4_d128(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi8_d128(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_rows_d128(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_fp8_d128(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi2_d256(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi4_d256(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_kivi8_d256(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_inplace_d256(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_rows_d256(TreeArgs& a, int N, cudaStream_t stream);
int launch_tree_fp8_d256(TreeArgs& a, int N, cudaStream_t stream);

namespace {

struct TreePlan {
    Layout lo;
    int N, RT, rows, TT, stages, share, blocks;
    int stage_at;
    int64_t stage, span_off, ml_off, o_off, bytes;
};

// Bytes of the operand tiles of k_tree<N, D> (TreeShape), and what a block may have next to the
// kernel's static arrays (under 8 KiB); where two blocks share an SM (heads of up to 128
// channels, up to 64 columns), half of its 228 KiB less 1 KiB reserved and those arrays (under
// 4.5 KiB).
int64_t tile_bytes(int N, int D) { return 256 * D + (D > 128 ? 65536 : 32768) + 2 * N * D + 256 * N; }
constexpr int64_t kTreeSmemLimit = 219 * 1024, kTreeSmemHalf = 108 * 1024 + 512;

// The row tile: the fewest columns, 16 to 128, that hold all queries of a KV head, or 128 (64
// for heads of 256 channels, whose tiles are twice as large).  The packed bytes of the next two
// tiles (else the next one) pass through shared memory where they fit next to the operand
// tiles: two blocks per SM come first, if need be with the weights in the key tile's place (the
// next keys then wait for their product), then two stages.  Fewer columns are taken if that makes
// the room; else (KIVI records of 256 channels at 8 bits or with many outliers) the kernel reads
// them in place.
int tree_plan(const kvq_config* cfg, int nodes, TreePlan* p) {
    const int rc = make_layout(cfg, cfg->max_tokens, &p->lo);
    if (rc != KVQ_OK) return rc;
    const Layout& lo = p->lo;
    if (nodes < 1 || nodes > KVQ_MAX_TREE_NODES) return KVQ_ERR_ARG;
    if (lo.dtype != KVQ_DTYPE_BF16) return KVQ_ERR_UNSUPPORTED;
    const int D = lo.D;
    p->rows = nodes * lo.gqa;
    p->N = 16;
    while (p->N < p->rows && p->N < (D > 128 ? 64 : 128)) p->N *= 2;
    if (lo.scheme == KVQ_SCHEME_KIVI) {
        p->TT = 128 / lo.G * lo.G;
        p->stage = (int64_t)(128 / lo.G) * lo.rec;
    } else {
        p->TT = 128;
        p->stage = lo.scheme == KVQ_SCHEME_INT8 ? 256 * D + 1024 : lo.scheme == KVQ_SCHEME_INT4 ? 128 * D + 1024 : 256 * D;
    }
    p->stage = (p->stage + 127) / 128 * 128;
    if (tile_bytes(16, D) + p->stage <= kTreeSmemLimit)
        while (tile_bytes(p->N, D) + p->stage > kTreeSmemLimit) p->N /= 2;
    const int64_t tiles = tile_bytes(p->N, D), room = kTreeSmemLimit - tiles;
    p->share = 0;
    p->blocks = p->N <= 64 && D <= 128 ? 2 : 1;
    if (p->blocks == 2 && tiles + p->stage > kTreeSmemHalf) {
        if (p->N <= D && tiles - 256 * p->N + p->stage <= kTreeSmemHalf)
            p->share = 1;
        else
            p->blocks = 1;
    }
    const int64_t left = p->blocks == 2 ? kTreeSmemHalf - tiles + (p->share ? 256 * p->N : 0) : room;
    p->stages = left >= 2 * p->stage ? 2 : left >= p->stage ? 1 : 0;
    p->stage_at = static_cast<int>(tiles - (p->share ? 256 * p->N : 0));
    if (p->stages == 0) {
        if (lo.scheme != KVQ_SCHEME_KIVI || D != 256) return KVQ_ERR_UNSUPPORTED;
        p->stage = 0;
    }
    p->RT = (p->rows + p->N - 1) / p->N;
    const int64_t slots = kMaxTreeBlocks + (int64_t)lo.B * lo.H * p->RT;
    p->span_off = 256;
    p->ml_off = align256(p->span_off + (int64_t)lo.B * lo.H * p->RT * 8);
    p->o_off = align256(p->ml_off + slots * p->N * 8);
    p->bytes = align256(p->o_off + slots * p->N * D * 4);
    return KVQ_OK;
}

int launch_tree(TreeArgs& a, int N, cudaStream_t st) {
    const int D = a.lo.D;
    if (is_rows(a.lo.scheme))
        return D == 32 ? launch_tree_rows_d32(a, N, st) : D == 64 ? launch_tree_rows_d64(a, N, st)
             : D == 128 ? launch_tree_rows_d128(a, N, st) : launch_tree_rows_d256(a, N, st);
    if (is_fp8(a.lo.scheme))
        return D == 32 ? launch_tree_fp8_d32(a, N, st) : D == 64 ? launch_tree_fp8_d64(a, N, st)
             : D == 128 ? launch_tree_fp8_d128(a, N, st) : launch_tree_fp8_d256(a, N, st);
    if (a.stages == 0) return launch_tree_inplace_d256(a, N, st);    // (of 256 channels: tree_plan)
    switch (a.lo.bits) {
        case 2:
            return D == 64 ? launch_tree_kivi2_d64(a, N, st) : D == 128 ? launch_tree_kivi2_d128(a, N, st)
                                                                        : launch_tree_kivi2_d256(a, N, st);
        case 4:
            return D == 64 ? launch_tree_kivi4_d64(a, N, st) : D == 128 ? launch_tree_kivi4_d128(a, N, st)
                                                                        : launch_tree_kivi4_d256(a, N, st);
        default:
            return D == 64 ? launch_tree_kivi8_d64(a, N, st) : D == 128 ? launch_tree_kivi8_d128(a, N, st)
                                                                        : launch_tree_kivi8_d256(a, N, st);
    }
}

}  // namespace
}  // namespace kvq

extern "C" {

int kvq_tree_workspace_bytes(const kvq_config* cfg, int32_t nodes, uint64_t* out_bytes) {
    if (!cfg || !out_bytes) return KVQ_ERR_ARG;
    kvq::TreePlan p;
    const int rc = kvq::tree_plan(cfg, nodes, &p);
    if (rc != KVQ_OK) return rc;
    *out_bytes = static_cast<uint64_t>(p.bytes);
    return KVQ_OK;
}

int kvq_tree_attention(const kvq_config* cfg, const void* cache, int32_t layer, int32_t nodes, const void* q,
                       const void* k_draft, const void* v_draft, const uint8_t* mask, const int32_t* n_nodes,
                       float softmax_scale, void* out, void* workspace, uint64_t workspace_bytes,
                       kvq_stream_t stream) {
    if (!cfg || !cache || !q || !k_draft || !v_draft || !out || !workspace) return KVQ_ERR_ARG;
    kvq::TreeArgs a;
    kvq::TreePlan p;
    const int rc = kvq::tree_plan(cfg, nodes, &p);
    if (rc != KVQ_OK) return rc;
    a.lo = p.lo;
    if (layer < 0 || layer >= a.lo.L) return KVQ_ERR_ARG;
    if (a.lo.PG > 0 && a.lo.NG > 0 && !a.lo.table) return KVQ_ERR_ARG;
    if (workspace_bytes < static_cast<uint64_t>(p.bytes)) return KVQ_ERR_WORKSPACE;
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
    a.qscale = softmax_scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ws = static_cast<uint8_t*>(workspace);
    a.rows = p.rows;
    a.RT = p.RT;
    a.gshift = a.lo.gqa == 1 ? 0 : a.lo.gqa == 2 ? 1 : a.lo.gqa == 4 ? 2 : 3;
    a.TT = p.TT;
    a.TG = a.lo.scheme == KVQ_SCHEME_KIVI ? p.TT / a.lo.G : 0;
    a.gvshift = 0;
    while ((1 << a.gvshift) < a.lo.Gv) ++a.gvshift;
    a.pieces = a.lo.scheme == KVQ_SCHEME_KIVI ? (a.lo.D + a.lo.NGv * a.lo.G) / 8 : 1;
    a.pieces_inverse = static_cast<uint32_t>((0x100000000ull + a.pieces - 1) / a.pieces);
    for (int i = 0; i < 8; ++i) a.group_of[i] = a.TG > 0 && 16 * i < p.TT ? 16 * i / a.lo.G : 0;
    a.stages = p.stages;
    a.share = p.share;
    a.blocks = p.blocks;
    a.stage_at = p.stage_at;
    a.stage_bytes = static_cast<int>(p.stage);
    a.span_off = p.span_off;
    a.ml_off = p.ml_off;
    a.o_off = p.o_off;
    if (a.lo.rope_base > 0.0f)
        for (int i = 0; i < a.lo.D / 2; ++i)
            a.rope_w[i] = static_cast<float>(std::pow(static_cast<double>(a.lo.rope_base), -2.0 * i / a.lo.D));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return kvq::launch_tree(a, p.N, st);
}

}  // extern "C"
