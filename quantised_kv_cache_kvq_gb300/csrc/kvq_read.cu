// kvq_read.cu -- reading cached tokens back as bf16 or fp32 rows.
#include <cstdint>

#include "kvq_elements.cuh"
#include "kvq_internal.cuh"
#include "kvq_launch.h"

namespace kvq {
namespace {

struct ReadArgs {
    Layout lo;
    uint8_t* cache;
    int layer, seq_begin, first, count;
    const int32_t* starts;
    void* out[2];
};

template <typename T>
__global__ void k_read(ReadArgs a) {
    const Layout& lo = a.lo;
    const int bi = blockIdx.y, b = a.seq_begin + bi;
    const int32_t* st = state_ptr(lo, a.cache, a.layer, b);
    const int n = st[0], qn = st[1];
    const int64_t row = blockIdx.x / lo.H, h = blockIdx.x % lo.H;
    const int64_t t = (a.starts ? a.starts[bi] : a.first) + row;
    bool bad = false;
    for (int c = threadIdx.x; c < lo.D; c += blockDim.x)
        for (int kv = 0; kv < 2; ++kv) {
            if (!a.out[kv]) continue;
            const float x = t >= 0 && t < n ? cached_element(lo, a.cache, a.layer, b, h, qn, t, c, kv, &bad) : 0.0f;
            static_cast<T*>(a.out[kv])[(((int64_t)bi * a.count + row) * lo.H + h) * lo.D + c] = static_cast<T>(x);
        }
    if (bad) atomicOr(reinterpret_cast<uint32_t*>(a.cache), KVQ_STATUS_BAD_PAGE);
}

}  // namespace
}  // namespace kvq

extern "C" int kvq_read_tokens(const kvq_config* cfg, void* cache, int32_t layer, int32_t seq_begin,
                               int32_t seq_count, const int32_t* starts, int32_t first, int32_t count, void* k_out,
                               void* v_out, int32_t out_dtype, kvq_stream_t stream) {
    if (!cfg || !cache) return KVQ_ERR_ARG;
    kvq::ReadArgs a;
    const int rc = kvq::make_layout(cfg, cfg->max_tokens, &a.lo);
    if (rc != KVQ_OK) return rc;
    if (layer < 0 || layer >= a.lo.L || seq_begin < 0 || seq_count < 0 || seq_begin + (int64_t)seq_count > a.lo.B)
        return KVQ_ERR_ARG;
    if (count < 0 || (!starts && first < 0)) return KVQ_ERR_ARG;
    if (out_dtype != KVQ_DTYPE_BF16 && out_dtype != KVQ_DTYPE_F32) return KVQ_ERR_ARG;
    if (a.lo.PG > 0 && a.lo.NG > 0 && !a.lo.table) return KVQ_ERR_ARG;
    auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(cache, 256) || off(k_out, 16) || off(v_out, 16) || off(starts, 4) || off(a.lo.table, 4)) return KVQ_ERR_ALIGN;
    if (seq_count == 0 || count == 0 || (!k_out && !v_out)) return KVQ_OK;
    a.cache = static_cast<uint8_t*>(cache);
    a.layer = layer;
    a.seq_begin = seq_begin;
    a.first = first;
    a.count = count;
    a.starts = starts;
    a.out[0] = k_out;
    a.out[1] = v_out;
    const dim3 grid(static_cast<unsigned>(count * a.lo.H), seq_count);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (out_dtype == KVQ_DTYPE_BF16)
        kvq::k_read<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
    else
        kvq::k_read<float><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
