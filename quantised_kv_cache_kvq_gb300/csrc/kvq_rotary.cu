// kvq_rotary.cu -- rotary positions of queries and keys.
//
// Pair (x, y) of a head at position t becomes m (x cos a - y sin a, y cos a + x sin a) with
// a = t * w_i in binary32.  The angle belongs to a token and a pair, not to a head, so a block
// computes a token's cosines and sines once, in shared memory, and turns all its heads with
// them; the sine of a far position costs nothing next to the rows then.  Every channel is
// read and written once: the kernel is bound by memory traffic (16384 tokens of 32 + 8 bf16
// heads of 128: 57 us, 5.9 TB/s, 87% of a plain copy; 4099 tokens of 16 + 16 float32 heads, half
// of each turned: 29 us, 4.7 TB/s), or by its launch for the few rows of a decode step (8
// tokens: 2.5 us on the device).
#include <cmath>
#include <cstdint>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = KVQ_MAX_ROTARY_DIM / 2;

struct RopeArgs {
    const int32_t* positions;
    const void* x[2];               // q, k
    void* y[2];
    int64_t x_stride[2], y_stride[2];
    int32_t heads[2];
    int64_t tokens;
    int32_t D, R, turn_units, units;   // units of a head: turn_units rotated, the rest copied
    float magnitude;
    float sign;                     // -1: the transposed product
    float w[kMaxPairs];
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

// One block per token: threads (u, v) turn unit u of heads v, v + blockDim.y, ...  A unit is
// VEC pairs (two vectors of VEC channels: the pairs' first and second channels, or 2 VEC
// adjacent ones), or VEC copied channels.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a) {
    __shared__ float2 table[kMaxPairs];
    using P = Pack<T, VEC>;
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const float pos = static_cast<float>(a.positions[t]);
    for (int i = tid; i < a.R / 2; i += blockDim.x * blockDim.y) {
        float s, c;
        sincosf(__fmul_rn(pos, a.w[i]), &s, &c);
        table[i] = make_float2(c * a.magnitude, s * a.magnitude * a.sign);
    }
    __syncthreads();
    for (int u = threadIdx.x; u < a.units; u += blockDim.x) {
        const bool turns = u < a.turn_units;
        // first channel of the unit's first and second vector
        const int c0 = turns ? (HALF ? u * VEC : u * 2 * VEC) : a.R + (u - a.turn_units) * VEC;
        const int c1 = HALF ? c0 + a.R / 2 : c0 + VEC;
        for (int hh = threadIdx.y; hh < a.heads[0] + a.heads[1]; hh += blockDim.y) {
            const int which = hh >= a.heads[0];
            const int h = hh - (which ? a.heads[0] : 0);
            const T* x = static_cast<const T*>(a.x[which]) + t * a.x_stride[which] + (int64_t)h * a.D;
            T* y = static_cast<T*>(a.y[which]) + t * a.y_stride[which] + (int64_t)h * a.D;
            if (!turns) {
                *reinterpret_cast<P*>(y + c0) = *reinterpret_cast<const P*>(x + c0);
                continue;
            }
            const P p0 = *reinterpret_cast<const P*>(x + c0), p1 = *reinterpret_cast<const P*>(x + c1);
            P o0, o1;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 cs = table[u * VEC + e];
                // pair e of the unit: element e of both vectors, or elements 2e, 2e + 1 of the
                // 2 VEC adjacent ones
                const int i0 = HALF ? e : 2 * e, i1 = HALF ? e + VEC : 2 * e + 1;
                const float v0 = to_float(i0 < VEC ? p0.v[i0 % VEC] : p1.v[i0 % VEC]);
                const float v1 = to_float(i1 < VEC ? p0.v[i1 % VEC] : p1.v[i1 % VEC]);
                T r0, r1;
                from_float(v0 * cs.x - v1 * cs.y, &r0);
                from_float(v1 * cs.x + v0 * cs.y, &r1);
                if (i0 < VEC) o0.v[i0 % VEC] = r0; else o1.v[i0 % VEC] = r0;
                if (i1 < VEC) o0.v[i1 % VEC] = r1; else o1.v[i1 % VEC] = r1;
            }
            *reinterpret_cast<P*>(y + c0) = o0;
            *reinterpret_cast<P*>(y + c1) = o1;
        }
    }
}

template <typename T, int VEC>
cudaError_t launch_rope(const kvq_rope_config& rc, RopeArgs& a, cudaStream_t stream) {
    a.turn_units = a.R / 2 / VEC;
    a.units = a.turn_units + (a.D - a.R) / VEC;
    // few rows: as many threads as there are; many: small blocks, more of them on an SM (16384
    // tokens of 40 heads of 128 bf16 channels: 57 us with 128 threads, 65 with 256; 8 tokens: 6.1
    // and 4.5)
    const int threads = a.tokens < 2 * 152 ? kRopeThreads : kRopeThreads / 2;
    const int ux = a.units < threads ? a.units : threads;
    const int total = a.heads[0] + a.heads[1];
    int uy = threads / ux;
    uy = uy < total ? uy : total;
    const dim3 grid(static_cast<unsigned>(a.tokens)), block(ux, uy);
    if (rc.layout == KVQ_ROPE_HALF)
        k_rope<T, VEC, true><<<grid, block, 0, stream>>>(a);
    else
        k_rope<T, VEC, false><<<grid, block, 0, stream>>>(a);
    return cudaGetLastError();
}

bool finite_above(float x, float lo) { return x > lo && x <= 3.0e38f; }

// Elements per vector access: the widest power of two up to 16 bytes that divides the row
// pieces and that the pointers and strides are aligned to.
int vector_width(const RopeArgs& a, int size) {
    int v = 16 / size;
    auto fits = [&](int vec) {
        if (a.R / 2 % vec || (a.D - a.R) % vec || a.D % vec) return false;
        for (int w = 0; w < 2; ++w) {
            if (a.heads[w] == 0) continue;
            if (reinterpret_cast<uintptr_t>(a.x[w]) % (vec * size) || reinterpret_cast<uintptr_t>(a.y[w]) % (vec * size))
                return false;
            if (a.tokens > 1 && (a.x_stride[w] % vec || a.y_stride[w] % vec)) return false;
        }
        return true;
    };
    while (v > 1 && !fits(v)) v /= 2;
    return v;
}

int check_rope(const kvq_rope_config* r) {
    if (!r) return KVQ_ERR_ARG;
    if (r->head_dim < 1 || r->head_dim > 1024) return KVQ_ERR_ARG;
    if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > r->head_dim || r->rotary_dim > KVQ_MAX_ROTARY_DIM)
        return KVQ_ERR_ARG;
    if (r->layout != KVQ_ROPE_HALF && r->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_ARG;
    if (r->dtype != KVQ_DTYPE_BF16 && r->dtype != KVQ_DTYPE_F32) return KVQ_ERR_ARG;
    return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" {

int kvq_rope_frequencies(const kvq_rope_config* rope, float* w) {
    const int rc = kvq::check_rope(rope);
    if (rc != KVQ_OK) return rc;
    if (!w) return KVQ_ERR_ARG;
    const int s = rope->scaling, R = rope->rotary_dim;
    if (s < KVQ_ROPE_SCALE_NONE || s > KVQ_ROPE_SCALE_BY_PARTS) return KVQ_ERR_ARG;
    if (!kvq::finite_above(rope->base, 0.0f)) return KVQ_ERR_ARG;
    if (s != KVQ_ROPE_SCALE_NONE && !kvq::finite_above(rope->factor, 0.0f)) return KVQ_ERR_ARG;
    if (s == KVQ_ROPE_SCALE_NTK && R < 4) return KVQ_ERR_ARG;
    if (s == KVQ_ROPE_SCALE_BY_PARTS &&
        (!(rope->low >= -3.0e38f) || !kvq::finite_above(rope->high, rope->low) || rope->original_context < 1))
        return KVQ_ERR_ARG;
    const double f = rope->factor;
    double base = rope->base;
    if (s == KVQ_ROPE_SCALE_NTK) base *= std::pow(f, static_cast<double>(R) / (R - 2));
    for (int i = 0; i < R / 2; ++i) {
        double v = std::pow(base, -2.0 * i / R);
        if (s == KVQ_ROPE_SCALE_LINEAR) v /= f;
        if (s == KVQ_ROPE_SCALE_BY_PARTS) {
            const double turns = rope->original_context * v / (2.0 * 3.14159265358979323846);
            double g = (turns - rope->low) / (static_cast<double>(rope->high) - rope->low);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            v = g * v + (1.0 - g) * v / f;
        }
        w[i] = static_cast<float>(v);
    }
    return KVQ_OK;
}

int kvq_rope(const kvq_rope_config* rope, const float* w, const int32_t* positions, int64_t tokens, const void* q,
             void* q_out, int32_t q_heads, int64_t q_stride, int64_t q_out_stride, const void* k, void* k_out,
             int32_t kv_heads, int64_t k_stride, int64_t k_out_stride, uint32_t flags, kvq_stream_t stream) {
    const int rc = kvq::check_rope(rope);
    if (rc != KVQ_OK) return rc;
    if (!w || tokens < 0 || tokens > 0x7fffffff || q_heads < 0 || kv_heads < 0 || q_heads > 65536 || kv_heads > 65536)
        return KVQ_ERR_ARG;
    if (flags & ~static_cast<uint32_t>(KVQ_ROPE_TRANSPOSE)) return KVQ_ERR_ARG;
    if (tokens == 0 || q_heads + kv_heads == 0) return KVQ_OK;
    if (!positions || (q_heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out))) return KVQ_ERR_ARG;
    const int size = rope->dtype == KVQ_DTYPE_BF16 ? 2 : 4;
    kvq::RopeArgs a;
    a.positions = positions;
    a.x[0] = q;
    a.x[1] = k;
    a.y[0] = q_out;
    a.y[1] = k_out;
    a.x_stride[0] = q_stride;
    a.x_stride[1] = k_stride;
    a.y_stride[0] = q_out_stride;
    a.y_stride[1] = k_out_stride;
    a.heads[0] = q_heads;
    a.heads[1] = kv_heads;
    a.tokens = tokens;
    a.D = rope->head_dim;
    a.R = rope->rotary_dim;
    a.magnitude = rope->magnitude;
    a.sign = (flags & KVQ_ROPE_TRANSPOSE) ? -1.0f : 1.0f;
    for (int i = 0; i < 2; ++i) {
        if (a.heads[i] == 0) continue;
        const int64_t row = (int64_t)a.heads[i] * a.D;
        if (tokens > 1 && (a.x_stride[i] < row || a.y_stride[i] < row)) return KVQ_ERR_ARG;
        if (a.x[i] == a.y[i] && tokens > 1 && a.x_stride[i] != a.y_stride[i]) return KVQ_ERR_ARG;
        if (reinterpret_cast<uintptr_t>(a.x[i]) % size || reinterpret_cast<uintptr_t>(a.y[i]) % size) return KVQ_ERR_ALIGN;
    }
    if (reinterpret_cast<uintptr_t>(positions) % 4) return KVQ_ERR_ALIGN;
    for (int i = 0; i < a.R / 2; ++i) a.w[i] = w[i];
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    const int vec = kvq::vector_width(a, size);
    if (size == 2) {
        e = vec == 8 ? kvq::launch_rope<__nv_bfloat16, 8>(*rope, a, s)
          : vec == 4 ? kvq::launch_rope<__nv_bfloat16, 4>(*rope, a, s)
          : vec == 2 ? kvq::launch_rope<__nv_bfloat16, 2>(*rope, a, s)
                     : kvq::launch_rope<__nv_bfloat16, 1>(*rope, a, s);
    } else {
        e = vec == 4 ? kvq::launch_rope<float, 4>(*rope, a, s)
          : vec == 2 ? kvq::launch_rope<float, 2>(*rope, a, s)
                     : kvq::launch_rope<float, 1>(*rope, a, s);
    }
    return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
