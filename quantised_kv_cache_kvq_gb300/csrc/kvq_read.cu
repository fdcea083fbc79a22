// kvq_read.cu -- reading cached tokens back as bf16 or fp32 rows.
//
// x = code * scale + zero (KIVI), code * scale (INT8, INT4, FP8), in binary32 as a product and
// then a sum, rounded once to the output's type; the window's and the outliers' bf16 values as
// they are.  A packed token's keys and values of one head come from about 100 to 270 bytes and
// go to 512 (bf16, 128 channels): the kernel is bound by its stores where codes are bytes (FP8,
// 24 x 8192 tokens, 8 heads: 214 us, 5.6 TB/s, 83% of a plain copy) and by the instructions that
// take 2-bit codes apart elsewhere (8 x 4096 tokens: 39 us, 61%).
//
// A block takes one tile of one sequence and KV head -- a KIVI group, or 64 tokens of the other
// caches -- and a thread 16 adjacent channels of a token at a time, so that the threads of a row
// write whole lines.  The record's value codes lie in the decode's order, in which the two
// tokens t and t + 8 of a 16-token piece share their words: a thread takes both.  FP8 values
// lie by channel, 16 tokens each: a thread turns 4 channels by 4 tokens around in registers.
#include <cstdint>

#include <cuda_fp8.h>

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
    int tile;       // tokens of a block: a KIVI group, or 64
    int dshift;     // log2 head_dim
    int gvshift;    // KIVI: log2 of the value group
    int64_t row;    // elements of an output token: kv_heads * head_dim
};

// 16 (or 4) adjacent channels to an output row.
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(bf16x2(x[8 * i], x[8 * i + 1]), bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                                    bf16x2(x[8 * i + 4], x[8 * i + 5]), bf16x2(x[8 * i + 6], x[8 * i + 7]));
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A small unsigned integer as binary32: its bits under 2^23's, less 2^23 (both exact).
__device__ __forceinline__ float small_float(uint32_t c) { return __uint_as_float(0x4b000000u | c) - 8388608.0f; }
__device__ __forceinline__ float code_value(uint32_t c, float s, float z) { return __fadd_rn(__fmul_rn(small_float(c), s), z); }
__device__ __forceinline__ void halves16(const uint8_t* p, float (&x)[16]) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ float fp8_value(uint32_t byte, bool e4m3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), e4m3 ? __NV_E4M3 : __NV_E5M2);
    return __half2float(__half(h));
}

// A block's part of the output: tokens [lo, hi) of sequence bi, whose rows begin at `first`.
template <typename T>
struct Rows {
    T* out[2];          // row of token 0, this head's channels (NULL: not asked for)
    int64_t row;
    int lo, hi;
    __device__ __forceinline__ T* at(int kv, int t, int c) const { return out[kv] + (int64_t)t * row + c; }
};

// One KIVI group: tokens t0 .. of record `rec`.
template <int BITS, int NT, typename T>
__device__ __forceinline__ void read_group(const ReadArgs& a, const uint8_t* rec, int t0, const Rows<T>& o) {
    const Layout& lo = a.lo;
    const int D = lo.D, G = lo.G, units = D / 16, ushift = a.dshift - 4;
    constexpr uint32_t MASK = (1u << BITS) - 1;
    if (o.out[0]) {
        const int u = threadIdx.x & (units - 1);
        float s[16], z[16];
        halves16(rec + lo.kc + lo.vc + 32 * u, s);
        halves16(rec + lo.kc + lo.vc + 2 * D + 32 * u, z);
        for (int i = threadIdx.x >> ushift; i < G; i += NT >> ushift) {
            const int t = t0 + i;
            if (t < o.lo || t >= o.hi) continue;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + (i * D + 16 * u) * BITS / 8);
            float x[16];
#pragma unroll
            for (int w = 0; w < BITS / 2; ++w) {
                const uint32_t v = src[w];
#pragma unroll
                for (int j = 0; j < 32 / BITS; ++j)
                    x[w * (32 / BITS) + j] = code_value((v >> (BITS * j)) & MASK, s[w * (32 / BITS) + j], z[w * (32 / BITS) + j]);
            }
            store16(o.at(0, t, 16 * u), x);
        }
    }
    if (o.out[1]) {
        // items (16-token piece, token pair, 16 channels): lane 4 g + i of the codes' order holds
        // channels 16 q + g + 8 r of tokens 2 i + s and 2 i + s + 8
        constexpr int HW = 16 / BITS;
        const int wpl = D * BITS / 64, sw = wpl < 4 ? wpl : 4;
        for (int it = threadIdx.x; it < G / 2 * units; it += NT) {
            const int q = it & (units - 1), pair = it >> ushift, piece = pair >> 3, tt = pair & 7;
            const int ta = t0 + 16 * piece + tt;
            const bool wa = ta >= o.lo && ta < o.hi, wb = ta + 8 >= o.lo && ta + 8 < o.hi;
            if (!wa && !wb) continue;
            const int w = 2 * (2 * q / HW) + (tt & 1), bit = BITS * (2 * q % HW);
            const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + lo.kc) + piece * 32 * wpl + (w / sw) * 32 * sw +
                                  (tt >> 1) * sw + w % sw;
            const int at = ((16 * q) >> a.gvshift) * G + 16 * piece + 2 * tt;
            const uint8_t* par = rec + lo.kc + lo.vc + lo.kp;
            const float2 s = __half22float2(*reinterpret_cast<const __half2*>(par + 2 * at));
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(par + 2 * (lo.NGv * G + at)));
            float x[16], y[16];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const uint32_t v = src[4 * g * sw] >> bit;
                x[g] = code_value(v & MASK, s.x, z.x);
                x[g + 8] = code_value((v >> BITS) & MASK, s.x, z.x);
                y[g] = code_value((v >> 16) & MASK, s.y, z.y);
                y[g + 8] = code_value((v >> (16 + BITS)) & MASK, s.y, z.y);
            }
            if (wa) store16(o.at(1, ta, 16 * q), x);
            if (wb) store16(o.at(1, ta + 8, 16 * q), y);
        }
    }
    if (lo.K > 0) {
        // the side lists' elements over the dense ones, behind them
        __syncthreads();
        const uint32_t* side = reinterpret_cast<const uint32_t*>(rec + lo.kc + lo.vc + lo.kp + lo.vp);
        if (o.out[0])
            for (int i = threadIdx.x; i < lo.K * D; i += NT) {
                const uint32_t e = side[i];
                const int t = t0 + static_cast<int>(e & 0xffffu);
                if (t >= o.lo && t < o.hi) store1(o.at(0, t, i & (D - 1)), __uint_as_float(e & 0xffff0000u));
            }
        if (o.out[1])
            for (int i = threadIdx.x; i < lo.K * lo.NGv * G; i += NT) {
                const uint32_t e = side[lo.K * D + i];
                const int at = i % (lo.NGv * G), in = at % G, tt = in & 15;
                const int t = t0 + in - tt + (tt >> 1) + 8 * (tt & 1);
                if (t >= o.lo && t < o.hi)
                    store1(o.at(1, t, ((at / G) << a.gvshift) + static_cast<int>(e & 0xffffu)), __uint_as_float(e & 0xffff0000u));
            }
    }
}

// bf16 rows of the KIVI window, tokens [max(lo, first), hi): token t in slot t mod C.
template <int NT, typename T>
__device__ __forceinline__ void read_window(const ReadArgs& a, const uint8_t* ring, int n, const Rows<T>& o) {
    const int D = a.lo.D, units = D / 16, ushift = a.dshift - 4;
    for (int it = threadIdx.x; it < (o.hi - o.lo) * 2 * units; it += NT) {
        const int u = it & (units - 1), kv = (it >> ushift) & 1, t = o.lo + (it >> (ushift + 1));
        if (!o.out[kv]) continue;
        float x[16] = {};
        if (t < n) {
            const uint8_t* src = ring + (int64_t)(static_cast<uint32_t>(t) % static_cast<uint32_t>(a.lo.C)) * (4 * D) + kv * 2 * D + 32 * u;
            const uint4 p = reinterpret_cast<const uint4*>(src)[0], q = reinterpret_cast<const uint4*>(src)[1];
            const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        store16(o.at(kv, t, 16 * u), x);
    }
}

// Rows of the tokens that the cache does not hold: 0.
template <int NT, typename T>
__device__ __forceinline__ void zero_rows(const ReadArgs& a, const Rows<T>& o) {
    const int units = a.lo.D / 16, ushift = a.dshift - 4;
    const float x[16] = {};
    for (int it = threadIdx.x; it < (o.hi - o.lo) * 2 * units; it += NT) {
        const int kv = (it >> ushift) & 1;
        if (o.out[kv]) store16(o.at(kv, o.lo + (it >> (ushift + 1)), 16 * (it & (units - 1))), x);
    }
}

// INT8 or INT4 rows.
template <bool INT8, int NT, typename T>
__device__ __forceinline__ void read_rows(const ReadArgs& a, const uint8_t* base, const Rows<T>& o) {
    const int D = a.lo.D, units = D / 16, ushift = a.dshift - 4;
    const int64_t width = INT8 ? D : D / 2;
    for (int it = threadIdx.x; it < (o.hi - o.lo) * 2 * units; it += NT) {
        const int u = it & (units - 1), kv = (it >> ushift) & 1, t = o.lo + (it >> (ushift + 1));
        if (!o.out[kv]) continue;
        const uint8_t* src = base + ((int64_t)kv * a.lo.T16 + t) * width + u * (INT8 ? 16 : 8);
        const float s = reinterpret_cast<const float*>(base + 2 * (int64_t)a.lo.T16 * width)[(int64_t)kv * a.lo.T16 + t];
        float x[16];
        if constexpr (INT8) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = __fmul_rn(small_float(((w[i / 4] ^ 0x80808080u) >> (8 * (i & 3))) & 0xffu) - 128.0f, s);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = __fmul_rn(small_float(((w[i / 8] ^ 0x88888888u) >> (4 * (i & 7))) & 0xfu) - 8.0f, s);
        }
        store16(o.at(kv, t, 16 * u), x);
    }
}

// FP8 tiles: key rows in quarters (channels 2i, 2i + 1, 2i + 8, 2i + 9 of block kb at byte 4 kb
// of quarter i), values [channel][16 tokens] per tile, token tt at byte 2 (tt mod 8) + tt / 8.
template <int NT, typename T>
__device__ __forceinline__ void read_fp8(const ReadArgs& a, const uint8_t* base, const float* scales, const Rows<T>& o) {
    const int D = a.lo.D, units = D / 16, ushift = a.dshift - 4;
    const bool e4m3 = a.lo.scheme == KVQ_SCHEME_FP8_E4M3;
    if (o.out[0]) {
        const float s = scales[0];
        for (int it = threadIdx.x; it < (o.hi - o.lo) * units; it += NT) {
            const int u = it & (units - 1), t = o.lo + (it >> ushift);
            float x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(base + (int64_t)t * D + i * (D / 4) + 4 * u);
                x[2 * i] = __fmul_rn(fp8_value(w & 0xffu, e4m3), s);
                x[2 * i + 1] = __fmul_rn(fp8_value((w >> 8) & 0xffu, e4m3), s);
                x[2 * i + 8] = __fmul_rn(fp8_value((w >> 16) & 0xffu, e4m3), s);
                x[2 * i + 9] = __fmul_rn(fp8_value(w >> 24, e4m3), s);
            }
            store16(o.at(0, t, 16 * u), x);
        }
    }
    if (o.out[1]) {
        const float s = scales[1];
        const uint8_t* vbase = base + (int64_t)a.lo.T16 * D;
        const int quads = D / 4, qshift = a.dshift - 2, p0 = o.lo >> 4, pieces = ((o.hi - 1) >> 4) - p0 + 1;
        for (int it = threadIdx.x; it < pieces * 4 * quads; it += NT) {
            const int q = it & (quads - 1), k = (it >> qshift) & 3, piece = p0 + (it >> (qshift + 2));
            const uint8_t* src = vbase + (int64_t)piece * 16 * D + 64 * q + 4 * k;      // bytes 4 k .. of channels 4 q ..
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(src + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {       // byte 4 k + j: token (4 k + j) / 2 + 8 ((4 k + j) mod 2)
                const int t = 16 * piece + 2 * k + (j >> 1) + 8 * (j & 1);
                if (t < o.lo || t >= o.hi) continue;
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __fmul_rn(fp8_value((w[i] >> (8 * j)) & 0xffu, e4m3), s);
                store4(o.at(1, t, 4 * q), x);
            }
        }
    }
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) k_read(const __grid_constant__ ReadArgs a) {
    const Layout& lo = a.lo;
    const int bi = blockIdx.z, b = a.seq_begin + bi, h = blockIdx.y;
    const int32_t* st = state_ptr(lo, a.cache, a.layer, b);
    const int n = st[0], qn = st[1];
    const int64_t first = a.starts ? a.starts[bi] : a.first, last = first + a.count;
    // tiles are aligned to token 0; the first one may lie before it
    const int64_t tile0 = first >= 0 ? first / a.tile : -((-first + a.tile - 1) / a.tile);
    const int64_t t0 = (tile0 + blockIdx.x) * a.tile;
    const int64_t from = t0 > first ? t0 : first, to = t0 + a.tile < last ? t0 + a.tile : last;
    if (from >= to) return;
    // rows are addressed by their token: back from the output's first row
    Rows<T> o;
    o.row = a.row;
    int64_t shift = 0;
    if (to <= 0 || from >= n) {                 // nothing of it is held
        shift = from;
        o.lo = 0;
        o.hi = static_cast<int>(to - from);
    } else {
        o.lo = static_cast<int>(from);          // (from < n < 2^31; to may lie past it)
        o.hi = static_cast<int>(to);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
        o.out[kv] = a.out[kv] ? static_cast<T*>(a.out[kv]) + ((int64_t)bi * a.count + shift - first) * a.row + (int64_t)h * lo.D : nullptr;
    if (shift != 0 || to <= 0 || from >= n) {
        zero_rows<NT>(a, o);
        return;
    }
    if (lo.scheme == KVQ_SCHEME_KIVI) {
        if (t0 >= qn) {
            read_window<NT>(a, a.cache + lo.ring_off + unit_index(lo, a.layer, b, h) * lo.C * (int64_t)(4 * lo.D), n, o);
            return;
        }
        const int64_t off = group_offset(lo, a.layer, b, h, t0 / lo.G);
        if (off < 0) {                          // a table entry outside the pool
            if (threadIdx.x == 0) atomicOr(reinterpret_cast<uint32_t*>(a.cache), KVQ_STATUS_BAD_PAGE);
            zero_rows<NT>(a, o);
            return;
        }
        if (lo.bits == 2) read_group<2, NT>(a, a.cache + off, static_cast<int>(t0), o);
        else if (lo.bits == 4) read_group<4, NT>(a, a.cache + off, static_cast<int>(t0), o);
        else read_group<8, NT>(a, a.cache + off, static_cast<int>(t0), o);
        return;
    }
    const uint8_t* base = a.cache + lo.data_off + unit_index(lo, a.layer, b, h) * lo.unit;
    if (o.hi > n) {                             // the rows past the sequence's tokens
        Rows<T> past = o;
        past.lo = n;
        zero_rows<NT>(a, past);
        o.hi = n;
    }
    if (lo.scheme == KVQ_SCHEME_INT8) read_rows<true, NT>(a, base, o);
    else if (lo.scheme == KVQ_SCHEME_INT4) read_rows<false, NT>(a, base, o);
    else read_fp8<NT>(a, base, reinterpret_cast<const float*>(a.cache + lo.scales_off) + ((int64_t)a.layer * lo.H + h) * 2, o);
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
    if (a.lo.H > 65535) return KVQ_ERR_UNSUPPORTED;
    a.cache = static_cast<uint8_t*>(cache);
    a.layer = layer;
    a.first = first;
    a.count = count;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.tile = a.lo.scheme == KVQ_SCHEME_KIVI ? a.lo.G : 64;
    a.row = (int64_t)a.lo.H * a.lo.D;
    a.dshift = a.gvshift = 0;
    while ((1 << a.dshift) < a.lo.D) ++a.dshift;
    while ((1 << a.gvshift) < a.lo.Gv) ++a.gvshift;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // sequences in launches of at most 65535, tiles of the widest range that a start allows
    for (int done = 0; done < seq_count; done += 65535) {
        const int now = seq_count - done < 65535 ? seq_count - done : 65535;
        const int64_t rows = (int64_t)done * count * a.row * (out_dtype == KVQ_DTYPE_BF16 ? 2 : 4);
        a.seq_begin = seq_begin + done;
        a.starts = starts ? starts + done : nullptr;
        a.out[0] = k_out ? static_cast<uint8_t*>(k_out) + rows : nullptr;
        a.out[1] = v_out ? static_cast<uint8_t*>(v_out) + rows : nullptr;
        const dim3 grid(static_cast<unsigned>((count + (int64_t)a.tile - 2) / a.tile + 1), a.lo.H, now);
        // many blocks: small ones, more of them on an SM at different points of their work (a
        // 2-bit layer of 8 x 4096 tokens: 40 us with 64 threads, 43 with 128, 59 with 256); few:
        // large ones, for latency (257 tokens of one sequence: 10.4, 8.3 and 7.3)
        const bool many = (int64_t)grid.x * grid.y * grid.z >= 8 * 152;
        if (out_dtype == KVQ_DTYPE_BF16) {
            if (many) kvq::k_read<__nv_bfloat16, 64><<<grid, 64, 0, s>>>(a);
            else kvq::k_read<__nv_bfloat16, 256><<<grid, 256, 0, s>>>(a);
        } else {
            if (many) kvq::k_read<float, 64><<<grid, 64, 0, s>>>(a);
            else kvq::k_read<float, 256><<<grid, 256, 0, s>>>(a);
        }
        if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
    }
    return KVQ_OK;
}
