// kvq_elements.cuh -- single dequantised elements of a cache (layout in kvq_internal.cuh).
#pragma once

#include <cuda_fp8.h>

#include "kvq_internal.cuh"

namespace kvq {

// Within a group record: the bit of the code of (token t, channel c) of the values, and the
// index of its (scale, zero) pair in the value parameters.
__device__ __forceinline__ int record_value_bit(const Layout& lo, int t, int c) {
    const int hw = 16 / lo.bits, wpl = lo.D * lo.bits / 64, sw = wpl < 4 ? wpl : 4;
    const int tt = t & 15, lane = 4 * (c & 7) + ((tt & 7) >> 1);
    const int j = 2 * (c >> 4) + ((c & 15) >> 3);
    const int w = 2 * (j / hw) + (tt & 1);
    const int word = (t >> 4) * 32 * wpl + (w / sw) * 32 * sw + lane * sw + w % sw;
    return word * 32 + 16 * (tt >> 3) + lo.bits * (j % hw);
}
__device__ __forceinline__ int record_value_param(const Layout& lo, int t, int c) {
    const int tt = t & 15;
    return (c / lo.Gv) * lo.G + (t - tt) + 2 * (tt & 7) + (tt >> 3);
}
__device__ __forceinline__ float scaled_code(int code, float s, float z) {
    return __fadd_rn(__fmul_rn(static_cast<float>(code), s), z);
}

// Key (kv = 0) or value (kv = 1) of channel c of token t < n of unit (l, b, h); qn as in the
// sequence's state.  *bad is set where the token's page is outside the pool.
__device__ inline float cached_element(const Layout& lo, const uint8_t* cache, int l, int b, int h, int qn, int64_t t,
                                       int c, int kv, bool* bad) {
    const int D = lo.D;
    if (lo.scheme == KVQ_SCHEME_KIVI) {
        if (t >= qn) {
            const uint16_t* slot = reinterpret_cast<const uint16_t*>(
                cache + lo.ring_off + (unit_index(lo, l, b, h) * lo.C + t % lo.C) * (int64_t)(4 * D));
            return bf16_bits_to_float(slot[kv * D + c]);
        }
        const int64_t off = group_offset(lo, l, b, h, t / lo.G);
        if (off < 0) {
            *bad = true;
            return 0.0f;
        }
        const uint8_t* rec = cache + off;
        const int i = static_cast<int>(t % lo.G);
        const int mask = (1 << lo.bits) - 1;
        const int gi = record_value_param(lo, i, c);
        if (lo.K > 0) {
            const uint32_t* side = reinterpret_cast<const uint32_t*>(rec + lo.kc + lo.vc + lo.kp + lo.vp);
            const int want = kv ? c % lo.Gv : i;
            for (int e = 0; e < lo.K; ++e) {
                const uint32_t x = kv ? side[lo.K * D + e * lo.NGv * lo.G + gi] : side[e * D + c];
                if (static_cast<int>(x & 0xffffu) == want) return bf16_bits_to_float(static_cast<uint16_t>(x >> 16));
            }
        }
        const __half* par = reinterpret_cast<const __half*>(rec + lo.kc + lo.vc + (kv ? lo.kp : 0));
        const int bit = kv ? record_value_bit(lo, i, c) : (i * D + c) * lo.bits;
        const int code = (rec[(kv ? lo.kc : 0) + (bit >> 3)] >> (bit & 7)) & mask;
        return kv ? scaled_code(code, __half2float(par[gi]), __half2float(par[lo.G * lo.NGv + gi]))
                  : scaled_code(code, __half2float(par[c]), __half2float(par[D + c]));
    }
    const uint8_t* base = cache + lo.data_off + unit_index(lo, l, b, h) * lo.unit;
    if (is_rows(lo.scheme)) {
        const int64_t width = lo.scheme == KVQ_SCHEME_INT8 ? D : D / 2;
        const uint8_t* row = base + ((int64_t)kv * lo.T16 + t) * width;
        const float s = reinterpret_cast<const float*>(base + 2 * (int64_t)lo.T16 * width)[(int64_t)kv * lo.T16 + t];
        const int code = lo.scheme == KVQ_SCHEME_INT8 ? static_cast<int8_t>(row[c])
                                                      : static_cast<int8_t>(row[c >> 1] << (c & 1 ? 0 : 4)) >> 4;
        return __fmul_rn(static_cast<float>(code), s);
    }
    const float s = reinterpret_cast<const float*>(cache + lo.scales_off)[((int64_t)l * lo.H + h) * 2 + kv];
    const int r = c & 15, tt = static_cast<int>(t & 15);
    const uint8_t code =
        kv ? base[(int64_t)lo.T16 * D + (t - tt) * D + c * 16 + 4 * ((tt & 7) >> 1) + 2 * (tt & 1) + (tt >> 3)]
           : base[t * D + ((r & 7) >> 1) * (D / 4) + 4 * (c >> 4) + 2 * (r >> 3) + (r & 1)];
    const __half_raw x = __nv_cvt_fp8_to_halfraw(code, lo.scheme == KVQ_SCHEME_FP8_E4M3 ? __NV_E4M3 : __NV_E5M2);
    return __fmul_rn(__half2float(__half(x)), s);
}

}  // namespace kvq
