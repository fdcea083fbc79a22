// kvq_elements.cuh -- places of single elements in a group record (layout in kvq_internal.cuh).
#pragma once

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

}  // namespace kvq
