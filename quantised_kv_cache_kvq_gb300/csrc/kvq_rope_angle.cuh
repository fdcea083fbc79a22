// kvq_rope_angle.cuh -- cosine and sine of a rotary angle, as the kernels over pre-RoPE
// caches take them.
#pragma once

namespace kvq {

// cos and sin of a binary32 angle a.  For |a| < 2^17, Cody and Waite's reduction by 2 pi
// in three binary32 parts (the first, 6.28125, has 8 significant bits, so k * C1 is exact
// for the |k| < 2^15 that occur; C2 and C3 carry the rest of 2 pi), then the hardware sine
// and cosine on the reduced |r| <= pi (absolute error about 1e-6).  Larger angles take the
// library's sincosf with its full argument reduction.
__device__ __forceinline__ void rope_sincos(float a, float* sn, float* cs) {
    if (fabsf(a) < 131072.0f) {
        constexpr float kInv2Pi = 0.159154943091895336f;
        constexpr float C1 = 6.28125f, C2 = 1.9353072e-3f, C3 = 1.0253132e-11f;
        const float k = rintf(a * kInv2Pi);
        float r = fmaf(-k, C1, a);
        r = fmaf(-k, C2, r);
        r = fmaf(-k, C3, r);
        __sincosf(r, sn, cs);
    } else {
        sincosf(a, sn, cs);
    }
}

}  // namespace kvq
