// gla_exp.cuh — an exponential for gates that multiply a state again and again.
#pragma once

namespace gla {

// exp(l) for l <= 0, within 2 roundings of 2^-24 and with no lean to either side: a state of long
// memory is multiplied by hundreds of factors near 1, where the hardware's 2^x, low by a third
// of a rounding on average, takes fp32 states from 5e-7 to 3e-6 off.
// l = n ln 2 + r by Cody and Waite's two-part reduction (ln 2 = 355/512 + the rest), e^r =
// 1 + r (1 + r q(r)) with q the degree-4 Chebyshev fit of (e^r - 1 - r) / r^2 on |r| <= ln 2 / 2
// (off by 0.18 roundings at most), and 2^n, which is exact and 0 below 2^-126.  Below exp(-1000)
// it is 0, -infinity among them; a NaN stays one.
__device__ __forceinline__ float exp_centred(float l) {
    float x, e;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(l), "f"(-1000.f));
    // adding 3 * 2^22 rounds to a whole number
    const float n = fmaf(x, 1.4426950408889634f, 12582912.f) + -12582912.f;
    const float r = fmaf(n, 2.1219444005469057e-4f, fmaf(n, -0.693359375f, x));
    float q = fmaf(1.3926213141530752e-3f, r, 8.363203145563602e-3f);
    q = fmaf(q, r, 4.1666556149721146e-2f);
    q = fmaf(q, r, 0.16666576266288757f);
    q = fmaf(q, r, 0.5f);
    q = fmaf(fmaf(q, r, 1.f), r, 1.f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(n));
    return q * e;
}

}  // namespace gla
