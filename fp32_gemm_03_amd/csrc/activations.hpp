// activations.hpp -- the gate's activations, their slopes, in 32 and 64 bits.
//
// With s(u) = 1 / (1 + exp(-u)) and c = 2 sqrt(2 / pi):
//   silu       g s(g)              slope s (1 + g (1 - s))
//   gelu       g Phi(g)            slope Phi + g phi(g),  Phi(g) = erfc(-g / sqrt 2) / 2
//   gelu_tanh  g s(u), u = c (g + 0.044715 g^3)   (= g (1 + tanh(u / 2)) / 2)
//                                  slope s + g s (1 - s) c (1 + 0.134145 g^2)
// s and 1 - s both come from exp(-|u|), so neither overflows nor cancels; erfc keeps
// Phi's relative accuracy below 0.  An infinite gate is taken to its limit: 0 at
// -infinity, slopes 0 and 1.
#pragma once

#include <hip/hip_runtime.h>

namespace normk {

constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2;  // SGEMM_ACT_*

template <class F> struct Pair {
    F s, rest;  // s(u), 1 - s(u)
};
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
__device__ __forceinline__ float erfc_of(float x) { return erfcf(x); }
__device__ __forceinline__ double erfc_of(double x) { return erfc(x); }
__device__ __forceinline__ float size_of(float x) { return fabsf(x); }
__device__ __forceinline__ double size_of(double x) { return fabs(x); }

// exp(x), x <= 0, in 64 bits to 2^-45: 2^k times the series of r = x - k ln 2, |r| <=
// 0.3466, up to r^11 (the next term is below 2^-47).  ln 2 is taken off in two parts (Cody and
// Waite): its first 32 bits, whose product with k is exact, and the rest, rounded to 64.  Half
// the instructions of exp(), which with the quotient below set the time of 8-bit rows behind
// SiLU and the tanh form.
__device__ __forceinline__ double exp_below_0(double x) {
    x = x < -800.0 ? -800.0 : x;  // (0 from -745 on; NaN stays)
    const double k = rint(x * 1.4426950408889634);
    const double r = fma(k, -0x1.a39ef35793c76p-33, fma(k, -0x1.62e42feep-1, x));
    double p = 1.0 / 39916800.0;
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)k);
}
// 1 / d, 1 <= d <= 2, to 2^-50: two Newton steps from the hardware's estimate
__device__ __forceinline__ double reciprocal_of(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    return fma(fma(-d, y, 1.0), y, y);
}
__device__ __forceinline__ float exp_below_0(float x) { return expf(x); }
__device__ __forceinline__ float reciprocal_of(float d) { return 1.0f / d; }

template <class F> __device__ __forceinline__ Pair<F> logistic(F u) {
    const F e = exp_below_0(-size_of(u)), high = reciprocal_of(F(1) + e), low = e * high;
    return u < F(0) ? Pair<F>{low, high} : Pair<F>{high, low};
}
// (NaN stays; beyond 20 the tanh form's s is 0 or 1 in 64 bits)
template <class F> __device__ __forceinline__ F within(F g, F most) { return g < -most ? -most : g > most ? most : g; }
template <class F> __device__ __forceinline__ F tanh_argument(F g) {
    const F b = within(g, F(20));
    return F(1.5957691216057308) * (b + F(0.044715) * b * b * b);
}

template <int ACT, class F> __device__ __forceinline__ F act(F g) {
    const F lowest = F(-3.4028234663852886e38);
    g = g < lowest ? lowest : g;
    if (ACT == kSilu) return g * logistic(g).s;
    if (ACT == kGelu) return F(0.5) * g * erfc_of(F(-0.70710678118654752) * g);
    return g * logistic(tanh_argument(g)).s;
}

template <int ACT, class F> __device__ __forceinline__ F act_slope(F g) {
    g = within(g, F(3.4028234663852886e38));
    if (ACT == kSilu) {
        const Pair<F> p = logistic(g);
        return p.s * (F(1) + g * p.rest);
    }
    if (ACT == kGelu)
        return F(0.5) * erfc_of(F(-0.70710678118654752) * g) + g * (F(0.39894228040143268) * exp_of(F(-0.5) * g * g));
    const Pair<F> p = logistic(tanh_argument(g));
    const F b = within(g, F(20));
    return p.s + b * p.s * p.rest * F(1.5957691216057308) * (F(1) + F(0.134145) * b * b);
}

}  // namespace normk
