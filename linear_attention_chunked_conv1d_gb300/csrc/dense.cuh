// Activations of the dense layers' calls (la_linear, la_gated_ffn) and their derivatives, in fp32.
#pragma once
#include "common.cuh"

namespace la {

// act(z). Large |z| neither overflows nor turns into NaN: the logistic function is 0 or 1 there.
__device__ __forceinline__ float logistic(float z) { return rcp_approx(1.f + ex2_approx(-kLog2e * z)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// GELU by the normal distribution function, z Phi(z): Phi(z) = erfc(-z / sqrt 2) / 2 keeps the small
// values of the left tail, where 1 + erf would cancel. Its tanh form is z logistic(2 c (z + a z^3)).
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case LA_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
        case LA_ACT_GELU: return 0.5f * z * erfcf(-z * kSqrtHalf);
        case LA_ACT_GELU_TANH: return z * logistic(2.f * kGeluC * z * fmaf(kGeluA * z, z, 1.f));
        case LA_ACT_SILU: return z * logistic(z);
        default: return z;
    }
}

// act'(z). Where a factor of z meets one that has vanished, z is cut off first: 0 times infinity would be NaN.
__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case LA_ACT_RELU: return z <= 0.f ? 0.f : 1.f;
        case LA_ACT_GELU: {
            const float c = fminf(fmaxf(z, -40.f), 40.f);
            return fmaf(c * kInvSqrt2Pi, ex2_approx(-0.5f * kLog2e * c * c), 0.5f * erfcf(-z * kSqrtHalf));
        }
        case LA_ACT_GELU_TANH: {
            const float s = logistic(2.f * kGeluC * z * fmaf(kGeluA * z, z, 1.f)), c = fminf(fmaxf(z, -40.f), 40.f);
            return fmaf(c * s * (1.f - s), 2.f * kGeluC * fmaf(3.f * kGeluA * c, c, 1.f), s);
        }
        case LA_ACT_SILU: {
            const float s = logistic(z), c = fminf(fmaxf(z, -200.f), 200.f);
            return s * fmaf(c, 1.f - s, 1.f);
        }
        default: return 1.f;
    }
}

// N values (16 bytes) of a row from column c on, of which those at or past `width` read as zero; and the
// store of those before it. Rows start on 16 bytes, so only a row's last piece is taken by elements.
template <class T>
__device__ __forceinline__ void load_piece(const T *row, int c, int width, float *f) {
    constexpr int N = Vec16<T>::N;
    if (c + N <= width) {
        Vec16<T>::load(row + c, f);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = c + e < width ? to_f(row[c + e]) : 0.f;
    }
}
template <class T>
__device__ __forceinline__ void store_piece(T *row, int c, int width, const float *f) {
    constexpr int N = Vec16<T>::N;
    if (c + N <= width) {
        Vec16<T>::store(row + c, f);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + e < width) row[c + e] = from_f<T>(f[e]);
    }
}

}  // namespace la
