// Activations of the dense layers' calls (la_linear, la_gated_ffn) and their derivatives, in fp32.
#pragma once
#include <cstring>
#include <type_traits>

#include "common.cuh"

namespace la {

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ uint64_t both(float x) { return pk2(x, x); }
// f of each of a pair
template <class F>
__device__ __forceinline__ uint64_t each(uint64_t v, F &&f) {
    float a, b;
    upk2(v, a, b);
    return pk2(f(a), f(b));
}
// 1 / (1 + e^-y): 0 or 1 for large |y|, without overflow on the way.
__device__ __forceinline__ uint64_t logistic2(uint64_t y) {
    const uint64_t e = each(mul2(y, both(-kLog2e)), [](float t) { return ex2_approx(t); });
    return each(add2(e, both(1.f)), [](float t) { return rcp_approx(t); });
}
// Phi(z), the normal distribution function, and e = exp(-z^2 / 2). For z < 0 it is erfc(x) / 2 with x = |z| / sqrt 2 and
// erfc(x) = e^(-x^2) t Q(t), t = 1 / (1 + 0.375 x), Q a polynomial of degree 6 fitted by a linear program to the least
// relative error at 400 Chebyshev points of 0 <= x <= 10. Its largest relative error over that range is 6.8e-7 (6.2e-7 at
// the points themselves), 1.1e-6 with t and Q in fp32. So the left tail keeps its relative accuracy: within 8e-6 to
// z = -12, most of it from rounding z^2. (8192 x 8192 outputs of 2048 summed indexes with
// bias, GELU and residual: 228 us with erfcf, 210 with this, value by value; 169 with a thread's values side by side.)
__device__ __forceinline__ uint64_t normal2(uint64_t z, uint64_t &e) {
    e = each(mul2(mul2(z, both(-0.5f * kLog2e)), z), [](float t) { return ex2_approx(t); });
    const uint64_t mag = each(z, [](float t) { return fabsf(t); });
    const uint64_t t = each(fma2(mag, both(0.375f * 0.7071067811865476f), both(1.f)), [](float v) { return rcp_approx(v); });
    uint64_t q = both(0.5f * -0.13514285171836257f);
    q = fma2(q, t, both(0.5f * 0.38810317057788546f));
    q = fma2(q, t, both(0.5f * -0.12983093239649302f));
    q = fma2(q, t, both(0.5f * 0.28323088875818103f));
    q = fma2(q, t, both(0.5f * 0.16659836329077654f));
    q = fma2(q, t, both(0.5f * 0.2157023216277419f));
    q = fma2(q, t, both(0.5f * 0.21133842107472253f));
    q = mul2(mul2(q, t), e);
    float z0, z1, q0, q1;
    upk2(z, z0, z1);
    upk2(q, q0, q1);
    return pk2(z0 < 0.f ? q0 : 1.f - q0, z1 < 0.f ? q1 : 1.f - q1);
}

// act(z), and act'(z), of a pair. GELU's tanh form is z logistic(2 c (z + a z^3)). Where a factor of z meets one that has
// vanished, z is cut off first: 0 times infinity would be NaN.
template <int ACT>
__device__ __forceinline__ uint64_t act_pair(uint64_t z, uint64_t &slope) {
    uint64_t s, e;
    const uint64_t c = each(z, [](float v) { return fminf(fmaxf(v, -200.f), 200.f); });
    if constexpr (ACT == LA_ACT_RELU) {
        slope = each(z, [](float v) { return v <= 0.f ? 0.f : 1.f; });
        return each(z, [](float v) { return v < 0.f ? 0.f : v; });  // NaN stays
    } else if constexpr (ACT == LA_ACT_GELU) {
        s = normal2(z, e);
        slope = fma2(mul2(c, both(kInvSqrt2Pi)), e, s);
        return mul2(z, s);
    } else if constexpr (ACT == LA_ACT_GELU_TANH) {
        s = logistic2(mul2(mul2(z, both(2.f * kGeluC)), fma2(mul2(z, both(kGeluA)), z, both(1.f))));
        const uint64_t rest = fma2(s, both(-1.f), both(1.f));
        slope = fma2(mul2(c, mul2(s, rest)), fma2(mul2(c, both(6.f * kGeluC * kGeluA)), c, both(2.f * kGeluC)), s);
        return mul2(z, s);
    } else if constexpr (ACT == LA_ACT_SILU) {
        s = logistic2(z);
        slope = mul2(s, fma2(c, fma2(s, both(-1.f), both(1.f)), both(1.f)));
        return mul2(z, s);
    } else {
        slope = both(1.f);
        return z;
    }
}
// f(integral_constant<int, act>): one branch around the values of a thread, so that their chains run side by side.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case LA_ACT_RELU: f(std::integral_constant<int, LA_ACT_RELU>{}); break;
        case LA_ACT_GELU: f(std::integral_constant<int, LA_ACT_GELU>{}); break;
        case LA_ACT_GELU_TANH: f(std::integral_constant<int, LA_ACT_GELU_TANH>{}); break;
        case LA_ACT_SILU: f(std::integral_constant<int, LA_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, LA_ACT_NONE>{}); break;
    }
}
template <int N>
__device__ __forceinline__ void act_values(float (&v)[N], int act) {
    if (act == LA_ACT_NONE) return;
    with_act(act, [&](auto which) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            uint64_t slope;
            upk2(act_pair<which>(pk2(v[i], v[i + 1]), slope), v[i], v[i + 1]);
        }
    });
}
// value and slope of N values
template <int N>
__device__ __forceinline__ void act_slopes(float (&v)[N], float (&slope)[N], int act) {
    with_act(act, [&](auto which) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            uint64_t s;
            upk2(act_pair<which>(pk2(v[i], v[i + 1]), s), v[i], v[i + 1]);
            upk2(s, slope[i], slope[i + 1]);
        }
    });
}

template <class T> constexpr int kPiece = Vec16<T>::N;  // values of 16 bytes

// 16 bytes of a row from column c on, what lies at or past `width` as zero bytes; and its values in fp32.
template <class T>
__device__ __forceinline__ uint4 load_raw(const T *row, int c, int width) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (c + kPiece<T> <= width) {
        v = *reinterpret_cast<const uint4 *>(row + c);
    } else if (c < width) {
        T e[kPiece<T>];
#pragma unroll
        for (int i = 0; i < kPiece<T>; ++i) e[i] = c + i < width ? row[c + i] : from_f<T>(0.f);
        memcpy(&v, e, 16);
    }
    return v;
}
// Values kept between forward and backward pass in 24 bits: fp32 without its last eight fraction bits, the upper 16
// bits in one plane and the next eight in another. (Relative error below 2^-15, and no rounding that could carry a NaN's
// pattern over.)
__device__ __forceinline__ uint32_t upper2(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }
__device__ __forceinline__ uint32_t lower4(float a, float b, float c, float d) {
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x51), __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x51), 0x5410);
}
__device__ __forceinline__ uint4 upper8(const float *v) {
    return make_uint4(upper2(v[0], v[1]), upper2(v[2], v[3]), upper2(v[4], v[5]), upper2(v[6], v[7]));
}
__device__ __forceinline__ uint2 lower8(const float *v) { return make_uint2(lower4(v[0], v[1], v[2], v[3]), lower4(v[4], v[5], v[6], v[7])); }
__device__ __forceinline__ void joined8(const uint4 &upper, const uint2 &lower, float (&v)[8]) {
    const uint32_t u[4] = {upper.x, upper.y, upper.z, upper.w}, l[2] = {lower.x, lower.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float((i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16) | (l[i / 4] >> i % 4 * 8 & 0xFFu) << 8);
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
