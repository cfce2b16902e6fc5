// Gate arithmetic shared by the gated recurrence kernels (scan, its backward pass, decode step), on
// four channels at a time as two packed pairs.
#pragma once
#include "common.cuh"

namespace la {

// Four fp32 values as two packed pairs.
struct F4 {
    uint64_t p[2];
};
__device__ __forceinline__ F4 all4(float v) { return F4{{pk2(v, v), pk2(v, v)}}; }
__device__ __forceinline__ F4 pack4(const float (&f)[4]) { return F4{{pk2(f[0], f[1]), pk2(f[2], f[3])}}; }
__device__ __forceinline__ void unpack4(const F4 &v, float (&f)[4]) {
    upk2(v.p[0], f[0], f[1]);
    upk2(v.p[1], f[2], f[3]);
}
__device__ __forceinline__ F4 fma4(const F4 &a, const F4 &b, const F4 &c) {
    return F4{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1])}};
}
__device__ __forceinline__ F4 mul4(const F4 &a, const F4 &b) {
    return F4{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1])}};
}
__device__ __forceinline__ F4 add4(const F4 &a, const F4 &b) {
    return F4{{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1])}};
}
__device__ __forceinline__ F4 load_f4(const float *p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    return F4{{v.x, v.y}};
}
__device__ __forceinline__ void store_f4(float *p, const F4 &v) {
    *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v.p[0], v.p[1]);
}
// Four activations as loaded, and to fp32.
template <typename T> __device__ __forceinline__ F4 widen4(const typename Vec4<T>::Raw &r) {
    float f[4];
    Vec4<T>::widen(r, f);
    return pack4(f);
}
template <typename T> __device__ __forceinline__ void store_act4(T *p, const F4 &v) {
    float f[4];
    unpack4(v, f);
    Vec4<T>::store(p, f);
}

// The decay 1 - d = sigmoid(-a) = exp(-softplus(a)) of four channels, by its smaller side. With t = a log2 e,
//   small = 2^-|t| / (1 + 2^-|t|) in 0 .. 1/2,  side = t < 0 ? -small : small,  neg = t < 0 ? 1 : 0,
// the decay neg + side and d = (1 - neg) - side are both right to their own last places: the one is small, the
// other 1 - small, rounded once. (From d = sigmoid(a) alone 1 - d is off by 2^-25: by 0.3% of it at a = 10, by
// all of it at 17.) Relative to small the error is that of the argument's rounding, |a| 2^-23 at most, and 2^-21
// of the hardware exponential and reciprocal and three roundings; below 2^-126 (|a| > 87.3) it is flushed to 0.
// Infinite gates give exactly 0 and 1.
// The rounded decay is what the few tokens of a run go by. Where tokens follow each other without end, a
// channel that remembers thousands of them would be off by up to 2^-25 at every one, the same way each time:
// there h goes on as left4, h - d h (or (1 - d) h), rounded once.
// kMark: a negative side has 2^-149 more, so that neg_of finds it again when small is 0. (Next to 1 it is nothing;
// d is then 2^-149, not 0.)
template <bool kMark> __device__ __forceinline__ F4 decay4(const F4 &a, F4 &neg) {
    const F4 one = all4(1.f);
    float f[4], n[4], e[4];
    unpack4(fma4(a, all4(kLog2e), all4(0.f)), f);  // + 0: -0 counts as 0 below, too
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = ex2_approx(-fabsf(f[i])), n[i] = f[i] < 0.f ? 1.f : 0.f;
    neg = pack4(n);
    const F4 E = pack4(e);
    unpack4(add4(E, one), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = rcp_approx(f[i]);
    const F4 small = mul4(E, pack4(f)), sign = fma4(neg, all4(-2.f), one);
    return kMark ? fma4(small, sign, mul4(neg, all4(-0x1p-149f))) : mul4(small, sign);
}
// neg of a marked side; the decay, -d and what is left of h.
__device__ __forceinline__ F4 neg_of(const F4 &side) {
    float f[4];
    unpack4(side, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f[i] < 0.f ? 1.f : 0.f;
    return pack4(f);
}
__device__ __forceinline__ F4 decay_of(const F4 &side, const F4 &neg) { return add4(neg, side); }
__device__ __forceinline__ F4 minus_d_of(const F4 &side, const F4 &neg) { return add4(add4(neg, all4(-1.f)), side); }
__device__ __forceinline__ F4 left4(const F4 &side, const F4 &neg, const F4 &h) { return fma4(side, h, mul4(neg, h)); }

// The input gate beta = sigmoid(b) = 1 / (1 + q) with q = e^-b, and 1 - beta = q beta: a product, which is right
// relative to itself for either sign of b. q is held to 2^127, where beta is flushed to 0 and the product is 0,
// not NaN: it is only ever a factor next to beta. min.NaN passes a NaN on.
__device__ __forceinline__ F4 input_exp4(const F4 &b) {
    float q[4];
    unpack4(mul4(b, all4(-kLog2e)), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q[e] = ex2_approx(q[e]);
        asm("min.NaN.f32 %0, %0, 0f7f000000;" : "+f"(q[e]));
    }
    return pack4(q);
}
__device__ __forceinline__ F4 input_of(const F4 &q) {
    float f[4];
    unpack4(add4(q, all4(1.f)), f);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = rcp_approx(f[e]);
    return pack4(f);
}
// beta where 1 - beta is not needed.
__device__ __forceinline__ F4 input4(const F4 &b) {
    float q[4];
    unpack4(mul4(b, all4(-kLog2e)), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = ex2_approx(q[e]);
    return input_of(pack4(q));
}

}  // namespace la
