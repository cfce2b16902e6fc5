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

// The gates of four channels: nd = -d = -sigmoid(a) and beta = sigmoid(b). The decay
// exp(-softplus(a)) is 1 + nd. The kernels carry d, which is exact to a few units in its last place
// however small it is, and never the rounded 1 - d: h - d h keeps the time constant of a channel that
// remembers thousands of tokens, where a decay rounded to 24 bits would be off by up to 2^-25 at every
// token, the same way each time. Infinite gates give exactly 0 or 1.
// (One reciprocal of the product (1 + e^-a)(1 + e^-b) for both gates saves a special function but
// needs a second way for gates beyond its range, and with it the scan's registers no longer sufficed:
// 1.15 ms instead of 0.69 for 262,144 x 2048, the chains left out.)
__device__ __forceinline__ void gates4(const F4 &a, const F4 &b, F4 &nd, F4 &beta) {
    const F4 l = all4(-kLog2e), one = all4(1.f), minus = all4(-1.f);
    float p[4], q[4];
    unpack4(mul4(a, l), p);
    unpack4(mul4(b, l), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(p[e]), q[e] = ex2_approx(q[e]);
    unpack4(fma4(pack4(p), minus, minus), p);
    unpack4(add4(pack4(q), one), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = rcp_approx(p[e]), q[e] = rcp_approx(q[e]);
    nd = pack4(p);
    beta = pack4(q);
}

// (1 - d) h, rounded once, so that a gate near 1 forgets a large state without its rounding errors
// staying behind.
__device__ __forceinline__ F4 left4(const F4 &nd, const F4 &h) { return fma4(nd, h, h); }

}  // namespace la
