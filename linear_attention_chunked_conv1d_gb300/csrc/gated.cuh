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
// token, the same way each time.
// One reciprocal serves both gates (the special function unit is the scarce one: 3 instead of 4
// operations a gate pair): with p = -(1 + e^-a), q = 1 + e^-b, r = 1 / (p q): -d = r q, beta = r p.
// That holds while p q is in range (|a| and |b| together below 87); `lowest` gathers the least p q,
// for gates_in_range to tell. kExact: a reciprocal for each gate, right for every value: infinite
// gates give exactly 0 or 1.
template <bool kExact>
__device__ __forceinline__ void gates4(const F4 &a, const F4 &b, F4 &nd, F4 &beta, float &lowest) {
    const F4 l = all4(-kLog2e), one = all4(1.f), minus = all4(-1.f);
    float ea[4], eb[4];
    unpack4(mul4(a, l), ea);
    unpack4(mul4(b, l), eb);
#pragma unroll
    for (int e = 0; e < 4; ++e) ea[e] = ex2_approx(ea[e]), eb[e] = ex2_approx(eb[e]);
    const F4 p = fma4(pack4(ea), minus, minus), q = add4(pack4(eb), one);
    float r[4];
    if (kExact) {
        float s[4];
        unpack4(p, r);
        unpack4(q, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = rcp_approx(r[e]), s[e] = rcp_approx(s[e]);
        nd = pack4(r);
        beta = pack4(s);
    } else {
        unpack4(mul4(p, q), r);
        lowest = fminf(lowest, fminf(fminf(r[0], r[1]), fminf(r[2], r[3])));
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = rcp_approx(r[e]);
        nd = mul4(pack4(r), q);
        beta = mul4(pack4(r), p);
    }
}
__device__ __forceinline__ bool gates_in_range(float lowest) { return lowest > -0x1p126f; }

// (1 - d) h, rounded once, so that a gate near 1 forgets a large state without its rounding errors
// staying behind.
__device__ __forceinline__ F4 left4(const F4 &nd, const F4 &h) { return fma4(nd, h, h); }

}  // namespace la
