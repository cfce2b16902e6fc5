// Gate arithmetic shared by the gated recurrence kernels (scan, its backward pass, decode step).
#pragma once
#include "common.cuh"

namespace la {

// d = sigmoid(a) and beta = sigmoid(b). The decay exp(-softplus(a)) is 1 - d; the kernels carry d,
// which is exact to a few units in its last place however small it is, and never the rounded 1 - d:
// h - d h keeps the time constant of a channel that remembers thousands of tokens, where a decay
// rounded to 24 bits would be off by up to 2^-25 at every token, the same way each time.
// One reciprocal serves both gates (the special function unit is the scarce one here):
// 1/p = q/(p q). Past the range of p q (|a| or |b| beyond 43), and for NaN, each has its own, so
// infinite gates give exactly 0 or 1 and a NaN in one gate stays out of the other.
__device__ __forceinline__ void gates(float a, float b, float &d, float &beta) {
    const float p = __fadd_rn(1.f, ex2_approx(__fmul_rn(a, -kLog2e)));
    const float q = __fadd_rn(1.f, ex2_approx(__fmul_rn(b, -kLog2e)));
    const float pq = __fmul_rn(p, q);
    if (pq < 0x1p126f) {
        const float r = rcp_approx(pq);
        d = __fmul_rn(r, q);
        beta = __fmul_rn(r, p);
    } else {
        d = rcp_approx(p);
        beta = rcp_approx(q);
    }
}

// h <- (1 - d) h + u: what the token leaves of the state first, rounded once, so that a gate near 1
// forgets a large state without its rounding errors staying behind.
__device__ __forceinline__ float gated_update(float h, float d, float u) {
    return __fadd_rn(fmaf(-d, h, h), u);
}

}  // namespace la
