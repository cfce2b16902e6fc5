// Products of a few rows with 4-bit weights that have a scale for each group of inputs:
//   y[m][n] = sum_k x[m][k] W[n][k],  W[n][k] = scales[n][k / group] (q(n, k) - 8),  q in 0..15.
// The projections of "split_prefill.rs", prefill_phase1_proj_batched, when a layer decodes a few
// tokens: reading the weights is all the time there is, and these take a quarter of bf16's.
//
// Layout of q [N][K / 2] bytes: eight weights of a row to a little-endian 32-bit word, weight 2i in
// bits 4i .. 4i+3 and weight 2i + 1 in bits 16+4i .. 16+4i+3, so that one shift and one mask give a
// pair (2i, 2i + 1) in the two halves of a word.
#include "common.cuh"
#include "launch.h"

namespace la {

namespace {

// Eight weights of one thread: the group's largest magnitude over its lanes, the scale max / 7
// rounded to bf16, and the nearest multiples of that scale (ties to even).
__global__ void w4_quantize_kernel(const W4QuantArgs a, int64_t words) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int per_row = a.K / 8, lanes = a.group / 8;  // 4, 8 or 16 lanes have one group
    const bool active = i < words;                     // whole groups: words is a multiple of lanes
    const int64_t n = active ? i / per_row : 0;
    const int k8 = active ? (int)(i % per_row) : 0;
    float v[8] = {};
    if (active) Vec16<__nv_bfloat16>::load((const __nv_bfloat16 *)a.w + n * a.ldw + k8 * 8, v);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
    for (int off = lanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(top, 7.f));
    const float sc = to_f(scale);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int q = sc > 0.f ? __float2int_rn(fminf(fmaxf(__fdiv_rn(v[e], sc), -8.f), 7.f)) : 0;
        word |= (uint32_t)(q + 8) << (4 * (e / 2) + 16 * (e % 2));
    }
    if (!active) return;
    ((uint32_t *)a.q)[i] = word;
    if (k8 % lanes == 0) ((__nv_bfloat16 *)a.scales)[n * (a.K / a.group) + k8 / lanes] = scale;
}

// One warp per output, up to 8 rows at a time; a lane has eight weights of every 256.
__global__ void __launch_bounds__(128) w4_matvec_kernel(const W4Args a) {
    const int n = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (n >= a.N) return;
    const uint32_t *q = (const uint32_t *)a.q + (int64_t)n * (a.K / 8);
    const __nv_bfloat16 *sc = (const __nv_bfloat16 *)a.scales + (int64_t)n * (a.K / a.group);
    const __nv_bfloat16 *x = (const __nv_bfloat16 *)a.x;
    for (int m0 = 0; m0 < a.M; m0 += 8) {
        float acc[8] = {};
        for (int k8 = lane; k8 < a.K / 8; k8 += 32) {
            const uint32_t word = q[k8];
            const float s = to_f(sc[k8 * 8 / a.group]);
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = s * (float)((int)(word >> (4 * (e / 2) + 16 * (e % 2)) & 15u) - 8);
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (m0 + m < a.M) {
                    float v[8];
                    Vec16<__nv_bfloat16>::load(x + (m0 + m) * a.ldx + k8 * 8, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[m] = fmaf(w[e], v[e], acc[m]);
                }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            for (int off = 16; off > 0; off >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], off);
            if (lane == 0 && m0 + m < a.M)
                ((__nv_bfloat16 *)a.y)[(m0 + m) * a.ldy + n] = __float2bfloat16_rn(acc[m]);
        }
    }
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Args &a, cudaStream_t st) {
    w4_matvec_kernel<<<(a.N + 3) / 4, 128, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_w4_quantize(const W4QuantArgs &a, cudaStream_t st) {
    const int64_t words = (int64_t)a.N * (a.K / 8);
    w4_quantize_kernel<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(a, words);
    return cudaGetLastError();
}

}  // namespace la
