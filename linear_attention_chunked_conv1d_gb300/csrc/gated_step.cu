// Decode step of a gated recurrent layer: one new token for each of B streams, the causal conv1d +
// SiLU on the carried window (optional) and one step of the gated recurrence, in one launch.
// "glm5next_kda/prefill.rs", decode_k: the layer applied to one token per stream on the states that
// a prefill leaves. The conv output stays in 32 bits on its way to the recurrence (it is not stored).
//
// HBM-bound: every state element is read and written once. One thread has 4 channels of one stream;
// all its loads are issued before the first is used. On the device, bf16 with K = 4: one stream of 2048
// channels 1.4 us (a launch and one trip to memory), 256 x 4096 4.3 us (30 MB, partly in L2). A thread's taps
// lie next to each other and come in K loads of 8 bytes: with one load a tap it was 6.8 us.
#include "gated.cuh"
#include "launch.h"
#include "overlap.cuh"

namespace la {

namespace {

constexpr int kThreads = 64;  // x 4 channels: a single stream of 2048 channels spreads over 8 SMs

template <typename T, int K>  // K = 0: no conv, x enters the recurrence as it is
__global__ void __launch_bounds__(kThreads) gated_step_kernel(const GatedStepArgs a) {
    using V = Vec4<T>;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 4;
    wait_for_previous();
    if (c >= a.channels) return;
    for (int s = blockIdx.y; s < a.B; s += gridDim.y) {
        float *h = reinterpret_cast<float *>(a.h_ptrs[s]) + c;
        float x[4], ga[4], gb[4], hv[4];
        Vec4<float>::load(h, hv);
        V::load((const T *)a.x + s * a.x_stride + c, x);
        V::load((const T *)a.ab + s * a.ab_stride + c, ga);
        V::load((const T *)a.ab + s * a.ab_stride + a.channels + c, gb);
        if constexpr (K > 0) {
            float win[K][4], w[4 * K], p[4] = {0.f, 0.f, 0.f, 0.f};  // w: four channels' taps, as they lie
            T *st = K > 1 ? reinterpret_cast<T *>(a.conv_state_ptrs[s]) + c : nullptr;
#pragma unroll
            for (int m = 0; m < K - 1; ++m) V::load(st + (int64_t)m * a.channels, win[m]);
#pragma unroll
            for (int j = 0; j < K; ++j) V::load((const T *)a.conv_w + (int64_t)c * K + 4 * j, w + 4 * j);
#pragma unroll
            for (int e = 0; e < 4; ++e) win[K - 1][e] = x[e];
            if (a.conv_bias) V::load((const T *)a.conv_bias + c, p);
#pragma unroll
            for (int m = 0; m < K - 1; ++m) V::store(st + (int64_t)m * a.channels, win[m + 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int j = 0; j < K; ++j) p[e] = fmaf(w[e * K + j], win[j][e], p[e]);
                x[e] = silu(p[e]);
            }
        }
        F4 neg;
        const F4 side = decay4<false>(pack4(ga), neg);
        unpack4(fma4(input4(pack4(gb)), pack4(x), left4(side, neg, pack4(hv))), hv);
        Vec4<float>::store(h, hv);
        V::store((T *)a.y + s * a.y_stride + c, hv);
    }
}

template <typename T>
cudaError_t launch_t(const GatedStepArgs &a, cudaStream_t st) {
    const dim3 grid((a.channels / 4 + kThreads - 1) / kThreads, a.B < 65535 ? a.B : 65535);
    switch (a.conv_kernel) {
        case 0: return launch_overlapped(gated_step_kernel<T, 0>, grid, dim3(kThreads), 0, 0, st, a);
        case 1: return launch_overlapped(gated_step_kernel<T, 1>, grid, dim3(kThreads), 0, 0, st, a);
        case 2: return launch_overlapped(gated_step_kernel<T, 2>, grid, dim3(kThreads), 0, 0, st, a);
        case 3: return launch_overlapped(gated_step_kernel<T, 3>, grid, dim3(kThreads), 0, 0, st, a);
        case 4: return launch_overlapped(gated_step_kernel<T, 4>, grid, dim3(kThreads), 0, 0, st, a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_gated_step(const GatedStepArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace la
