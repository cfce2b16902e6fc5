// Backward pass of the causal depthwise conv1d + SiLU with a carried window, single stream or packed
// streams ("glm5next_kda/prefill.rs", conv_prefill launch, is the forward pass). With
//   xh = [window (K-1 rows) ; x], p_t = bias + sum_j w_j xh[t + j], out_t = SiLU(p_t):
//   dp_t = dout_t SiLU'(p_t),  SiLU'(p) = s (1 + p (1 - s)), s = sigmoid(p),
//   dx_i = sum_n w_{K-1-n} dp_{i+n} (within the stream; i < 0: rows of the window),
//   dw_j = sum_t dp_t xh[t + j],  dbias = sum_t dp_t;
// a row that the window of the next call holds also takes that window's gradient.
//
// One thread has 4 channels of a run of consecutive tokens of one stream, with the last K rows of xh
// and of dp in registers: x and dout are read once (plus K-1 rows on each side of a run), dx is
// written once. p is computed again, never stored. The sums over tokens are kept per run in 32 bits
// and joined run by run in a fixed order by a second kernel, so they come out the same every time.
#include "common.cuh"
#include "launch.h"

namespace la {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;  // tokens of a run

struct Ctl {
    int bad;  // an offset of cu_seqlens is out of order: nothing is computed
};

__global__ void conv_bwd_init_kernel(const int32_t *cu, int B, int total, Ctl *ctl, int *status) {
    int bad = 0;
    if (threadIdx.x == 0) bad = cu[0] != 0 || cu[B] != total;
    for (int s = threadIdx.x; s < B; s += blockDim.x) bad |= cu[s + 1] < cu[s];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        ctl->bad = bad;
        if (bad) raise_status(status, LA_DEV_BAD_SEQLENS);
    }
}

// First run of stream s: every stream, an empty one too, has at least one.
__device__ __forceinline__ int run_base(const ConvBwdArgs &a, int s) {
    return a.cu ? a.cu[s] / kRows + s : s * ((a.T_each + kRows - 1) / kRows);
}

__host__ __device__ inline int run_slots(int B, int T_each, int total, bool varlen) {
    return varlen ? total / kRows + B : B * ((T_each + kRows - 1) / kRows);
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvBwdArgs a, const Ctl *ctl, float *part) {
    using V = Vec4<T>;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * 4;
    if (c >= a.channels || (a.cu && ctl->bad)) return;
    const int slot = blockIdx.x;
    int s = 0, hi = a.B - 1;
    while (s < hi) {  // last s with run_base(s) <= slot
        const int mid = (s + hi + 1) >> 1;
        if (run_base(a, mid) <= slot) s = mid; else hi = mid - 1;
    }
    const int sb = a.cu ? a.cu[s] : s * a.T_each, se = a.cu ? a.cu[s + 1] : sb + a.T_each;
    const int len = se - sb, run = slot - run_base(a, s);
    const int64_t C = a.channels;
    const int r0 = sb + run * kRows, r1 = min(r0 + kRows, se);

    float w[K][4], bias[4] = {0.f, 0.f, 0.f, 0.f}, dw[K][4] = {}, db[4] = {};
    float win[K][4] = {}, dpw[K][4] = {};  // rows t-K+1 .. t of xh, and dp of the same tokens
    if (r0 < se) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][e] = to_f(((const T *)a.w)[(c + e) * K + j]);
        if (a.bias) V::load((const T *)a.bias + c, bias);
    }
    const T *fin = a.dstate_final_ptrs ? reinterpret_cast<const T *>(a.dstate_final_ptrs[s]) : nullptr;
    T *dst = a.dstate_ptrs ? reinterpret_cast<T *>(a.dstate_ptrs[s]) : nullptr;
    if (len == 0 && dst) {  // the window passes through an empty stream
#pragma unroll
        for (int m = 0; m < K - 1; ++m) {
            float v[4] = {};
            if (fin) V::load(fin + m * C + c, v);
            V::store(dst + m * C + c, v);
        }
    }
    if (r0 < se) {
#pragma unroll
        for (int m = 0; m < K - 1; ++m) {
            if (run == 0) V::load(reinterpret_cast<const T *>(a.state_ptrs[s]) + m * C + c, win[m + 1]);
            else V::load((const T *)a.x + (r0 - (K - 1) + m) * a.x_stride + c, win[m + 1]);
        }
        for (int t = r0; t < r1 + K - 1; ++t) {
            float x[4] = {}, dout[4] = {};
            if (t < se) {
                V::load((const T *)a.x + t * a.x_stride + c, x);
                V::load((const T *)a.dout + t * a.dout_stride + c, dout);
            }
            float g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int j = 0; j < K - 1; ++j) {
                    win[j][e] = win[j + 1][e];
                    dpw[j][e] = dpw[j + 1][e];
                }
                win[K - 1][e] = x[e];
                float p = bias[e];
#pragma unroll
                for (int j = 0; j < K; ++j) p = fmaf(w[j][e], win[j][e], p);
                const float sg = rcp_approx(1.f + ex2_approx(p * -kLog2e));
                const float dp = t < se ? dout[e] * sg * fmaf(p, 1.f - sg, 1.f) : 0.f;
                dpw[K - 1][e] = dp;
                if (t < r1) {
                    db[e] += dp;
#pragma unroll
                    for (int j = 0; j < K; ++j) dw[j][e] = fmaf(dp, win[j][e], dw[j][e]);
                }
                g[e] = 0.f;
#pragma unroll
                for (int n = 0; n < K; ++n) g[e] = fmaf(w[K - 1 - n][e], dpw[n][e], g[e]);
            }
            const int i = t - (K - 1);  // the row whose gradient is complete now
            if (i < r0 && run > 0) continue;
            const int m = i - sb + (K - 1) - len;  // its row in the window that the stream leaves
            if (m >= 0 && fin) {
                float v[4];
                V::load(fin + m * C + c, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] += v[e];
            }
            if (i >= sb) V::store((T *)a.dx + i * a.dx_stride + c, g);
            else if (dst) V::store(dst + (i - sb + K - 1) * C + c, g);
        }
    }
    float *out = part + (int64_t)slot * (K + 1) * C + c;  // runs without tokens add zeros
#pragma unroll
    for (int j = 0; j < K; ++j) Vec4<float>::store(out + j * C, dw[j]);
    Vec4<float>::store(out + K * C, db);
}

// Sum of the runs' parts: one thread per (tap or bias, channel).
__global__ void conv_bwd_sum_kernel(const float *part, int slots, int K, int C, float *dw, float *dbias,
                                    const Ctl *ctl) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (K + 1) * C || (ctl && ctl->bad)) return;
    float v = 0.f;
    for (int s = 0; s < slots; ++s) v += part[(int64_t)s * (K + 1) * C + i];
    const int j = i / C, c = i % C;
    if (j < K) dw[(int64_t)c * K + j] = v;
    else if (dbias) dbias[c] = v;
}

template <typename T, int K>
cudaError_t launch_t(const ConvBwdArgs &a, cudaStream_t st) {
    Ctl *ctl = (Ctl *)a.workspace;
    float *part = (float *)((char *)a.workspace + 16);
    const int slots = run_slots(a.B, a.T_each, a.total, a.cu != nullptr);
    if (a.cu) conv_bwd_init_kernel<<<1, 1024, 0, st>>>(a.cu, a.B, a.total, ctl, a.status);
    const dim3 grid(slots, (a.channels / 4 + kThreads - 1) / kThreads);
    conv_bwd_kernel<T, K><<<grid, kThreads, 0, st>>>(a, ctl, part);
    conv_bwd_sum_kernel<<<((K + 1) * a.channels + 127) / 128, 128, 0, st>>>(
        part, slots, K, a.channels, a.dw, a.dbias, a.cu ? ctl : nullptr);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_k(const ConvBwdArgs &a, cudaStream_t st) {
    switch (a.kernel) {
        case 1: return launch_t<T, 1>(a, st);
        case 2: return launch_t<T, 2>(a, st);
        case 3: return launch_t<T, 3>(a, st);
        case 4: return launch_t<T, 4>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

size_t conv_backward_workspace_bytes(int B, int total, int channels, int kernel, int) {
    // a run of a stream of equal lengths ends with it: no more runs than packed streams have
    return 16 + ((size_t)total / kRows + B) * (kernel + 1) * channels * sizeof(float);
}

cudaError_t launch_conv1d_silu_backward(const ConvBwdArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? launch_k<__nv_bfloat16>(a, st) : launch_k<float>(a, st);
}

}  // namespace la
