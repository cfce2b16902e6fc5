// Gated linear recurrence with one state per channel, over packed streams, and its backward pass:
//   d_t = sigmoid(a_t), beta_t = sigmoid(b_t), h_t = (1 - d_t) h_{t-1} + beta_t x_t, y_t = h_t.
// 1 - d = exp(-softplus(a)) and beta are the gates of la_gate_activations ("split_prefill.rs",
// prefill_phase1_proj_batched) on the same rows a | b; the recurrence is the per-channel counterpart
// of the KDA state update ("glm5next_kda/prefill.rs"), without its key and value dimensions.
//
// Backward: with m the gradient of the state that a token finds (for the last token's successor: the
// gradient of the stream's final state),
//   lam_t = dy_t + m_{t+1},  m_t = (1 - d_t) lam_t,  dh_0 = m at the stream's first token,
//   dx = lam beta,  db = lam x beta (1 - beta),  da = -lam h_{t-1} d (1 - d).
// h_{t-1} is computed again from the states that the forward pass saved every kTile tokens.
#include "gated.cuh"
#include "launch.h"

namespace la {

namespace {

constexpr int kTile = 64;       // tokens between two saved states (at packed positions 0, 64, ...)
constexpr int kThreads = 128;   // channels per block

struct Ctl {
    int bad;  // an offset of cu_seqlens is out of order: no stream runs
};

__global__ void scan_init_kernel(const int32_t *cu, int B, int total, Ctl *ctl, int *status) {
    int bad = 0;
    if (threadIdx.x == 0) bad = cu[0] != 0 || cu[B] != total;
    for (int s = threadIdx.x; s < B; s += blockDim.x) bad |= cu[s + 1] < cu[s];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        ctl->bad = bad;
        if (bad) raise_status(status, LA_DEV_BAD_SEQLENS);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) scan_kernel(const GatedScanArgs a, const Ctl *ctl) {
    const int c = blockIdx.x * kThreads + threadIdx.x, s = blockIdx.y;
    if (c >= a.channels || (a.cu && ctl->bad)) return;
    const int t0 = a.cu ? a.cu[s] : s * a.T_each, t1 = a.cu ? a.cu[s + 1] : t0 + a.T_each;
    const T *x = (const T *)a.x, *ab = (const T *)a.ab;
    T *y = (T *)a.y;
    float *h0 = a.h_ptrs ? reinterpret_cast<float *>(a.h_ptrs[s]) + c : nullptr;
    float h = h0 ? *h0 : 0.f;
    const int tiles = (a.total + kTile - 1) / kTile;
    if (a.saved) a.saved[((int64_t)tiles + s) * a.channels + c] = h;
    for (int t = t0; t < t1; ++t) {
        if (a.saved && t % kTile == 0) a.saved[(int64_t)(t / kTile) * a.channels + c] = h;
        float d, beta;
        gates(to_f(ab[t * a.ab_stride + c]), to_f(ab[t * a.ab_stride + a.channels + c]), d, beta);
        h = gated_update(h, d, beta * to_f(x[t * a.x_stride + c]));
        y[t * a.y_stride + c] = from_f<T>(h);
    }
    if (h0 && t1 > t0) *h0 = h;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
scan_backward_kernel(const GatedScanBwdArgs a, const Ctl *ctl) {
    const int c = blockIdx.x * kThreads + threadIdx.x, s = blockIdx.y;
    if (c >= a.channels || (a.cu && ctl->bad)) return;
    const int t0 = a.cu ? a.cu[s] : s * a.T_each, t1 = a.cu ? a.cu[s + 1] : t0 + a.T_each;
    const T *x = (const T *)a.x, *ab = (const T *)a.ab, *dy = (const T *)a.dy;
    T *dx = (T *)a.dx, *dab = (T *)a.dab;
    const int tiles = (a.total + kTile - 1) / kTile;
    float m = a.dh_final_ptrs ? reinterpret_cast<const float *>(a.dh_final_ptrs[s])[c] : 0.f;
    float before[kTile];
    for (int end = t1; end > t0;) {
        const int begin = max(t0, (end - 1) / kTile * kTile);
        float h = a.saved[(begin == t0 ? (int64_t)tiles + s : (int64_t)(begin / kTile)) * a.channels + c];
        for (int t = begin; t < end; ++t) {
            before[t - begin] = h;
            float d, beta;
            gates(to_f(ab[t * a.ab_stride + c]), to_f(ab[t * a.ab_stride + a.channels + c]), d, beta);
            h = gated_update(h, d, beta * to_f(x[t * a.x_stride + c]));
        }
        for (int t = end - 1; t >= begin; --t) {
            float d, beta;
            gates(to_f(ab[t * a.ab_stride + c]), to_f(ab[t * a.ab_stride + a.channels + c]), d, beta);
            const float lam = to_f(dy[t * a.dy_stride + c]) + m;
            m = fmaf(-d, lam, lam);
            dx[t * a.dx_stride + c] = from_f<T>(lam * beta);
            dab[t * a.dab_stride + c] = from_f<T>(-lam * before[t - begin] * d * (1.f - d));
            dab[t * a.dab_stride + a.channels + c] =
                from_f<T>(lam * to_f(x[t * a.x_stride + c]) * beta * (1.f - beta));
        }
        end = begin;
    }
    if (a.dh0_ptrs) reinterpret_cast<float *>(a.dh0_ptrs[s])[c] = m;
}

}  // namespace

size_t gated_scan_workspace_bytes(int, int, int, int) { return 16; }
size_t gated_scan_saved_bytes(int B, int total, int channels, int) {
    return (((size_t)total + kTile - 1) / kTile + B) * channels * sizeof(float);
}

cudaError_t launch_gated_scan(const GatedScanArgs &a, cudaStream_t st) {
    Ctl *ctl = (Ctl *)a.workspace;
    if (a.cu) scan_init_kernel<<<1, 1024, 0, st>>>(a.cu, a.B, a.total, ctl, a.status);
    const dim3 grid((a.channels + kThreads - 1) / kThreads, a.B);
    if (a.dtype == LA_BF16) scan_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, ctl);
    else scan_kernel<float><<<grid, kThreads, 0, st>>>(a, ctl);
    return cudaGetLastError();
}

cudaError_t launch_gated_scan_backward(const GatedScanBwdArgs &a, cudaStream_t st) {
    Ctl *ctl = (Ctl *)a.workspace;
    if (a.cu) scan_init_kernel<<<1, 1024, 0, st>>>(a.cu, a.B, a.total, ctl, a.status);
    const dim3 grid((a.channels + kThreads - 1) / kThreads, a.B);
    if (a.dtype == LA_BF16) scan_backward_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, ctl);
    else scan_backward_kernel<float><<<grid, kThreads, 0, st>>>(a, ctl);
    return cudaGetLastError();
}

}  // namespace la
