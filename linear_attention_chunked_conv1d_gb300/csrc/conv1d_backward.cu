// Backward pass of the causal depthwise conv1d + SiLU with a carried window, single stream or packed
// streams ("glm5next_kda/prefill.rs", conv_prefill launch, is the forward pass). With
//   xh = [window (K-1 rows) ; x], p_t = bias + sum_j w_j xh[t + j], out_t = SiLU(p_t):
//   dp_t = dout_t SiLU'(p_t),  SiLU'(p) = s (1 + p (1 - s)), s = sigmoid(p),
//   dx_i = sum_n w_{K-1-n} dp_{i+n} (within the stream; i < 0: rows of the window),
//   dw_j = sum_t dp_t xh[t + j],  dbias = sum_t dp_t;
// a row that the window of the next call holds also takes that window's gradient.
//
// HBM-bound: x and dout are read once (plus K-1 rows on each side of a run), dx is written once; p is
// computed again, never stored. One thread has 4 channels, in packed pairs, of a run of consecutive
// tokens of one stream, with the last K rows of xh and of dp in registers. Rows come through a ring in
// shared memory, each thread's its own (no barriers), two groups of rows ahead of the one at work: with
// one group in registers instead, a third of the time went into waiting for it. The sums over tokens are
// kept per run in 32 bits and joined run by run in a fixed order by a second kernel, so they come out the
// same every time. 100003 x 8192 bf16 in 32 streams, K = 4: 0.86 ms, 5.7 TB/s of what has to move.
#include "gated.cuh"
#include "launch.h"
#include "overlap.cuh"

namespace la {

namespace {

constexpr int kThreads = 128;
// Rows of a group, and groups of the ring: 48 KB a block, four blocks on an SM.
template <typename T> constexpr int kGroupOf = 16 / sizeof(T);
constexpr int kRing = 3;
template <typename T> constexpr int kRingBytes = kRing * kGroupOf<T> * 2 * kThreads * 4 * (int)sizeof(T);

// Four activations to shared memory, or zeros.
template <typename T> __device__ __forceinline__ void copy_row(void *to, const T *from, bool there) {
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    const int bytes = there ? 4 * (int)sizeof(T) : 0;
    if constexpr (sizeof(T) == 2)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
}

// Tokens of a run: long ones read and write less for what runs share (K-1 rows at each end, the sums),
// short ones make more blocks. The longest that still makes 1000 blocks (152 SMs have 608 at a time; a
// fixed number of SMs, so that sums do not depend on the device). K = 4, runs of 384, 256, 192, 128, 96 and
// 64 (*: taken), us:
//   16384 x 6144, 8 streams, bf16    136  137 *127  133  136  143
//   16384 x 4096, 8 streams, bf16    105   96  103  *92   98  102
//   65536 x 2048, 32 streams, bf16   192 *176  177  183  190  208
//   100003 x 8192, 32 streams, bf16 *861  869  890  914  949 1030
//   8192 x 8192, 4 streams, bf16     104   95  101  *89   95   97
//   32768 x 1024, 16 streams, bf16    77   58   61   59   64  *69
//   16384 x 4096, 4 streams, fp32    151  151  144 *135  140  141
//   40001 x 2000, 33 streams, fp32   203  179  175 *177  178  187
// The best or within 2% of it, but for the few channels of 32768 x 1024, where longer runs are 20% better.
__host__ __device__ inline int run_rows(int B, int total, int channels) {
    const int64_t cols = (channels / 4 + kThreads - 1) / kThreads;
    const auto blocks = [&](int rows) { return (total / rows + B) * cols; };
    return blocks(384) >= 1000 ? 384 : blocks(256) >= 1000 ? 256 : blocks(192) >= 1000 ? 192 : blocks(128) >= 1000 ? 128
           : blocks(96) >= 1000 ? 96 : 64;
}

struct Runs {
    const int32_t *cu;  // or nullptr: B streams of T_each tokens
    int B, T_each, total, rows;
    __device__ __forceinline__ int start(int s) const { return cu ? cu[s] : s * T_each; }
    // First run of stream s: every stream, an empty one too, has at least one.
    __device__ __forceinline__ int base(int s) const { return cu ? cu[s] / rows + s : s * ((T_each + rows - 1) / rows); }
    __host__ __device__ int slots() const { return cu ? total / rows + B : B * ((T_each + rows - 1) / rows); }
    // Every thread of the block looks at its share of the offsets.
    __device__ bool bad() const {
        int b = 0;
        if (cu) {
            if (threadIdx.x == 0) b = cu[0] != 0 || cu[B] != total;
            for (int s = threadIdx.x; s < B; s += blockDim.x) b |= cu[s + 1] < cu[s];
        }
        return __syncthreads_or(b);
    }
};

template <typename T, int K>
__global__ void __launch_bounds__(kThreads, 4) conv_bwd_kernel(const ConvBwdArgs a, const Runs runs, float *part) {
    using V = Vec4<T>;
    constexpr int kGroup = kGroupOf<T>;
    extern __shared__ __align__(16) unsigned char smem[];
    auto *ring = reinterpret_cast<typename V::Raw (*)[kGroup][2][kThreads]>(smem);  // [kRing]
    wait_for_previous();
    if (runs.bad()) {
        if (threadIdx.x == 0) raise_status(a.status, LA_DEV_BAD_SEQLENS);
        return;
    }
    const int c = (blockIdx.y * kThreads + threadIdx.x) * 4;
    if (c >= a.channels) return;
    const int slot = blockIdx.x;
    int s = 0, hi = a.B - 1;
    while (s < hi) {  // last s with base(s) <= slot
        const int mid = (s + hi + 1) >> 1;
        if (runs.base(mid) <= slot) s = mid; else hi = mid - 1;
    }
    const int sb = runs.start(s), se = runs.start(s + 1), len = se - sb, run = slot - runs.base(s);
    const int64_t C = a.channels;
    const int r0 = sb + run * runs.rows, r1 = min(r0 + runs.rows, se);
    const T *fin = a.dstate_final_ptrs ? reinterpret_cast<const T *>(a.dstate_final_ptrs[s]) + c : nullptr;
    T *dst = a.dstate_ptrs ? reinterpret_cast<T *>(a.dstate_ptrs[s]) + c : nullptr;

    F4 dw[K], db = all4(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j] = all4(0.f);
    if (len == 0 && dst) {  // the window passes through an empty stream
#pragma unroll
        for (int m = 0; m < K - 1; ++m)
            store_act4<T>(dst + m * C, fin ? widen4<T>(V::load_raw(fin + m * C)) : all4(0.f));
    }
    if (r0 < se) {
        F4 w[K], bias = all4(0.f), win[K], dpw[K];  // win, dpw: rows t-K+1 .. t of xh and of dp
        {
            float f[K][4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < K; ++j) f[j][e] = to_f(((const T *)a.w)[(c + e) * K + j]);
#pragma unroll
            for (int j = 0; j < K; ++j) w[j] = pack4(f[j]), win[j] = dpw[j] = all4(0.f);
            if (a.bias) bias = widen4<T>(V::load_raw((const T *)a.bias + c));
        }
#pragma unroll
        for (int m = 0; m < K - 1; ++m)
            win[m + 1] = widen4<T>(V::load_raw(run == 0 ? reinterpret_cast<const T *>(a.state_ptrs[s]) + m * C + c
                                                        : (const T *)a.x + (r0 - (K - 1) + m) * a.x_stride + c));
        const F4 one = all4(1.f), minus = all4(-1.f), l2e = all4(-kLog2e);

        // Token t: its dp, its part of the sums, and the gradient of row t - (K-1), complete now.
        const auto token = [&](const F4 &x, const F4 &dout) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = win[j + 1], dpw[j] = dpw[j + 1];
            win[K - 1] = x;
            F4 p = bias;
#pragma unroll
            for (int j = 0; j < K; ++j) p = fma4(w[j], win[j], p);
            float f[4];
            unpack4(mul4(p, l2e), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = ex2_approx(f[e]);
            unpack4(add4(pack4(f), one), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = rcp_approx(f[e]);
            const F4 sg = pack4(f);
            dpw[K - 1] = mul4(mul4(dout, sg), fma4(p, fma4(sg, minus, one), one));
        };
        const auto add = [&](const F4 &dp) {
            db = add4(db, dp);
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j] = fma4(dp, win[j], dw[j]);
        };
        const auto row = [&]() {
            F4 g = mul4(w[K - 1], dpw[0]);
#pragma unroll
            for (int n = 1; n < K; ++n) g = fma4(w[K - 1 - n], dpw[n], g);
            return g;
        };

        const int last = min(r1 + K - 1, se);  // tokens that the run's rows depend on
        const int groups = (r1 + K - 1 - r0 + kGroup - 1) / kGroup;
        const T *x0 = (const T *)a.x + r0 * a.x_stride + c, *d0 = (const T *)a.dout + r0 * a.dout_stride + c;
        const auto fetch = [&](int g) {  // group g into the ring
            if (g < groups) {
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    const int n = g * kGroup + q;
                    const bool there = r0 + n < last;
                    copy_row(&ring[g % kRing][q][0][threadIdx.x], there ? x0 + n * a.x_stride : x0, there);
                    copy_row(&ring[g % kRing][q][1][threadIdx.x], there ? d0 + n * a.dout_stride : d0, there);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch(0);
        fetch(1);
        T *dxp = (T *)a.dx + (r0 - (K - 1)) * a.dx_stride + c;
        for (int g = 0; g < groups; ++g) {
            fetch(g + 2);
            asm volatile("cp.async.wait_group 2;" ::: "memory");
            const int t0 = r0 + g * kGroup;
            const auto &rows = ring[g % kRing];
            if (t0 >= r0 + K - 1 && t0 + kGroup <= r1) {  // every row of these is the run's own
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    token(widen4<T>(rows[q][0][threadIdx.x]), widen4<T>(rows[q][1][threadIdx.x]));
                    add(dpw[K - 1]);
                    store_act4<T>(dxp + q * a.dx_stride, row());
                }
            } else {
#pragma unroll
                for (int q = 0; q < kGroup; ++q) {
                    const int t = t0 + q, i = t - (K - 1);
                    token(widen4<T>(rows[q][0][threadIdx.x]), widen4<T>(rows[q][1][threadIdx.x]));
                    if (t >= last) dpw[K - 1] = all4(0.f);  // no such token (its dout is 0, its p need not be finite)
                    if (t < r1) add(dpw[K - 1]);
                    if ((i < r0 && run > 0) || i >= r1) continue;
                    F4 grad = row();
                    const int m = i - sb + (K - 1) - len;  // its row in the window that the stream leaves
                    if (m >= 0 && fin) grad = add4(grad, widen4<T>(V::load_raw(fin + m * C)));
                    if (i >= sb) store_act4<T>(dxp + q * a.dx_stride, grad);
                    else if (dst) store_act4<T>(dst + (i - sb + K - 1) * C, grad);
                }
            }
            dxp += kGroup * a.dx_stride;
        }
    }
    float *out = part + (int64_t)slot * (K + 1) * C + c;  // runs without tokens add zeros
#pragma unroll
    for (int j = 0; j < K; ++j) store_f4(out + j * C, dw[j]);
    store_f4(out + K * C, db);
}

// Sums of the runs' parts. A block has 128 columns (of (K + 1) C) and eight groups of the runs; each
// thread adds every eighth run of its four columns, then the groups are joined.
constexpr int kGroups = 8;
__global__ void __launch_bounds__(32 * kGroups)
conv_bwd_sum_kernel(const float *part, const Runs runs, int K, int C, float *dw, float *dbias) {
    __shared__ __align__(16) float sums[kGroups][128];
    wait_for_previous();
    if (runs.bad()) return;
    const int lane = threadIdx.x % 32, g = threadIdx.x / 32, width = (K + 1) * C, slots = runs.slots();
    const int i = (blockIdx.x * 32 + lane) * 4;
    F4 v = all4(0.f);
    if (i < width) {
#pragma unroll 4
        for (int s = g; s < slots; s += kGroups) v = add4(v, load_f4(part + (int64_t)s * width + i));
    }
    store_f4(&sums[g][lane * 4], v);
    __syncthreads();
    const int col = blockIdx.x * 128 + threadIdx.x;
    if (threadIdx.x >= 128 || col >= width) return;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) sum += sums[k][threadIdx.x];
    const int j = col / C, c = col % C;
    if (j < K) dw[(int64_t)c * K + j] = sum;
    else if (dbias) dbias[c] = sum;
}

template <typename T, int K>
cudaError_t launch_t(const ConvBwdArgs &a, cudaStream_t st) {
    const Runs runs{a.cu, a.B, a.T_each, a.total, run_rows(a.B, a.total, a.channels)};
    float *part = static_cast<float *>(a.workspace);
    const dim3 grid(runs.slots(), (a.channels / 4 + kThreads - 1) / kThreads);
    cudaError_t e = cudaFuncSetAttribute(conv_bwd_kernel<T, K>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes<T>);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(conv_bwd_kernel<T, K>, grid, dim3(kThreads), kRingBytes<T>, 0, st, a, runs, part);
    if (e != cudaSuccess) return e;
    return launch_overlapped(conv_bwd_sum_kernel, dim3(((K + 1) * a.channels + 127) / 128), dim3(32 * kGroups), 0, 0, st,
                             (const float *)part, runs, K, a.channels, a.dw, a.dbias);
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

int conv_backward_max_channels() { return 65535 * 4 * kThreads; }  // blocks along a grid's y

size_t conv_backward_workspace_bytes(int B, int total, int channels, int kernel, int) {
    // streams of equal lengths have no more runs than packed ones
    return ((size_t)total / run_rows(B, total, channels) + B) * (kernel + 1) * channels * sizeof(float);
}

cudaError_t launch_conv1d_silu_backward(const ConvBwdArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? launch_k<__nv_bfloat16>(a, st) : launch_k<float>(a, st);
}

}  // namespace la
