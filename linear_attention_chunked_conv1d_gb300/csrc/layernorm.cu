// Layer norm of rows and its backward pass, with the reduction of the weight's and bias's gradients.
//
//   mean = sum_c x_c / n,  rstd = 1 / sqrt(sum_c (x_c - mean)^2 / n + eps),  xh = (x - mean) rstd,
//   y = xh w + b;
//   u = dy w,  dx = rstd (u - mean(u) - xh mean(u xh)) (+ dskip),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// Both are bound by memory: the forward pass reads x and writes y, the backward pass reads x and dy
// and writes dx, each once. A row stays in the registers of its threads between the sums and the
// result (the variance is the sum of the squared differences from the mean, not E x^2 - mean^2, which
// cancels where a row's mean is large). In the backward pass a block takes every gridDim-th row and its
// threads keep the sums over rows of their own columns in registers; what the blocks have is added up
// in the blocks' order by a second launch, so the gradients are the same bits in every run.
#include "dense.cuh"
#include "launch.h"
#include "overlap.cuh"

namespace la {

namespace {

// Sum of v over the TPR threads of a row (all threads of a group get it). Groups are warps (TPR = 32)
// or whole blocks; part: one of two buffers of 32 that successive calls take in turn, so that one barrier
// a call is enough.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float *part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if (TPR == 32) return;
    constexpr int W = TPR / 32;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) part[(threadIdx.x >> 5) * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += part[w * NV + i];
        v[i] = s;
    }
}

// TPR threads a row (32: eight rows a block), P pieces of 16 bytes a thread.
template <class T, int TPR, int P>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
layernorm_kernel(const T *x, const T *__restrict__ w, const T *__restrict__ b, T *y,
                 float2 *__restrict__ stats, int rows, int width, int64_t ldx, int64_t ldy, float eps) {
    constexpr int N = Vec16<T>::N, RPB = TPR == 32 ? 8 : 1;
    __shared__ float part[2][32];
    wait_for_previous();
    const int t = threadIdx.x % TPR;
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (r >= rows) return;  // whole warps of one-warp rows; never where a row has a block
    const T *xr = x + r * ldx;
    float v[P][N];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        if (c < width) {
            load_piece(xr, c, width, v[i]);
#pragma unroll
            for (int e = 0; e < N; ++e) s[0] += v[i][e];
        }
    }
    row_sum<TPR>(s, part[0]);
    const float mean = s[0] / width;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        if (c < width) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] -= mean;
                if (c + e < width) s[0] = fmaf(v[i][e], v[i][e], s[0]);
            }
        }
    }
    row_sum<TPR>(s, part[1]);
    const float rstd = 1.f / sqrtf(s[0] / width + eps);
    if (stats && t == 0) stats[r] = make_float2(mean, rstd);
    T *yr = y + r * ldy;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        if (c < width) {
            float wv[N], bv[N];
            load_piece(w, c, width, wv);
            if (b) load_piece(b, c, width, bv);
#pragma unroll
            for (int e = 0; e < N; ++e) v[i][e] = fmaf(v[i][e] * rstd, wv[e], b ? bv[e] : 0.f);
            store_piece(yr, c, width, v[i]);
        }
    }
}

// partial [gridDim.x][2][width]: a block's sums of dy xh and of dy.
template <class T, int TPR, int P>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR)
layernorm_backward_kernel(const T *__restrict__ x, const T *__restrict__ w, const float2 *__restrict__ stats,
                          const T *dy, const T *dskip, T *dx, float *__restrict__ partial, int rows,
                          int width, int64_t ldx, int64_t lddy, int64_t ldskip, int64_t lddx) {
    constexpr int N = Vec16<T>::N, RPB = TPR == 32 ? 8 : 1;
    __shared__ float part[2][64];
    extern __shared__ float cross[];  // RPB > 1: [RPB][2][width]
    wait_for_previous();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    float aw[P][N] = {}, ab[P][N] = {};
    const float inv = 1.f / width;
    int turn = 0;
    for (int64_t r = (int64_t)blockIdx.x * RPB + g; r < rows; r += (int64_t)gridDim.x * RPB, turn ^= 1) {
        const float2 st = stats[r];
        float xh[P][N], u[P][N];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * TPR) * N;
            if (c < width) {
                load_piece(x + r * ldx, c, width, xh[i]);
                load_piece(dy + r * lddy, c, width, u[i]);
                float wv[N];
                load_piece(w, c, width, wv);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    xh[i][e] = (xh[i][e] - st.x) * st.y;
                    ab[i][e] += u[i][e];
                    aw[i][e] = fmaf(u[i][e], xh[i][e], aw[i][e]);
                    u[i][e] *= wv[e];
                    s[0] += u[i][e];  // zero past the row's end, where dy and w read as zero
                    s[1] = fmaf(u[i][e], xh[i][e], s[1]);
                }
            }
        }
        row_sum<TPR>(s, part[turn]);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * TPR) * N;
            if (c < width) {
                float d[N];
                if (dskip) load_piece(dskip + r * ldskip, c, width, d);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float v = st.y * (u[i][e] - m0 - xh[i][e] * m1);
                    d[e] = dskip ? d[e] + v : v;
                }
                store_piece(dx + r * lddx, c, width, d);
            }
        }
    }
    float *out = partial + (int64_t)blockIdx.x * 2 * width;
    if (RPB > 1) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = (t + i * TPR) * N + e;
                if (c < width) {
                    cross[(g * 2) * width + c] = aw[i][e];
                    cross[(g * 2 + 1) * width + c] = ab[i][e];
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < RPB; ++k) s += cross[k * 2 * width + c];
            out[c] = s;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int c = (t + i * TPR) * N + e;
            if (c < width) {
                out[c] = aw[i][e];
                out[width + c] = ab[i][e];
            }
        }
}

// dw and db from the blocks' sums [blocks][2][width], added up in the blocks' order.
constexpr int SUM_Y = 16;
__global__ void __launch_bounds__(32 * SUM_Y)
layernorm_sums_kernel(const float *__restrict__ partial, int blocks, int width, float *__restrict__ dw,
                      float *__restrict__ db) {
    __shared__ float sh[SUM_Y][33];
    wait_for_previous();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < 2 * width)
        for (int k = threadIdx.y; k < blocks; k += SUM_Y) s += partial[(int64_t)k * 2 * width + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * width) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < SUM_Y; ++k) s += sh[k][threadIdx.x];
        if (c < width) dw[c] = s;
        else if (db) db[c - width] = s;
    }
}

// The least number of pieces a thread that covers a row: f(integral_constant TPR, integral_constant P).
template <int A> using Int = std::integral_constant<int, A>;
template <class T, class F>
cudaError_t with_forward_shape(int width, F &&f) {
    const int pieces = (width + Vec16<T>::N - 1) / Vec16<T>::N;
    if (pieces <= 32) return f(Int<32>{}, Int<1>{});
    if (pieces <= 64) return f(Int<32>{}, Int<2>{});
    if (pieces <= 128) return f(Int<128>{}, Int<1>{});
    if (pieces <= 256) return f(Int<256>{}, Int<1>{});
    if (pieces <= 512) return f(Int<256>{}, Int<2>{});
    if (pieces <= 1024) return f(Int<256>{}, Int<4>{});
    return f(Int<512>{}, Int<4>{});
}
template <class T, class F>
cudaError_t with_backward_shape(int width, F &&f) {
    const int pieces = (width + Vec16<T>::N - 1) / Vec16<T>::N;
    if (pieces <= 32) return f(Int<32>{}, Int<1>{});
    if (pieces <= 64) return f(Int<32>{}, Int<2>{});
    if (pieces <= 128) return f(Int<128>{}, Int<1>{});
    if (pieces <= 256) return f(Int<256>{}, Int<1>{});
    if (pieces <= 512) return f(Int<256>{}, Int<2>{});
    if (pieces <= 1024) return f(Int<512>{}, Int<2>{});
    return f(Int<512>{}, Int<4>{});
}

// Blocks of the backward pass: a few on each SM, no more than there are rows for.
int backward_blocks(int rows, int rpb) {
    const int most = 152 * 4;
    const int need = (rows + rpb - 1) / rpb;
    return need < most ? need : most;
}

template <class T>
cudaError_t forward(const LayerNormArgs &a, cudaStream_t st) {
    return with_forward_shape<T>(a.width, [&](auto tpr, auto p) {
        constexpr int TPR = tpr, RPB = TPR == 32 ? 8 : 1;
        return launch_overlapped(layernorm_kernel<T, TPR, p>, dim3((a.rows + RPB - 1) / RPB), dim3(TPR * RPB), 0, 0, st,
                                 (const T *)a.x, (const T *)a.w, (const T *)a.b, (T *)a.y, (float2 *)a.stats, a.rows,
                                 a.width, a.ldx, a.ldy, a.eps);
    });
}

template <class T>
cudaError_t backward(const LayerNormBwdArgs &a, cudaStream_t st) {
    int blocks = 0;
    cudaError_t e = with_backward_shape<T>(a.width, [&](auto tpr, auto p) {
        constexpr int TPR = tpr, RPB = TPR == 32 ? 8 : 1;
        blocks = backward_blocks(a.rows, RPB);
        const size_t smem = RPB > 1 ? (size_t)RPB * 2 * a.width * sizeof(float) : 0;  // widths up to 512: 32 KB
        return launch_overlapped(layernorm_backward_kernel<T, TPR, p>, dim3(blocks), dim3(TPR * RPB), smem, 0, st,
                                 (const T *)a.x, (const T *)a.w, (const float2 *)a.stats, (const T *)a.dy,
                                 (const T *)a.dskip, (T *)a.dx, (float *)a.workspace, a.rows, a.width, a.ldx, a.lddy,
                                 a.ldskip, a.lddx);
    });
    if (e != cudaSuccess) return e;
    return launch_overlapped(layernorm_sums_kernel, dim3((2 * a.width + 31) / 32), dim3(32, SUM_Y), 0, 0, st,
                             (const float *)a.workspace, blocks, a.width, a.dw, a.db);
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? forward<__nv_bfloat16>(a, st) : forward<float>(a, st);
}
cudaError_t launch_layernorm_backward(const LayerNormBwdArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
}
int layernorm_max_width() { return 512 * 4 * 4; }  // fp32: 512 threads of four pieces of four
size_t layernorm_backward_workspace_bytes(int rows, int width, int) {
    return (size_t)backward_blocks(rows, 1) * 2 * width * sizeof(float);
}

}  // namespace la
