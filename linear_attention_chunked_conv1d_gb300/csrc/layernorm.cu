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
#include <cstring>
#include <type_traits>

#include "dense.cuh"
#include "launch.h"
#include "overlap.cuh"

namespace la {

namespace {

// The pieces of a thread, TPR apart. Whole pieces are loaded without branches, so that all of them are under way at
// one time; then the one that a row may end in.
template <class T, int TPR, int P>
__device__ __forceinline__ void load_row(uint4 (&raw)[P], const T *row, int t, int width) {
    constexpr int N = kPiece<T>;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c + N <= width) raw[i] = *reinterpret_cast<const uint4 *>(row + c);
    }
    if (width % N == 0) return;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        if (c < width && c + N > width) raw[i] = load_raw(row, c, width);
    }
}
// The values of 16 bytes in fp32, as packed pairs (the arithmetic below is on pairs: half the instructions, of
// which a bf16 row takes as long as of its bytes).
__device__ __forceinline__ void widen(const uint4 &v, uint64_t (&f)[2]) {
    f[0] = pk2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pk2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void widen(const uint4 &v, uint64_t (&f)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}
__device__ __forceinline__ float sum_of(uint64_t v) {
    float a, b;
    upk2(v, a, b);
    return a + b;
}
template <class T, int H>
__device__ __forceinline__ void store_pairs(T *row, int c, int width, const uint64_t (&v)[H]) {
    float f[2 * H];
#pragma unroll
    for (int i = 0; i < H; ++i) upk2(v[i], f[2 * i], f[2 * i + 1]);
    store_piece(row, c, width, f);
}

// Sums over the TPR threads of a row (all of them get the sums). part: the row's buffer, of which successive
// calls take one half or the other in turn (turn), so that one barrier a call is enough.
template <int TPR, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float *part, int turn) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if (TPR == 32) return;
    constexpr int W = TPR / 32;
    float *p = part + turn * W * NV;
    const int w = threadIdx.x / 32 % W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) p[w * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) s += p[k * NV + i];
        v[i] = s;
    }
}

// A block is one row's threads, or four rows' of one warp each.
constexpr int block_threads(int tpr) { return tpr == 32 ? 128 : tpr; }

// TPR threads a row, P pieces of 16 bytes a thread.
template <class T, int TPR, int P>
__global__ void __launch_bounds__(block_threads(TPR), (P == 8 ? 768 : 1024) / block_threads(TPR))
layernorm_kernel(const T *x, const T *__restrict__ w, const T *__restrict__ b, T *y, float2 *__restrict__ stats, int rows,
                 int width, int64_t ldx, int64_t ldy, float eps) {
    constexpr int N = kPiece<T>, H = N / 2, G = block_threads(TPR) / TPR;
    __shared__ float part[G][2 * (TPR / 32)];
    wait_for_previous();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int64_t r = (int64_t)blockIdx.x * G + g;
    if (r >= rows) return;  // whole warps, where a block has four rows
    const T *xr = x + r * ldx;
    uint4 raw[P];
    load_row<T, TPR>(raw, xr, t, width);
    uint64_t s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        uint64_t v[H];
        widen(raw[i], v);
#pragma unroll
        for (int e = 0; e < H; ++e) s2 = add2(s2, v[e]);
    }
    float s[1] = {sum_of(s2)};
    row_sum<TPR>(s, part[g], 0);
    const float mean = s[0] / width;
    const uint64_t minus = both(-mean);
    s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        uint64_t v[H];
        widen(raw[i], v);
        if (c + N <= width) {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                v[e] = add2(v[e], minus);
                s2 = fma2(v[e], v[e], s2);
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                float lo, hi;
                upk2(add2(v[e], minus), lo, hi);
                const uint64_t d = pk2(c + 2 * e < width ? lo : 0.f, c + 2 * e + 1 < width ? hi : 0.f);
                s2 = fma2(d, d, s2);
            }
        }
    }
    s[0] = sum_of(s2);
    row_sum<TPR>(s, part[g], 1);
    const float rstd = 1.f / sqrtf(s[0] / width + eps);
    if (stats && t == 0) stats[r] = make_float2(mean, rstd);
    const uint64_t scale = both(rstd);
    T *yr = y + r * ldy;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * TPR) * N;
        if (c < width) {
            uint64_t v[H], wv[H], bv[H] = {};
            widen(raw[i], v);
            widen(load_raw(w, c, width), wv);
            if (b) widen(load_raw(b, c, width), bv);
#pragma unroll
            for (int e = 0; e < H; ++e) v[e] = fma2(mul2(add2(v[e], minus), scale), wv[e], bv[e]);
            store_pairs(yr, c, width, v);
        }
    }
}

// 16 bytes (or, at a row's end, fewer and zeros) from global to shared memory, asynchronously.
template <class T>
__device__ __forceinline__ void copy_piece(void *dst, const T *row, int c, int width) {
    const int n = width - c < kPiece<T> ? (width - c) * (int)sizeof(T) : 16;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(row + c),
                 "r"(n)
                 : "memory");
}

// partial [gridDim.x][2][width]: a block's sums of dy xh and of dy; a single block's are dw and db. Rows come DEPTH ahead through a ring in
// shared memory to which each thread copies its own columns, so that nothing but the row's two sums is shared.
constexpr int depth(int bufs, int p, int threads) { return 3 * bufs * p * threads * 16 > 220 * 1024 ? 2 : 3; }
template <class T, int TPR, int P, bool SKIP>
__global__ void __launch_bounds__(block_threads(TPR), TPR > 128 ? 1 : TPR == 64 ? 4 : 3)
layernorm_backward_kernel(const T *__restrict__ x, const T *__restrict__ w, const float2 *__restrict__ stats, const T *dy,
                          const T *dskip, T *dx, float *__restrict__ partial, float *__restrict__ dw, float *__restrict__ db, int rows, int width, int64_t ldx, int64_t lddy,
                          int64_t ldskip, int64_t lddx) {
    constexpr int N = kPiece<T>, H = N / 2, G = block_threads(TPR) / TPR, BUFS = SKIP ? 3 : 2;
    constexpr int DEPTH = depth(BUFS, P, block_threads(TPR));
    __shared__ float part[G][4 * (TPR / 32)];
    extern __shared__ uint4 ring[];  // [DEPTH][BUFS][P][threads]; then, where G > 1, [G][2][width] fp32
    wait_for_previous();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * G;
    auto slot = [&](int stage, int buf, int i) { return ring + ((stage * BUFS + buf) * P + i) * block_threads(TPR) + threadIdx.x; };
    auto fetch = [&](int64_t r, int stage) {
        if (r < rows)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * TPR) * N;
                if (c < width) {
                    copy_piece(slot(stage, 0, i), x + r * ldx, c, width);
                    copy_piece(slot(stage, 1, i), dy + r * lddy, c, width);
                    if (SKIP) copy_piece(slot(stage, 2, i), dskip + r * ldskip, c, width);
                }
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint64_t aw[P][H] = {}, ab[P][H] = {};
    uint4 wr[P];
    load_row<T, TPR>(wr, w, t, width);
    const float inv = 1.f / width;
    const int64_t first = (int64_t)blockIdx.x * G + g;
    for (int i = 0; i < DEPTH - 1; ++i) fetch(first + i * step, i);
    float2 st = first < rows ? stats[first] : make_float2(0.f, 0.f);
    int stage = 0, turn = 0;
    for (int64_t r = first; r < rows; r += step, turn ^= 1) {
        fetch(r + (DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
        const float2 next = r + step < rows ? stats[r + step] : st;
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        const uint64_t minus = both(-st.x), scale = both(st.y);
        uint64_t s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if ((t + i * TPR) * N >= width) continue;
            uint64_t xv[H], u[H], wv[H];
            widen(*slot(stage, 0, i), xv);
            widen(*slot(stage, 1, i), u);
            widen(wr[i], wv);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const uint64_t xh = mul2(add2(xv[e], minus), scale), uw = mul2(u[e], wv[e]);
                ab[i][e] = add2(ab[i][e], u[e]);
                aw[i][e] = fma2(u[e], xh, aw[i][e]);
                s0 = add2(s0, uw);  // zero past the row's end, where dy and w are zero
                s1 = fma2(uw, xh, s1);
            }
        }
        float s[2] = {sum_of(s0), sum_of(s1)};
        row_sum<TPR>(s, part[g], turn);
        const uint64_t m0 = both(-s[0] * inv), m1 = both(-s[1] * inv);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * TPR) * N;
            if (c >= width) continue;
            uint64_t xv[H], u[H], wv[H], d[H] = {};
            widen(*slot(stage, 0, i), xv);
            widen(*slot(stage, 1, i), u);
            widen(wr[i], wv);
            if (SKIP) widen(*slot(stage, 2, i), d);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const uint64_t xh = mul2(add2(xv[e], minus), scale);
                d[e] = fma2(scale, fma2(xh, m1, fma2(u[e], wv[e], m0)), d[e]);
            }
            store_pairs(dx + r * lddx, c, width, d);
        }
        st = next;
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
    }
    float *out_w = gridDim.x == 1 ? dw : partial + (int64_t)blockIdx.x * 2 * width;
    float *out_b = gridDim.x == 1 ? db : out_w + width;
    float fw[P][N], fb[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < H; ++e) {
            upk2(aw[i][e], fw[i][2 * e], fw[i][2 * e + 1]);
            upk2(ab[i][e], fb[i][2 * e], fb[i][2 * e + 1]);
        }
    if constexpr (G > 1) {
        float *cross = reinterpret_cast<float *>(ring + DEPTH * BUFS * P * block_threads(TPR));
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = (t + i * TPR) * N + e;
                if (c < width) {
                    cross[(g * 2) * width + c] = fw[i][e];
                    cross[(g * 2 + 1) * width + c] = fb[i][e];
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < G; ++k) s += cross[k * 2 * width + c];
            if (c < width) out_w[c] = s;
            else if (out_b) out_b[c - width] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = (t + i * TPR) * N + e;
                if (c < width) {
                    out_w[c] = fw[i][e];
                    if (out_b) out_b[c] = fb[i][e];
                }
            }
    }
}

// dw and db from the blocks' sums [blocks][2][width], added up in the blocks' order.
constexpr int SUM_Y = 32;
__global__ void __launch_bounds__(32 * SUM_Y)
layernorm_sums_kernel(const float *__restrict__ partial, int blocks, int width, float *__restrict__ dw,
                      float *__restrict__ db) {
    __shared__ float sh[SUM_Y][33];
    wait_for_previous();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < 2 * width)
#pragma unroll 8
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

// Threads a row (TPR) and pieces a thread (P): f(integral_constant TPR, integral_constant P).
template <int A> using Int = std::integral_constant<int, A>;
template <class T> int pieces_of(int width) { return (width + kPiece<T> - 1) / kPiece<T>; }

// Many rows: few threads a row, so that its sums take few steps and each thread has several loads under way.
// Few rows: as many threads as a row has pieces for.
template <class T, class F>
cudaError_t with_forward_shape(int rows, int width, F &&f) {
    const int pieces = pieces_of<T>(width);
    if (pieces <= 32) return f(Int<32>{}, Int<1>{});
    if (pieces <= 64) return f(Int<32>{}, Int<2>{});
    if (rows >= 1024) {
        if (pieces <= 128) return f(Int<32>{}, Int<4>{});
        if (pieces <= 256) return f(Int<64>{}, Int<4>{});
        if (pieces <= 512) return f(Int<128>{}, Int<4>{});
        if (pieces <= 1024) return f(Int<256>{}, Int<4>{});
        return f(Int<256>{}, Int<8>{});
    }
    if (pieces <= 128) return f(Int<128>{}, Int<1>{});
    if (pieces <= 256) return f(Int<256>{}, Int<1>{});
    if (pieces <= 512) return f(Int<512>{}, Int<1>{});
    if (pieces <= 1024) return f(Int<512>{}, Int<2>{});
    return f(Int<512>{}, Int<4>{});
}
// A thread keeps the sums of at most 32 columns, in 64 registers.
template <class T, class F>
cudaError_t with_backward_shape(int width, F &&f) {
    const int pieces = pieces_of<T>(width);
    constexpr int Q = 32 / kPiece<T>;
    if (pieces <= 32) return f(Int<32>{}, Int<1>{});
    if (pieces <= 64) return f(Int<32>{}, Int<2>{});
    // (fp32 5001 x 1001: 18.8 us so, 16.1 with twice the threads; bf16 65,536 x 1024: 71 and 88)
    if (pieces <= 32 * Q) return sizeof(T) == 4 ? f(Int<64>{}, Int<Q / 2>{}) : f(Int<32>{}, Int<Q>{});
    if (pieces <= 64 * Q) return f(Int<64>{}, Int<Q>{});
    if (pieces <= 128 * Q) return f(Int<128>{}, Int<Q>{});
    return f(Int<512>{}, Int<Q / 2>{});
}

// Blocks of the backward pass: as many as the SMs' shared memory (and, for three, registers) holds, and no
// more than leave each group of threads four rows (a block's sums are 8 bytes a column, its rows' values six).
constexpr int MOST_BLOCKS = 152 * 4;
int backward_blocks(int rows, int groups, int threads, size_t smem) {
    const int room = (int)(227 * 1024 / (smem + 1024 + 256)), held = threads == 64 ? 4 : threads == 128 ? 3 : 1;
    const int most = 152 * (room < 1 ? 1 : room < held ? room : held);
    if (rows <= 8 * groups) return 1;  // and no second launch
    const int need = (int)(((int64_t)rows + 4 * groups - 1) / (4 * groups));
    return need < most ? need : most;
}

template <class T>
cudaError_t forward(const LayerNormArgs &a, cudaStream_t st) {
    return with_forward_shape<T>(a.rows, a.width, [&](auto tpr, auto p) {
        constexpr int TPR = tpr, G = block_threads(TPR) / TPR;
        return launch_overlapped(layernorm_kernel<T, TPR, p>, dim3((a.rows + G - 1) / G), dim3(block_threads(TPR)), 0, 0, st,
                                 (const T *)a.x, (const T *)a.w, (const T *)a.b, (T *)a.y, (float2 *)a.stats, a.rows, a.width,
                                 a.ldx, a.ldy, a.eps);
    });
}

template <class T>
cudaError_t backward(const LayerNormBwdArgs &a, cudaStream_t st) {
    int blocks = 0;
    cudaError_t e = with_backward_shape<T>(a.width, [&](auto tpr, auto p) {
        constexpr int TPR = tpr, P = p, G = block_threads(TPR) / TPR;
        auto launch = [&](auto kernel, int bufs) {
            const size_t smem = (size_t)depth(bufs, P, block_threads(TPR)) * bufs * P * block_threads(TPR) * 16 + (G > 1 ? (size_t)G * 2 * a.width * 4 : 0);
            blocks = backward_blocks(a.rows, G, block_threads(TPR), smem);
            const cudaError_t set = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (set != cudaSuccess) return set;
            return launch_overlapped(kernel, dim3(blocks), dim3(block_threads(TPR)), smem, 0, st, (const T *)a.x, (const T *)a.w,
                                     (const float2 *)a.stats, (const T *)a.dy, (const T *)a.dskip, (T *)a.dx, (float *)a.workspace, a.dw, a.db,
                                     a.rows, a.width, a.ldx, a.lddy, a.ldskip, a.lddx);
        };
        return a.dskip ? launch(layernorm_backward_kernel<T, TPR, P, true>, 3) : launch(layernorm_backward_kernel<T, TPR, P, false>, 2);
    });
    if (e != cudaSuccess || blocks == 1) return e;
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
int layernorm_max_width() { return 8192; }  // the backward pass: 256 threads of 32 columns
size_t layernorm_backward_workspace_bytes(int rows, int width, int) {
    return (size_t)(rows < MOST_BLOCKS ? rows : MOST_BLOCKS) * 2 * width * sizeof(float);
}

}  // namespace la
