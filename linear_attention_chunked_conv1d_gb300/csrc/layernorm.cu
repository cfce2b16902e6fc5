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
// in the blocks' order, in a cluster or by a second launch, so the gradients are the same bits in every run.
// 16384 x 4096 bf16: forward 44 us (6.1 TB/s), backward 74 (5.4), with dskip 92 (5.8); fp32 forward 77 (7.0).
#include <atomic>
#include <cstring>
#include <type_traits>

#include "dense.cuh"
#include "launch.h"
#include "overlap.cuh"
#include "tc.cuh"

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

// partial [clusters][2][width]: a cluster's sums of dy xh and of dy; a single cluster's are dw and db. Rows come DEPTH ahead
// through a ring in shared memory to which each thread copies its own columns, so that nothing but the row's two sums
// is shared. At the end the blocks of a cluster (as many as `cluster`) add up what they have, each a share of the columns.
constexpr int CLUSTER = 8;
constexpr int depth(int bufs, int p, int threads) { return 3 * bufs * p * threads * 16 > 220 * 1024 ? 2 : 3; }
template <class T, int TPR, int P, bool SKIP>
__global__ void __launch_bounds__(block_threads(TPR), TPR > 128 ? 1 : TPR == 64 ? 4 : 3)
layernorm_backward_kernel(const T *__restrict__ x, const T *__restrict__ w, const float2 *__restrict__ stats, const T *dy,
                          const T *dskip, T *dx, float *__restrict__ partial,
                          float *__restrict__ dw, float *__restrict__ db, int rows, int width, int cluster, int64_t ldx, int64_t lddy,
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
    // what the block has: c, then the sums of columns c and c + 1
    auto each_pair = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < H; ++e) {
                float w0, w1, b0, b1;
                upk2(aw[i][e], w0, w1);
                upk2(ab[i][e], b0, b1);
                f((t + i * TPR) * N + 2 * e, w0, w1, b0, b1);
            }
    };
    const bool whole = gridDim.x == cluster;
    float *out_w = whole ? dw : partial + (int64_t)(blockIdx.x / cluster) * 2 * width, *out_b = whole ? db : out_w + width;
    if (G == 1 && cluster == 1) {
        each_pair([&](int c, float w0, float w1, float b0, float b1) {
            if (c < width) out_w[c] = w0;
            if (c + 1 < width) out_w[c + 1] = w1;
            if (out_b && c < width) out_b[c] = b0;
            if (out_b && c + 1 < width) out_b[c + 1] = b1;
        });
        return;
    }
    float *mine = reinterpret_cast<float *>(G > 1 ? ring + DEPTH * BUFS * P * block_threads(TPR) : ring);  // [G][2][width]
    __syncthreads();  // the ring has been read
    each_pair([&](int c, float w0, float w1, float b0, float b1) {
        float *m = mine + g * 2 * width;
        if (c < width) m[c] = w0, m[width + c] = b0;
        if (c + 1 < width) m[c + 1] = w1, m[width + c + 1] = b1;
    });
    if constexpr (G > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * width; c += blockDim.x) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < G; ++k) s += mine[k * 2 * width + c];
            if (cluster > 1) mine[c] = s;
            else if (c < width) out_w[c] = s;
            else if (out_b) out_b[c - width] = s;
        }
        if (cluster == 1) return;
    }
    const uint32_t rank = tc::cluster_rank(), at = tc::smem_u32(mine);
    tc::cluster_sync();
    for (int c = rank * blockDim.x + threadIdx.x; c < 2 * width; c += cluster * blockDim.x) {
        float v[CLUSTER], s = 0.f;
#pragma unroll
        for (int k = 0; k < CLUSTER; ++k) v[k] = k < cluster ? tc::ld_shared_cluster(tc::map_to_rank(at + c * 4, k)) : 0.f;
#pragma unroll
        for (int k = 0; k < CLUSTER; ++k) s += v[k];
        if (c < width) out_w[c] = s;
        else if (out_b) out_b[c - width] = s;
    }
    tc::cluster_sync();  // the others have read this block's
}

// dw and db from the clusters' sums [blocks][2][width], added up in their order.
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

// Blocks of the backward pass: as many as are resident (looked up once a device), and no more than leave each group of
// threads four rows (a block's sums are 8 bytes a column, its rows' values six). What the blocks have is added up
//  - in one cluster of up to eight, where that leaves a group no more than eight rows: no second launch;
//  - in clusters of four, then by a second launch, where the blocks' sums are 12 MB or more and clusters leave next
//    to no SM idle (16384 x 4096 bf16: 80 us without clusters, 74 with; 32768 x 2048, 10 MB: 78 and 80; fp32 16384 x 4096,
//    where clusters find 288 places of 304: 124 and 137);
//  - by the second launch alone.
constexpr int MOST_BLOCKS = SMS * 4, BIG_CLUSTER = 4;
constexpr size_t CLUSTER_BYTES = 12 << 20;

struct Resident {
    int blocks, in_clusters;  // at one time, without clusters and in clusters of four
};
template <class K>
cudaError_t look_up_resident(K kernel, int threads, size_t smem, Resident *r) {
    int dev = 0, sms = 0, per = 0, clusters = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = BIG_CLUSTER;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(BIG_CLUSTER);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    const int b = per < 1 ? 1 : sms * per, c = clusters * BIG_CLUSTER;
    r->blocks = b < MOST_BLOCKS ? b : MOST_BLOCKS;
    r->in_clusters = c < MOST_BLOCKS ? c : MOST_BLOCKS;
    return e;
}

template <class T, int TPR, int P, bool SKIP>
cudaError_t launch_backward(const LayerNormBwdArgs &a, cudaStream_t st, int *sums) {
    constexpr int G = block_threads(TPR) / TPR, BT = block_threads(TPR), BUFS = SKIP ? 3 : 2;
    constexpr size_t RING = (size_t)depth(BUFS, P, BT) * BUFS * P * BT * 16;
    constexpr size_t MOST_SMEM = RING + (G > 1 ? (size_t)G * 2 * TPR * P * kPiece<T> * 4 : 0);  // at the shape's widest
    auto kernel = layernorm_backward_kernel<T, TPR, P, SKIP>;
    static std::atomic<uint64_t> known[64];  // a Resident
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    Resident r;
    const uint64_t have = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (have) {
        memcpy(&r, &have, sizeof r);
    } else {
        e = look_up_resident(kernel, BT, MOST_SMEM, &r);
        if (e != cudaSuccess) return e;
        uint64_t keep;
        memcpy(&keep, &r, sizeof r);
        if (dev < 64) known[dev].store(keep, std::memory_order_relaxed);
    }
    const int need = (int)(((int64_t)a.rows + 4 * G - 1) / (4 * G));
    int blocks = need < r.blocks ? need : r.blocks, cluster = 1;
    if (a.rows <= 64 * G) {
        blocks = cluster = (a.rows + G - 1) / G < CLUSTER ? (a.rows + G - 1) / G : CLUSTER;
    } else if ((size_t)blocks * 8 * a.width >= CLUSTER_BYTES && r.in_clusters * 20 >= blocks * 19) {
        cluster = BIG_CLUSTER;
        blocks = (blocks < r.in_clusters ? blocks : r.in_clusters) / BIG_CLUSTER * BIG_CLUSTER;
    }
    *sums = blocks / cluster;
    const size_t smem = RING + (G > 1 ? (size_t)G * 2 * a.width * 4 : 0);
    return launch_overlapped(kernel, dim3(blocks), dim3(BT), smem, cluster > 1 ? cluster : 0, st, (const T *)a.x,
                             (const T *)a.w, (const float2 *)a.stats, (const T *)a.dy, (const T *)a.dskip, (T *)a.dx,
                             (float *)a.workspace, a.dw, a.db, a.rows, a.width, cluster, a.ldx, a.lddy, a.ldskip, a.lddx);
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
    int sums = 0;
    const cudaError_t e = with_backward_shape<T>(a.width, [&](auto tpr, auto p) {
        return a.dskip ? launch_backward<T, tpr, p, true>(a, st, &sums) : launch_backward<T, tpr, p, false>(a, st, &sums);
    });
    if (e != cudaSuccess || sums == 1) return e;
    return launch_overlapped(layernorm_sums_kernel, dim3((2 * a.width + 31) / 32), dim3(32, SUM_Y), 0, 0, st,
                             (const float *)a.workspace, sums, a.width, a.dw, a.db);
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? forward<__nv_bfloat16>(a, st) : forward<float>(a, st);
}
cudaError_t launch_layernorm_backward(const LayerNormBwdArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
}
int layernorm_max_width() { return 8192; }  // the backward pass: 512 threads of 16 columns
size_t layernorm_backward_workspace_bytes(int rows, int width, int) {
    return (size_t)(rows < MOST_BLOCKS ? rows : MOST_BLOCKS) * 2 * width * sizeof(float);
}

}  // namespace la
