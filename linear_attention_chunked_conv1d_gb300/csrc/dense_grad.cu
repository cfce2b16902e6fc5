// The elementwise halves of the dense layers' backward passes: gradients before the activation, and the
// bias's gradient.
//
//   linear:  dz = dy act'(z),  dbias = sum_rows dz
//   gated:   dgate = dh up act'(gate),  dup = dh act(gate)
//
// Bound by memory: each value is read and written once. dz, dgate and dup are rounded to bf16, the type in
// which the tensor cores take them; the bias's gradient is summed from dz before that rounding.
// 8192 x 8192: dz 70 us (5.7 TB/s; 83 with one row's loads under way at a time), dgate and dup 120 us (6.7 TB/s).
#include "dense.cuh"
#include "launch.h"
#include "overlap.cuh"
#include "tc.cuh"

namespace la {

namespace {

using bf16 = __nv_bfloat16;
constexpr int COLS = 256, WARPS = 8, ROWS = 2;  // a block: 32 lanes of 8 columns, eight warps of a row at a time, twice

// dz may be null (act none: dz is dy). The sums of a block's rows go to partial [gridDim.y][N]; where the blocks of the
// same columns are one cluster (along y) or one block, they add them up, each of some columns, to dbias.
__global__ void __launch_bounds__(32 * WARPS, 4)
linear_grad_kernel(const bf16 *__restrict__ saved, const bf16 *__restrict__ dy, bf16 *__restrict__ dz,
                   float *__restrict__ partial, bf16 *__restrict__ dbias, int M, int N, int64_t lds, int64_t lddy, int64_t ldz, int act, int cluster) {
    __shared__ float sh[WARPS][COLS], mine[COLS];
    wait_for_previous();
    const int c = blockIdx.x * COLS + threadIdx.x * 8;
    float sum[8] = {};
    if (c < N)
        for (int64_t first = blockIdx.y * WARPS + threadIdx.y; first < M; first += (int64_t)gridDim.y * WARPS * ROWS) {
            uint4 dr[ROWS], zr[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {  // several rows' loads are under way at one time
                const int64_t r = first + (int64_t)i * gridDim.y * WARPS;
                if (r >= M) continue;
                dr[i] = load_raw(dy + r * lddy, c, N);
                if (saved) zr[i] = *reinterpret_cast<const uint4 *>(saved + r * lds + c);  // whole pieces: the buffer's rows are
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int64_t r = first + (int64_t)i * gridDim.y * WARPS;
                if (r >= M) break;
                float d[8], z[8], slope[8];
                Vec16<bf16>::load(reinterpret_cast<const bf16 *>(&dr[i]), d);
                if (saved) {
                    Vec16<bf16>::load(reinterpret_cast<const bf16 *>(&zr[i]), z);
                    act_slopes(z, slope, act);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] *= slope[e];
                    Vec16<bf16>::store(dz + r * ldz + c, d);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += d[e];
            }
        }
    if (!dbias) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[threadIdx.y][threadIdx.x * 8 + e] = sum[e];
    __syncthreads();
    const int k = threadIdx.y * 32 + threadIdx.x;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sh[w][k];
    const int at = blockIdx.x * COLS + k;
    if (gridDim.y > 1 && cluster == 1) {
        if (at < N) partial[(int64_t)blockIdx.y * N + at] = s;
        return;
    }
    if (cluster > 1) {
        mine[k] = s;
        tc::cluster_sync();
        if (k % cluster == (int)tc::cluster_rank()) {
            s = 0.f;
            for (int i = 0; i < cluster; ++i) s += tc::ld_shared_cluster(tc::map_to_rank(tc::smem_u32(mine + k), i));
            if (at < N) dbias[at] = __float2bfloat16_rn(s);
        }
        tc::cluster_sync();  // the others have read this block's
    } else if (at < N) {
        dbias[at] = __float2bfloat16_rn(s);
    }
}

__global__ void __launch_bounds__(32 * 16)
bias_sum_kernel(const float *__restrict__ partial, int runs, int N, bf16 *__restrict__ dbias) {
    __shared__ float sh[16][33];
    wait_for_previous();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < N)
        for (int k = threadIdx.y; k < runs; k += 16) s += partial[(int64_t)k * N + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < N) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += sh[k][threadIdx.x];
        dbias[c] = __float2bfloat16_rn(s);
    }
}

// d: [M][2 * half], gate in columns 0.., up from column half on; saved: the same in 24 bits, one plane of 16 and one of 8.
__global__ void __launch_bounds__(256)
gated_grad_kernel(const uint8_t *__restrict__ saved, const uint8_t *__restrict__ lower, const bf16 *__restrict__ dh,
                  bf16 *__restrict__ d, int M, int F, int half, int64_t lddh, int act) {
    wait_for_previous();
    const int c = (blockIdx.x * 32 + threadIdx.x) * 8;
    if (c >= F) return;
    for (int64_t r = blockIdx.y * 8 + threadIdx.y; r < M; r += (int64_t)gridDim.y * 8) {
        float gate[8], up[8], g[8], slope[8];
        const int64_t at = r * 2 * half + c;  // whole pieces: the buffers' rows are
        const uint4 gu = *reinterpret_cast<const uint4 *>(saved + 2 * at), uu = *reinterpret_cast<const uint4 *>(saved + 2 * (at + half));
        const uint2 gl = *reinterpret_cast<const uint2 *>(lower + at), ul = *reinterpret_cast<const uint2 *>(lower + at + half);
        load_piece(dh + r * lddh, c, F, g);
        joined8(gu, gl, gate);
        joined8(uu, ul, up);
        act_slopes(gate, slope, act);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            up[e] *= g[e] * slope[e];
            gate[e] *= g[e];
        }
        Vec16<bf16>::store(d + at, up);
        Vec16<bf16>::store(d + at + half, gate);
    }
}

// Rows are shared out so that the grid has `held` blocks for each SM, or 64 rows a block where that is fewer.
int row_runs(int M, int N, int held) {
    const int cols = (N + COLS - 1) / COLS, most = (int)(((int64_t)M + 8 * WARPS - 1) / (8 * WARPS));
    const int runs = SMS * held / cols < 1 ? 1 : SMS * held / cols;
    return runs < most ? runs : most;
}

}  // namespace

size_t linear_backward_partial_bytes(int M, int N) { return (size_t)row_runs(M, N, 4) * N * sizeof(float); }

cudaError_t launch_linear_grad(const LinearGradArgs &a, cudaStream_t st) {
    // up to eight blocks to a column are one cluster, which needs no second launch for its sums
    const int runs = row_runs(a.M, a.N, 4), cluster = a.dbias && runs <= 8 ? runs : 1;
    cudaError_t e = launch_overlapped(linear_grad_kernel, dim3((a.N + COLS - 1) / COLS, runs), dim3(32, WARPS), 0,
                                      dim3(cluster > 1 ? 1 : 0, cluster, 1), st, (const bf16 *)a.saved, (const bf16 *)a.dy, (bf16 *)a.dz,
                                      a.partial, (bf16 *)a.dbias, a.M, a.N, a.lds, a.lddy, a.ldz, a.act, cluster);
    if (e != cudaSuccess || !a.dbias || runs == cluster) return e;
    return launch_overlapped(bias_sum_kernel, dim3((a.N + 31) / 32), dim3(32, 16), 0, 0, st, (const float *)a.partial, runs,
                             a.N, (bf16 *)a.dbias);
}

cudaError_t launch_gated_grad(const GatedGradArgs &a, cudaStream_t st) {
    return launch_overlapped(gated_grad_kernel, dim3((a.F + COLS - 1) / COLS, row_runs(a.M, a.F, 6)), dim3(32, 8), 0, 0, st,
                             (const uint8_t *)a.saved, (const uint8_t *)a.lower, (const bf16 *)a.dh, (bf16 *)a.d, a.M, a.F, a.half, a.lddh, a.act);
}

}  // namespace la
