// The matrix products of the dense layers' calls on the 5th-generation tensor cores, bf16 operands, fp32
// accumulation in TMEM, one rounding of the result:
//
//   LINEAR  y  = act(x W^T + bias) + residual          x [M][K],  W [N][K]
//   GATED   h  = act(x Wg^T) * (x Wu^T)                x [M][K],  Wg, Wu [N][K]
//   DX      dx = sum_p dz_p W_p                        dz_p [M][K], W_p [K][N]      (p: one or two parts)
//   DW      dW_i = dz_i^T x                            dz_i [K][M], x [K][N]        (i: one or two outputs)
//
// In DX the rows of W, in DW those of both operands run along the summed index: their tiles are taken as they
// lie in memory (MN-major operands), nothing is transposed.
#include <cuda.h>

#include <atomic>

#include "dense.cuh"
#include "dense_maps.cuh"
#include "launch.h"
#include "overlap.cuh"
#include "tc.cuh"

namespace la {

namespace {

constexpr int TM = 256, TN = 256, TK = 64, STAGES = 6;  // a pair's tile; a block holds half of each operand
constexpr uint32_t HALF_BYTES = 128 * TK * 2, STAGE_BYTES = 2 * HALF_BYTES;
constexpr uint32_t OFF_BAR = STAGES * STAGE_BYTES;
constexpr size_t SMEM = OFF_BAR + 256 + 1024;  // barriers, alignment
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr uint32_t SLEEP_NS = 1000000u;
constexpr int BAND = 8;  // tiles of rows that are walked together

// 16 columns from c on of a row with N columns.
__device__ __forceinline__ void store16(__nv_bfloat16 *row, int c, int N, const float *v) {
    if (c < N) store_piece(row, c, N, v);
    if (c + 8 < N) store_piece(row, c + 8, N, v + 8);
}
__device__ __forceinline__ void load16(const __nv_bfloat16 *row, int c, int N, float *v) {
    if (c < N) load_piece(row, c, N, v);
    if (c + 8 < N) load_piece(row, c + 8, N, v + 8);
}

// Tile `t` of an output of mt x nt tiles: bands of BAND tiles of rows, column by column, so that the tiles
// under way at one time share few rows and columns and find them in L2.
__device__ __forceinline__ void tile_place(int64_t t, int64_t mt, int64_t nt, int &m, int &n) {
    const int64_t band = t / (BAND * nt), r = t - band * BAND * nt;
    const int64_t high = mt - band * BAND < BAND ? mt - band * BAND : BAND;
    n = (int)(r / high);
    m = (int)(band * BAND + (r - n * high));
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1)
dense_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue ep, int M, int N, int K, int parts, int outs, int *status,
             uint64_t wait_ns, int debug_stall) {
    constexpr bool A_MN = KIND == DENSE_DW, B_MN = KIND == DENSE_DX || KIND == DENSE_DW;
    constexpr int OUT_N = KIND == DENSE_GATED ? TN / 2 : TN;  // columns of the result a tile holds
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + OFF_BAR);  // the leader's: both blocks' copies of a stage
    uint64_t *empty = full + STAGES;                              // each block's: the MMAs that read a stage
    uint64_t *accf = empty + STAGES;                              // each block's: an accumulator is complete
    uint64_t *acce = accf + 2;                                    // the leader's: both blocks have read it
    uint64_t *fin = acce + 2;                                     // the leader's: its last MMA
    uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(fin + 1);
    volatile int *err = reinterpret_cast<volatile int *>(tmem_sh + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(full + s, 1);
            tc::mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(accf + b, 1);
            tc::mbar_init(acce + b, 2 * EPI_WARPS);
        }
        tc::mbar_init(fin, 1);
        *err = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tmem_sh, 2 * TN);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    wait_for_previous();
    const uint32_t tm = *tmem_sh;
    const int64_t mt = (M + TM - 1) / TM, nt = (N + OUT_N - 1) / OUT_N, per = mt * nt, ntiles = per * outs;
    const int kp = (K + TK - 1) / TK;
    const int64_t kb = (int64_t)kp * parts;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
    const uint32_t sbase = tc::smem_u32(sm);

    if (warp == 0) {
        if (tc::elect_one()) {
            uint32_t it = 0;
            uint64_t t_last = 0;
            for (int64_t tile = first; tile < ntiles && !*err; tile += step) {
                const int o = (int)(tile / per);
                int m, n;
                tile_place(tile - o * per, mt, nt, m, n);
                const int m0 = m * TM + (int)rank * 128;
                const int n0 = KIND == DENSE_GATED ? n * OUT_N : n * TN + (int)rank * 128;
                const CUtensorMap *ma = &maps.a[KIND == DENSE_DW ? o : 0], *mb = &maps.b[KIND == DENSE_GATED ? rank : 0];
                int k0 = 0;
                for (int64_t k = 0; k < kb; ++k, ++it, k0 += TK) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!tc::mbar_wait(empty + s, ph ^ 1u, wait_ns, SLEEP_NS) || *err) {
                        *err = 1;
                        break;
                    }
                    if (KIND == DENSE_DX && k == kp) {
                        ma = &maps.a[1];
                        mb = &maps.b[1];
                        k0 = 0;
                    }
                    const uint32_t da = sbase + s * STAGE_BYTES, db = da + HALF_BYTES;
                    const uint32_t bar = tc::map_to_rank(tc::smem_u32(full + s), 0);
                    if (rank == 0) tc::mbar_expect_tx(full + s, 2 * STAGE_BYTES);
                    if (A_MN) {
                        tc::tma_load_2d_pair(da, ma, m0, k0, bar);
                        tc::tma_load_2d_pair(da + HALF_BYTES / 2, ma, m0 + 64, k0, bar);
                    } else {
                        tc::tma_load_2d_pair(da, ma, k0, m0, bar);
                    }
                    if (B_MN) {
                        tc::tma_load_2d_pair(db, mb, n0, k0, bar);
                        tc::tma_load_2d_pair(db + HALF_BYTES / 2, mb, n0 + 64, k0, bar);
                    } else {
                        tc::tma_load_2d_pair(db, mb, k0, n0, bar);
                    }
                }
            }
            // Every copy has landed before the blocks exit: the leader waits for the last one of each stage, its
            // own and the other block's. Where something went wrong the two may have stopped at different
            // stages; a copy takes microseconds, so each then gives its last ones a millisecond.
            if (*err) {
                t_last = tc::globaltimer_ns();
                while (tc::globaltimer_ns() - t_last < 1000000u) __nanosleep(1000);
            } else if (rank == 0) {
                for (uint32_t s = 0; s < STAGES && s < it; ++s) {
                    const uint32_t last = it - 1 - ((it - 1 - s) % STAGES);
                    if (!tc::mbar_wait(full + s, (last / STAGES) & 1u, WAIT_NS, SLEEP_NS)) *err = 1;
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && tc::elect_one()) {
            constexpr uint32_t id = tc::idesc(TM, TN, tc::FMT_BF16, A_MN, B_MN);
            uint32_t it = 0, tcnt = 0;
            if (debug_stall && !tc::mbar_wait(fin, 0, wait_ns, SLEEP_NS)) *err = 1;
            for (int64_t tile = first; tile < ntiles && !*err; tile += step, ++tcnt) {
                const uint32_t acc = tcnt & 1u, aph = (tcnt >> 1) & 1u;
                if (!tc::mbar_wait(acce + acc, aph ^ 1u, wait_ns, SLEEP_NS)) {
                    *err = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t d = tm + acc * TN;
                bool ok = true;
                for (int64_t k = 0; k < kb; ++k, ++it) {
                    const uint32_t s = it % STAGES, ph = (it / STAGES) & 1u;
                    if (!tc::mbar_wait(full + s, ph, wait_ns, SLEEP_NS) || *err) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t a = sbase + s * STAGE_BYTES, b = a + HALF_BYTES;
#pragma unroll
                    for (uint32_t kk = 0; kk < TK / 16; ++kk)
                        tc::mma_bf16_ss_pair(
                            d, A_MN ? tc::sdesc_sw128_mn(a + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(a + kk * 32u),
                            B_MN ? tc::sdesc_sw128_mn(b + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(b + kk * 32u), id,
                            (k | kk) != 0);
                    tc::mma_commit_pair(empty + s, 3);
                }
                if (!ok) {
                    *err = 1;
                    break;
                }
                tc::mma_commit_pair(accf + acc, 3);
            }
            tc::mma_commit_pair(fin, 1);
            if (!tc::mbar_wait(fin, 0, WAIT_NS, SLEEP_NS)) *err = 1;
        }
    } else {
        const uint32_t q = warp & 3;
        constexpr int COLS = OUT_N / (EPI_WARPS / 4);  // columns of a warp
        const int c_first = (warp - 2) / 4 * COLS;
        const uint64_t acc_ns = wait_ns + kb * 1000;  // a tile takes as long as its summed index is
        uint32_t tcnt = 0;
        for (int64_t tile = first; tile < ntiles; tile += step, ++tcnt) {
            if (__any_sync(0xffffffffu, *err != 0)) break;
            const uint32_t acc = tcnt & 1u, aph = (tcnt >> 1) & 1u;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(accf + acc, aph, acc_ns, SLEEP_NS))) {
                *err = 1;
                break;
            }
            tc::fence_after_sync();
            const int o = (int)(tile / per);
            int m, n;
            tile_place(tile - o * per, mt, nt, m, n);
            const int n0 = n * OUT_N;
            const int64_t row = (int64_t)m * TM + rank * 128 + 32 * q + lane;
#pragma unroll 1
            for (int c = c_first; c < c_first + COLS; c += 16) {
                float v[16], u[16];
                const int col = n0 + c;
                tc::tmem_ld16(tc::tmem_addr(tm + acc * TN, 32 * q, c), v);
                if (KIND == DENSE_GATED) tc::tmem_ld16(tc::tmem_addr(tm + acc * TN, 32 * q, c + TN / 2), u);
                tc::tmem_wait_ld();
                if (row >= M || col >= N) continue;
                if (KIND == DENSE_LINEAR) {
                    if (ep.bias) {
                        load16(ep.bias, col, N, u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += u[e];
                    }
                    if (ep.saved) store16(ep.saved + row * ep.lds, col, N, v);
                    if (ep.act != LA_ACT_NONE)
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = act_value(v[e], ep.act);
                    if (ep.residual) {
                        load16(ep.residual + row * ep.ldr, col, N, u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] += u[e];
                    }
                }
                if (KIND == DENSE_GATED) {
                    if (ep.saved) {
                        store16(ep.saved + row * ep.lds, col, N, v);
                        store16(ep.saved + row * ep.lds + ep.half, col, N, u);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = act_value(v[e], ep.act) * u[e];
                }
                store16(ep.out[o] + row * ep.ldo[o], col, N, v);
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(tc::map_to_rank(tc::smem_u32(acce + acc), 0));
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    tc::cluster_sync();  // the other block's copies, MMAs and arrivals reach this one's memory
    if (warp == 1) tc::tmem_dealloc_pair(tm, 2 * TN);
    if (*err && threadIdx.x == 0) raise_status(status, LA_DEV_TIMEOUT);
}

// Pairs that are resident at one time (looked up once a device).
template <int KIND>
int resident_pairs() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    cudaFuncSetAttribute(dense_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, dense_kernel<KIND>, &cfg) != cudaSuccess || n < 1) return 1;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int KIND>
cudaError_t launch(const DenseArgs &a, cudaStream_t st) {
    constexpr bool A_MN = KIND == DENSE_DW, B_MN = KIND == DENSE_DX || KIND == DENSE_DW;
    constexpr int OUT_N = KIND == DENSE_GATED ? TN / 2 : TN;
    Maps maps;
    if (!make_maps(&maps, a, A_MN, B_MN, 128, 128)) return cudaErrorInvalidValue;
    const Epilogue ep = make_epilogue(a);
    const int parts = KIND == DENSE_DX ? a.count : 1, outs = KIND == DENSE_DW ? a.count : 1;
    const int64_t ntiles = (int64_t)((a.M + TM - 1) / TM) * ((a.N + OUT_N - 1) / OUT_N) * outs;
    const int pairs = resident_pairs<KIND>();
    return launch_overlapped(dense_kernel<KIND>, dim3(2 * (int)(ntiles < pairs ? ntiles : pairs)), dim3(THREADS), SMEM, 2, st,
                             maps, ep, a.M, a.N, a.K, parts, outs, a.status, a.wait_ns ? a.wait_ns : WAIT_NS, a.debug_stall);
}

}  // namespace

cudaError_t launch_dense(const DenseArgs &a, cudaStream_t st) {
    if (dense_split_serves(a)) return launch_dense_split(a, st);
    switch (a.kind) {
        case DENSE_LINEAR: return launch<DENSE_LINEAR>(a, st);
        case DENSE_GATED: return launch<DENSE_GATED>(a, st);
        case DENSE_DX: return launch<DENSE_DX>(a, st);
        default: return launch<DENSE_DW>(a, st);
    }
}

}  // namespace la
