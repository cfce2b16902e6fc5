// The dense layers' products where few tiles of 256 x 256 come out: few rows (decoding, short prompts) or few
// columns. Such a call is bound by the bytes of its weights, or by having too few tiles for the SMs, so
//  - a block's tile is 128 columns of the result x 16 to 128 of its rows: the columns are the M index of
//    tcgen05.mma (TMEM lanes), the rows its N index, so one token wastes no more than 15 of 16 columns of a tile
//    whose operand bytes are the weights';
//  - the summed index is split over the blocks of a cluster (up to eight): each lays its fp32 part of the tile
//    out in its shared memory, and each adds up a share of the rows over the cluster through distributed shared
//    memory, in the blocks' order, with the epilogue;
//  - two blocks fit an SM, so that one's copies run under the other's prologue and epilogue.
// Operands as in dense_tc.cu, with the roles of rows and columns exchanged.
#include <cuda.h>

#include <atomic>
#include <cmath>

#include "dense.cuh"
#include "dense_maps.cuh"
#include "launch.h"
#include "overlap.cuh"
#include "tc.cuh"

namespace la {

namespace {

constexpr int PT = 128, TK = 64;  // columns of the result, summed indexes of a stage
constexpr uint32_t P_BYTES = PT * TK * 2;
constexpr int THREADS = 192, MAX_STAGES = 8;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr uint32_t SLEEP_NS = 1000000u;

struct Plan {
    int rows;    // rows of the result in a tile (MMA N): 16, 32, 64 or 128
    int split;   // blocks that share the summed index
    int stages;
    uint32_t smem;
};

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Four values of a row from column c on; those at or past N read as zero and are not stored.
__device__ __forceinline__ void load4(const __nv_bfloat16 *row, int c, int N, float *v) {
    if (c + 4 <= N) {
        Vec4<__nv_bfloat16>::load(row + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + e < N ? to_f(row[c + e]) : 0.f;
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16 *row, int c, int N, const float *v) {
    if (c + 4 <= N) {
        Vec4<__nv_bfloat16>::store(row + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < N) row[c + e] = __float2bfloat16_rn(v[e]);
    }
}

// Four values of gate or up for the backward pass (whole pieces: the buffer's rows are).
__device__ __forceinline__ void keep4(const Epilogue &ep, int64_t row, int64_t c, const float *v) {
    *reinterpret_cast<uint2 *>(ep.saved + row * ep.lds + c) = make_uint2(upper2(v[0], v[1]), upper2(v[2], v[3]));
    *reinterpret_cast<uint32_t *>(ep.lower + row * ep.lds + c) = lower4(v[0], v[1], v[2], v[3]);
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 2)
dense_split_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue ep, const Plan plan, int M, int N, int K,
                   int parts, int *status, uint64_t wait_ns, int debug_stall) {
    constexpr bool P_MN = KIND == DENSE_DX || KIND == DENSE_DW, R_MN = KIND == DENSE_DW;
    constexpr int OUT_P = KIND == DENSE_GATED ? PT / 2 : PT;  // columns of the result a tile holds
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(sm);
    uint64_t *empty = full + MAX_STAGES;
    uint64_t *done = empty + MAX_STAGES;
    uint32_t *tmem_sh = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *err = reinterpret_cast<volatile int *>(tmem_sh + 1);
    unsigned char *ring = sm + 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rows = plan.rows, cols = rows < 32 ? 32 : rows;  // TMEM columns
    const uint32_t stage_bytes = P_BYTES + rows * TK * 2;
    const uint32_t rank = plan.split > 1 ? tc::cluster_rank() : 0;
    const int64_t tile = blockIdx.x / plan.split;
    const int pt = (N + OUT_P - 1) / OUT_P;
    const int64_t rt = (M + rows - 1) / rows, per = pt * rt;
    const int o = (int)(tile / per);
    const int p0 = (int)(tile % per % pt) * OUT_P;
    const int64_t r0 = tile % per / pt * rows;
    const int kp = (K + TK - 1) / TK;
    const int64_t kb = (int64_t)kp * parts;
    const int64_t k_first = kb * rank / plan.split, k_end = kb * (rank + 1) / plan.split;
    if (threadIdx.x == 0) {
        for (int s = 0; s < plan.stages; ++s) {
            tc::mbar_init(full + s, 1);
            tc::mbar_init(empty + s, 1);
        }
        tc::mbar_init(done, 1);
        *err = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_sh, cols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    launch_next();
    wait_for_previous();
    const uint32_t tm = *tmem_sh;
    const uint32_t rbase = tc::smem_u32(ring);
    const int nr = (int)(M - r0 < (int64_t)rows ? M - r0 : rows);  // the tile's rows, and those that this block finishes
    const int f = nr * (int)rank / plan.split, l = nr * ((int)rank + 1) / plan.split;

    if (warp == 0) {
        if (tc::elect_one()) {
            uint32_t s = 0, ph = 0, issued = 0;
            for (int64_t k = k_first; k < k_end; ++k) {
                if (!tc::mbar_wait(empty + s, ph ^ 1u, wait_ns, SLEEP_NS) || *err) {
                    *err = 1;
                    break;
                }
                const int part = k >= kp;
                const int k0 = (int)(k - (int64_t)part * kp) * TK;
                const CUtensorMap *mp = &maps.b[KIND == DENSE_DX ? part : 0], *mr = &maps.a[KIND == DENSE_DW ? o : KIND == DENSE_DX ? part : 0];
                const uint32_t dp = rbase + s * stage_bytes, dr = dp + P_BYTES;
                tc::mbar_expect_tx(full + s, stage_bytes);
                if (P_MN) {
                    tc::tma_load_2d(dp, mp, p0, k0, full + s);
                    tc::tma_load_2d(dp + P_BYTES / 2, mp, p0 + 64, k0, full + s);
                } else {
                    tc::tma_load_2d(dp, mp, k0, p0, full + s);
                    tc::tma_load_2d(dp + P_BYTES / 2, KIND == DENSE_GATED ? &maps.b[1] : mp, k0, KIND == DENSE_GATED ? p0 : p0 + 64, full + s);
                }
                if (R_MN) {
                    for (uint32_t i = 0; i < rows / 64; ++i) tc::tma_load_2d(dr + i * 8192, mr, (int)r0 + i * 64, k0, full + s);
                } else {
                    tc::tma_load_2d(dr, mr, k0, (int)r0, full + s);
                }
                ++issued;
                if (++s == (uint32_t)plan.stages) s = 0, ph ^= 1u;
            }
            // every copy has landed before the ring is used for the sums, or the block exits
            for (int i = 0; i < plan.stages && (uint32_t)i < issued; ++i) {
                const uint32_t last = issued - 1 - (issued - 1 - i) % plan.stages;
                if (!tc::mbar_wait(full + i, (last / plan.stages) & 1u, WAIT_NS, SLEEP_NS)) *err = 1;
            }
        }
    } else if (warp == 1) {
        if (tc::elect_one()) {
            const uint32_t id = tc::idesc(PT, rows, tc::FMT_BF16, P_MN, R_MN);
            uint32_t s = 0, ph = 0;
            if (debug_stall && !tc::mbar_wait(done, 0, wait_ns, SLEEP_NS)) *err = 1;
            for (int64_t k = k_first; k < k_end; ++k) {
                if (*err || !tc::mbar_wait(full + s, ph, wait_ns, SLEEP_NS)) {
                    *err = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t p = rbase + s * stage_bytes, r = p + P_BYTES;
#pragma unroll
                for (uint32_t kk = 0; kk < TK / 16; ++kk)
                    tc::mma_bf16_ss(tm, P_MN ? tc::sdesc_sw128_mn(p + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(p + kk * 32u),
                                    R_MN ? tc::sdesc_sw128_mn(r + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(r + kk * 32u), id,
                                    (k > k_first) || kk != 0);
                tc::mma_commit(empty + s);
                if (++s == (uint32_t)plan.stages) s = 0, ph ^= 1u;
            }
            tc::mma_commit(done);
            if (!tc::mbar_wait(done, 0, WAIT_NS + (k_end - k_first) * 1000, SLEEP_NS)) *err = 1;
        }
    } else if (KIND == DENSE_LINEAR && ep.residual) {  // the residual's lines are on their way to L2 meanwhile
        for (int i = threadIdx.x - 64; i < 2 * (l - f); i += THREADS - 64) {
            const int col = p0 + i % 2 * 64;
            if (col < N) asm volatile("prefetch.global.L2 [%0];" ::"l"(ep.residual + (r0 + f + i / 2) * ep.ldr + col));
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();  // copies have landed, MMAs are done: the ring is free
    tc::fence_after_sync();
    // the block's part of the tile, [rows][128 lanes] fp32
    float *part = reinterpret_cast<float *>(ring);
    if (warp >= 2) {
        const uint32_t q = warp & 3;
#pragma unroll 1
        for (uint32_t c = 0; c < rows; c += 16) {
            float v[16];
            tc::tmem_ld16(tc::tmem_addr(tm, 32 * q, c), v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) part[(c + e) * PT + 32 * q + lane] = v[e];
        }
        tc::fence_before_sync();
    }
    if (plan.split > 1) tc::cluster_sync();
    else __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, cols);
    constexpr int LANES = OUT_P / 4, ROWS_AT = 32 / LANES;  // lanes and rows of a warp at one time
    const int c4 = lane % LANES * 4, col = p0 + c4;
    constexpr int AT = THREADS / 32 * ROWS_AT, U = 4;  // rows of the block at one time; how many times over
    for (int first = f + warp * ROWS_AT + lane / LANES; first < l && col < N && !*err; first += U * AT) {
        float v[U][4] = {}, u[U][4] = {}, res[U][4];
        if (KIND == DENSE_LINEAR && ep.residual) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (first + i * AT < l) load4(ep.residual + (r0 + first + i * AT) * ep.ldr, col, N, res[i]);
        }
        float bias[4] = {};
        if (KIND == DENSE_LINEAR && ep.bias) load4(ep.bias, col, N, bias);
        for (int k = 0; k < plan.split; ++k) {
            const uint32_t at = rbase + (first * PT + c4) * 4, src = plan.split > 1 ? tc::map_to_rank(at, k) : at;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (first + i * AT < l) {
                    const float4 t = ld_cluster(src + i * AT * PT * 4);
                    v[i][0] += t.x; v[i][1] += t.y; v[i][2] += t.z; v[i][3] += t.w;
                    if (KIND == DENSE_GATED) {
                        const float4 t2 = ld_cluster(src + i * AT * PT * 4 + PT / 2 * 4);
                        u[i][0] += t2.x; u[i][1] += t2.y; u[i][2] += t2.z; u[i][3] += t2.w;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (first + i * AT >= l) break;
            const int64_t row = r0 + first + i * AT;
            if (KIND == DENSE_LINEAR) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] += bias[e];
                if (ep.saved) store4(ep.saved + row * ep.lds, col, N, v[i]);
                act_values(v[i], ep.act);
                if (ep.residual) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] += res[i][e];
                }
            }
            if (KIND == DENSE_GATED) {
                if (ep.saved) {
                    keep4(ep, row, col, v[i]);
                    keep4(ep, row, col + ep.half, u[i]);
                }
                act_values(v[i], ep.act);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] *= u[i][e];
            }
            store4(ep.out[o] + row * ep.ldo[o], col, N, v[i]);
        }
    }
    if (plan.split > 1) tc::cluster_sync();  // the others have read this block's part
    if (*err && threadIdx.x == 0) raise_status(status, LA_DEV_TIMEOUT);
}

int out_cols(const DenseArgs &a) { return a.kind == DENSE_GATED ? PT / 2 : PT; }

Plan make_plan(const DenseArgs &a) {
    Plan p{};
    p.rows = a.kind == DENSE_DW ? 128 : a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
    const int64_t tiles = (int64_t)((a.N + out_cols(a) - 1) / out_cols(a)) * ((a.M + p.rows - 1) / p.rows) * (a.kind == DENSE_DW ? a.count : 1);
    const int64_t kb = (int64_t)((a.K + TK - 1) / TK) * (a.kind == DENSE_DX ? a.count : 1);
    int64_t split = 304 / tiles;  // two blocks on each SM
    if (split > kb / 4) split = kb / 4;
    p.split = split < 1 ? 1 : split > 8 ? 8 : (int)split;
    const uint32_t stage = P_BYTES + p.rows * TK * 2, room = 110 * 1024;
    p.stages = room / stage < MAX_STAGES ? room / stage : MAX_STAGES;
    p.smem = 2048 + p.stages * stage;
    return p;
}

template <int KIND>
cudaError_t launch(const DenseArgs &a, cudaStream_t st) {
    constexpr bool P_MN = KIND == DENSE_DX || KIND == DENSE_DW, R_MN = KIND == DENSE_DW;
    const Plan plan = make_plan(a);
    Maps maps;
    if (!make_maps(&maps, a, R_MN, P_MN, plan.rows, 64)) return cudaErrorInvalidValue;
    const Epilogue ep = make_epilogue(a);
    const int parts = KIND == DENSE_DX ? a.count : 1, outs = KIND == DENSE_DW ? a.count : 1;
    const int64_t tiles = (int64_t)((a.N + out_cols(a) - 1) / out_cols(a)) * ((a.M + plan.rows - 1) / plan.rows) * outs;
    static std::atomic<uint64_t> set;  // devices on which the kernel may have its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(dense_split_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, 113 * 1024);
        if (e != cudaSuccess) return e;
        if (dev < 64) set.fetch_or(1ull << dev);
    }
    return launch_overlapped(dense_split_kernel<KIND>, dim3((unsigned)(tiles * plan.split)), dim3(THREADS), plan.smem,
                             plan.split > 1 ? plan.split : 0, st, maps, ep, plan, a.M, a.N, a.K, parts, a.status,
                             a.wait_ns ? a.wait_ns : WAIT_NS, a.debug_stall);
}

}  // namespace

// Which kernel a call takes: the one whose time is the shorter by what both were measured to take, in us:
//   pairs (dense_tc.cu)  5 + for each time the tiles go round the 76 pairs 0.29 a stage of 64 summed indexes and no less
//                        than 3.2, the epilogue's; and no less than 7 + bytes / 6 TB/s;
//   this one             2 + for each time the blocks go round the 304 places 6 and 0.41 a stage of 32 KB; and no less
//                        than 6 + bytes / 6 TB/s.
// Pairs and this kernel, M x N x K: linear 1 x 4096 x 4096 23.9 and 10.0, 128: 24.2 and 16.0, 512: 24.8 and 23.5,
// 1024: 26.0 and 36.2; 1024 x 1024 x 8192 41.1 and 22.8; 2048 x 2048 x 2048 17.4 and 23.9; 777 x 5008 x 2048 24.6 and
// 21.0, with bias, GELU and residual 29.5 and 30.5; 8192 x 8192 x 64 46.5 and 112; gated 32 x 8192 x 4096 29.5 and 25.5,
// 256: 30.8 and 35.6; dx 256 x 8192 x 4096 40.7 and 24.2, 1024: 43.0 and 57.3; dw of 16384 rows, 1024 x 1024: 74.2 and
// 35.9, of 1024 rows, 2048 x 2048: 12.1 and 16.1.
bool dense_split_serves(const DenseArgs &a) {
    const Plan p = make_plan(a);
    const double twice = a.kind == DENSE_GATED ? 2 : 1, outs = a.kind == DENSE_DW ? a.count : 1, parts = a.kind == DENSE_DX ? a.count : 1;
    const double M = a.M, N = a.N * twice, K = a.K * parts, kb = ceil(a.K / 64.) * parts;
    const double memory = 2 * (a.kind == DENSE_DW ? outs * (M * K + M * N) + K * N : M * K + N * K + M * a.N) * (1 / 6e6);
    const double pairs = fmax(5 + ceil(ceil(M / 256) * ceil(N / 256) * outs / 76) * fmax(0.29 * kb, 3.2), 7 + memory);
    const double blocks = ceil(M / p.rows) * ceil(N / PT) * outs * p.split;
    const double stage = 0.41 * (P_BYTES + p.rows * TK * 2) / 32768;
    return blocks < 1e6 && fmax(2 + ceil(blocks / 304) * (6 + stage * kb / p.split), 6 + memory) < pairs;
}

cudaError_t launch_dense_split(const DenseArgs &a, cudaStream_t st) {
    switch (a.kind) {
        case DENSE_LINEAR: return launch<DENSE_LINEAR>(a, st);
        case DENSE_GATED: return launch<DENSE_GATED>(a, st);
        case DENSE_DX: return launch<DENSE_DX>(a, st);
        default: return launch<DENSE_DW>(a, st);
    }
}

}  // namespace la
