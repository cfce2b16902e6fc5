// The dense layers' products where few tiles of 256 x 256 come out: few rows (decoding, short prompts) or few
// columns. Such a call is bound by the bytes of its weights, or by having too few tiles for the SMs, so
//  - a block's tile is 128 columns of the result x 16 to 128 of its rows: the columns are the M index of
//    tcgen05.mma (TMEM lanes), the rows its N index, so one token wastes no more than 15 of 16 columns of a tile
//    whose operand bytes are the weights';
//  - the summed index is split over the blocks of a cluster (up to eight): each lays its fp32 part of the tile
//    out in its shared memory, and each adds up a share of the rows over the cluster through distributed shared
//    memory, in the blocks' order, with the epilogue;
//  - two blocks fit an SM, so that one's copies run under the other's prologue and epilogue.
// 1 x 8192 x 2048 takes 9.3 us in a row of calls (33.6 MB; alone, the last of 256 blocks starts 1.3 us after the first, and
// of a block's time 1.0 are its barriers and tensor memory, 2.3 its first copy, 3.2 the way from there to its last MMA, 1.4 the
// cluster's meeting, 1.3 the sums and its leave),
// gated 32 x 8192 x 4096 25 us (5.4 TB/s), gated 1 x 16384 x 4096 42 us (6.3 TB/s).
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
constexpr int THREADS = 256, MAX_STAGES = 8;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr uint32_t SLEEP_NS = 1000000u;

enum { LINEAR = DENSE_LINEAR, GATED = DENSE_GATED, BACKWARD };

// One product of a launch (BACKWARD: up to two; the blocks that share a summed index are as many for both).
struct Job {
    int M, N, K, parts;
    bool dw;      // BACKWARD: DW, else DX
    int rows;     // rows of the result in a tile (MMA N): 16, 32, 64 or 128
    int stages;
    int64_t tiles;
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
dense_split_kernel(const __grid_constant__ Maps maps0, const __grid_constant__ Maps maps1, const __grid_constant__ Epilogue ep0,
                   const __grid_constant__ Epilogue ep1, const __grid_constant__ Job job0, const __grid_constant__ Job job1,
                   int split, int beside, int *status, uint64_t wait_ns, int debug_stall) {
    constexpr bool P_MN = KIND == BACKWARD;
    constexpr int OUT_P = KIND == GATED ? PT / 2 : PT;  // columns of the result a tile holds
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
    const uint32_t rank = split > 1 ? tc::cluster_rank() : 0;
    const int64_t at_tile = blockIdx.x / split;
    const bool second = KIND == BACKWARD && at_tile >= job0.tiles;
    const Job &job = second ? job1 : job0;
    const Maps &maps = second ? maps1 : maps0;
    const Epilogue &ep = second ? ep1 : ep0;
    const int64_t tile = second ? at_tile - job0.tiles : at_tile;
    const int M = job.M, N = job.N, K = job.K, stages = job.stages;
    const bool r_mn = KIND == BACKWARD && job.dw;
    const uint32_t rows = job.rows, cols = rows < 32 ? 32 : rows;  // TMEM columns
    const uint32_t stage_bytes = P_BYTES + rows * TK * 2;
    const int pt = (N + OUT_P - 1) / OUT_P;
    const int64_t rt = (M + rows - 1) / rows, per = pt * rt;
    const int o = (int)(tile / per);
    const int p0 = (int)(tile % per % pt) * OUT_P;
    const int64_t r0 = tile % per / pt * rows;
    const int kp = (K + TK - 1) / TK;
    const int64_t kb = (int64_t)kp * job.parts;
    const int64_t k_first = kb * rank / split, k_end = kb * (rank + 1) / split;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
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
    if (beside == 2) start_beside();  // the kernel ahead has waited, and this one's rows are not that one's
    else wait_for_previous();
    const uint32_t tm = *tmem_sh;
    const uint32_t rbase = tc::smem_u32(ring);
    const int nr = (int)(M - r0 < (int64_t)rows ? M - r0 : rows);  // the tile's rows, and those that this block finishes
    const int f = nr * (int)rank / split, l = nr * ((int)rank + 1) / split;

    if (warp == 0) {
        if (tc::elect_one()) {
            uint32_t s = 0, ph = 0, issued = 0;
            if (beside == 2) beside_tma();
            for (int64_t k = k_first; k < k_end; ++k) {
                if (!tc::mbar_wait(empty + s, ph ^ 1u, wait_ns, SLEEP_NS) || *err) {
                    *err = 1;
                    break;
                }
                const int part = k >= kp;
                const int k0 = (int)(k - (int64_t)part * kp) * TK;
                const CUtensorMap *mp = &maps.b[KIND == BACKWARD ? part : 0], *mr = &maps.a[r_mn ? o : part];
                const uint32_t dp = rbase + s * stage_bytes, dr = dp + P_BYTES;
                tc::mbar_expect_tx(full + s, stage_bytes);
                if (P_MN) {
                    tc::tma_load_2d(dp, mp, p0, k0, full + s);
                    tc::tma_load_2d(dp + P_BYTES / 2, mp, p0 + 64, k0, full + s);
                } else {
                    tc::tma_load_2d(dp, mp, k0, p0, full + s);
                    tc::tma_load_2d(dp + P_BYTES / 2, KIND == GATED ? &maps.b[1] : mp, k0, KIND == GATED ? p0 : p0 + 64, full + s);
                }
                if (r_mn) {
                    for (uint32_t i = 0; i < rows / 64; ++i) tc::tma_load_2d(dr + i * 8192, mr, (int)r0 + i * 64, k0, full + s);
                } else {
                    tc::tma_load_2d(dr, mr, k0, (int)r0, full + s);
                }
                ++issued;
                if (++s == (uint32_t)stages) s = 0, ph ^= 1u;
            }
            // every copy has landed before the ring is used for the sums, or the block exits
            for (int i = 0; i < stages && (uint32_t)i < issued; ++i) {
                const uint32_t last = issued - 1 - (issued - 1 - i) % stages;
                if (!tc::mbar_wait(full + i, (last / stages) & 1u, WAIT_NS, SLEEP_NS)) *err = 1;
            }
        }
    } else if (warp == 1) {
        if (tc::elect_one()) {
            const uint32_t id = tc::idesc(PT, rows, tc::FMT_BF16, P_MN, r_mn);
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
                                    r_mn ? tc::sdesc_sw128_mn(r + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(r + kk * 32u), id,
                                    (k > k_first) || kk != 0);
                tc::mma_commit(empty + s);
                if (++s == (uint32_t)stages) s = 0, ph ^= 1u;
            }
            tc::mma_commit(done);
            if (!tc::mbar_wait(done, 0, WAIT_NS + (k_end - k_first) * 1000, SLEEP_NS)) *err = 1;
        }
    } else if (KIND == LINEAR && ep.residual) {  // the residual's lines are on their way to L2 meanwhile
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
    const uint32_t q = warp & 3;  // the warp's TMEM lanes; its columns are every other 16
#pragma unroll 1
    for (uint32_t c = warp / 4 * 16; c < rows; c += 32) {
        float v[16] = {};
        if (k_first < k_end) {  // a short sum may leave some blocks nothing
            tc::tmem_ld16(tc::tmem_addr(tm, 32 * q, c), v);
            tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * PT + 32 * q + lane] = v[e];
    }
    tc::fence_before_sync();
    if (split > 1) tc::cluster_sync();
    else __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, cols);
    constexpr int LANES = OUT_P / 4, ROWS_AT = 32 / LANES;  // lanes and rows of a warp at one time
    const int c4 = lane % LANES * 4, col = p0 + c4;
    constexpr int AT = THREADS / 32 * ROWS_AT, U = 4;  // rows of the block at one time; how many times over
    for (int first = f + warp * ROWS_AT + lane / LANES; first < l && col < N && !*err; first += U * AT) {
        float v[U][4] = {}, u[U][4] = {}, res[U][4];
        if (KIND == LINEAR && ep.residual) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (first + i * AT < l) load4(ep.residual + (r0 + first + i * AT) * ep.ldr, col, N, res[i]);
        }
        float bias[4] = {};
        if (KIND == LINEAR && ep.bias) load4(ep.bias, col, N, bias);
        for (int k = 0; k < split; ++k) {
            const uint32_t at = rbase + (first * PT + c4) * 4, src = split > 1 ? tc::map_to_rank(at, k) : at;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (first + i * AT < l) {
                    const float4 t = ld_cluster(src + i * AT * PT * 4);
                    v[i][0] += t.x; v[i][1] += t.y; v[i][2] += t.z; v[i][3] += t.w;
                    if (KIND == GATED) {
                        const float4 t2 = ld_cluster(src + i * AT * PT * 4 + PT / 2 * 4);
                        u[i][0] += t2.x; u[i][1] += t2.y; u[i][2] += t2.z; u[i][3] += t2.w;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (first + i * AT >= l) break;
            const int64_t row = r0 + first + i * AT;
            if (KIND == LINEAR) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] += bias[e];
                if (ep.saved) store4(ep.saved + row * ep.lds, col, N, v[i]);
                act_values(v[i], ep.act);
                if (ep.residual) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] += res[i][e];
                }
            }
            if (KIND == GATED) {
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
    if (split > 1) tc::cluster_sync();  // the others have read this block's part
    if (beside == 2) end_beside();
    if (*err && threadIdx.x == 0) raise_status(status, LA_DEV_TIMEOUT);
}

constexpr uint32_t ROOM = 110 * 1024;  // a block's ring: two blocks fit an SM
constexpr int PLACES = 2 * SMS;

Job make_job(const DenseArgs &a) {
    const int64_t out = a.kind == DENSE_GATED ? PT / 2 : PT;
    Job j{a.M, a.N, a.K, a.kind == DENSE_DX ? a.count : 1, a.kind == DENSE_DW, 0, 0, 0};
    j.rows = a.kind == DENSE_DW ? 128 : a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
    const uint32_t stage = P_BYTES + j.rows * TK * 2;
    j.stages = ROOM / stage < MAX_STAGES ? ROOM / stage : MAX_STAGES;
    j.tiles = (a.N + out - 1) / out * (((int64_t)a.M + j.rows - 1) / j.rows) * (a.kind == DENSE_DW ? a.count : 1);
    return j;
}
int64_t stages_of(const Job &j) { return (int64_t)((j.K + TK - 1) / TK) * j.parts; }

// Never launched: what the runtime is asked about in place of the kernels above, of which it counts one block an SM, as they
// take tensor memory. Two are there: 128 of 512 columns, 128 registers for each of 256 threads and 112 KB leave room for both.
__global__ void __launch_bounds__(THREADS, 2) places_kernel() {}

// Clusters of s blocks (2..8) that are resident at one time: the SMs of a GPC hold whole clusters only, so some sizes leave
// many places empty (36 clusters of 8, 38 of 7, 46 of 6, 58, 74, 97, 152 of 2). One more takes another round: 49 tiles of one row,
// 2048 summed, 12.3 us in clusters of 6 and 7.8 of 5; 59 tiles 13.7 of 5 and 8.8 of 4; 75 tiles 16.6 of 4 and 10.6 of 3; 98
// tiles 18.4 of 3 and 13.3 of 2. Looked up once a device.
int resident_clusters(int s) {
    static std::atomic<int> known[64][9];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PLACES / s;
    n = known[dev][s].load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = ROOM + 2048;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(places_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ROOM + 2048) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, places_kernel, &cfg) != cudaSuccess || n < 1)
        return PLACES / s;
    known[dev][s].store(n, std::memory_order_relaxed);
    return n;
}

// Blocks of a cluster: as many as there are places for, each with four stages or more of the longer sum. Not seven, though: one
// row, 37 and 38 tiles of 8192 summed take 17.1 and 17.4 us in sevens, 16.5 and 16.7 in sixes, of 4096 10.7 and 11.1 to 10.5 and
// 10.8; of 1792 to 2048, where four stages a block allow no more than seven, 4 to 39 tiles are the same in both.
int choose_split(const Job &a, const Job *b, int places) {
    const int64_t tiles = a.tiles + (b ? b->tiles : 0), kb = b && stages_of(*b) > stages_of(a) ? stages_of(*b) : stages_of(a);
    int64_t s = places / tiles;
    if (s > kb / 4) s = kb / 4;
    if (s > 8) s = 8;
    while (s > 1 && resident_clusters((int)s) < tiles) --s;
    if (s == 7) s = 6;
    return s < 1 ? 1 : (int)s;
}

template <int KIND>
cudaError_t launch(const DenseArgs &a, const DenseArgs *b, cudaStream_t st) {
    const Job j0 = make_job(a), j1 = b ? make_job(*b) : Job{};
    const int split = choose_split(j0, b ? &j1 : nullptr, a.places ? a.places : PLACES);
    Maps maps[2];
    if (!make_maps(&maps[0], a, j0.dw, KIND == BACKWARD, j0.rows, 64) || (b && !make_maps(&maps[1], *b, j1.dw, KIND == BACKWARD, j1.rows, 64)))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> set;  // devices on which the kernel may have its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(dense_split_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, ROOM + 2048);
        if (e != cudaSuccess) return e;
        if (dev < 64) set.fetch_or(1ull << dev);
    }
    return launch_overlapped(dense_split_kernel<KIND>, dim3((unsigned)((j0.tiles + j1.tiles) * split)), dim3(THREADS), ROOM + 2048,
                             split > 1 ? split : 0, st, maps[0], b ? maps[1] : maps[0], make_epilogue(a), make_epilogue(b ? *b : a), j0,
                             j1, split, a.beside, a.status, a.wait_ns ? a.wait_ns : WAIT_NS, a.debug_stall);
}

// What the operands and results of a product weigh, in us at 6 TB/s.
double memory_us(const DenseArgs &a) {
    const double M = a.M, N = a.N, K = a.K, c = a.count;
    const double values = a.kind == DENSE_DW ? c * (M * K + M * N) + K * N : a.kind == DENSE_DX ? c * (M * K + N * K) + M * N
                                                                           : M * K + (a.kind == DENSE_GATED ? 2 : 1) * N * K + M * N;
    return values * (2 / 6e6);
}
// n things that take a and m that take b, side by side in `places`; the rest of a last round takes `last` of its time
// where it fills no more than half the places.
double rounds(double a, double n, double b, double m, double places, double last) {
    const double longest = m > 0 && b > a ? b : a, all = n + m, rest = all - places * floor(all / places);
    const double tail = rest == 0 ? 0 : 2 * rest <= places ? last : 1;
    if (all <= places) return longest * tail + (tail == 0 ? longest : 0);
    return m > 0 ? fmax(longest, (a * n + b * m) / places) + longest / 2 : a * (floor(n / places) + tail);
}

}  // namespace

// What a product, or two in one launch, take by either kernel, in us, as far as sizes say:
//   pairs (dense_tc.cu)  5 + for each time the tiles go round the 76 pairs 0.29 a stage of 64 summed indexes and no less
//                        than 3.2, the epilogue's (0.7 of it for a round of halves); and no less than 7 + bytes / 6 TB/s;
//   this one             2 + for each time the blocks go round the 304 places 3, 0.04 a row of the tile and 0.41 a stage
//                        of 32 KB; and no less than 6 + bytes / 6 TB/s.
// Pairs and this kernel as measured, M x N x K: linear 1 x 4096 x 4096 23.9 and 10.0, 256: 20.0 and 17.3, 512: 20.5 and
// 21.4, 1024: 26.0 and 36.2; 256 x 2048 x 2048 12.5 and 13.4; 300 x 1000 x 1000 10.7 and 11.4; 1024 x 1024 x 8192 32.1 and
// 23.3; 777 x 5008 x 2048 22.7 and 20.2, with bias, GELU and residual 27.6 and 27.9; 8192 x 8192 x 64 46.5 and 112; gated
// 32 x 8192 x 4096 29.5 and 25.5, 128: 29.5 and 28.9, 256: 30.8 and 35.6; dx 512 x 4096 x 4096 19.9 and 20.6; dw of 16384
// rows, 1024 x 1024: 57.1 and 36.0, of 4096 rows: 18.5 and 16.3, of 1024 rows: 8.5 and 10.8.
//   Parts of dW's sum (split) add a launch of 4 us and their values, written and read at 4 TB/s.
double dense_pairs_us(const DenseArgs &a, const DenseArgs *b) {
    auto parts = [](const DenseArgs &q) { return q.kind == DENSE_DW && q.split > 1 ? q.split : 1.; };
    auto tiles = [&](const DenseArgs &q) {
        return ceil(q.M / 256.) * ceil(q.N * (q.kind == DENSE_GATED ? 2. : 1.) / 256) * (q.kind == DENSE_DW ? q.count : 1) * parts(q);
    };
    auto time = [&](const DenseArgs &q) { return fmax(0.29 * ceil(ceil(q.K / 64.) / parts(q)) * (q.kind == DENSE_DX ? q.count : 1), 3.2); };
    auto join = [&](const DenseArgs &q) { return parts(q) > 1 ? 4 + parts(q) * q.count * q.M * (double)q.N * (8 / 4e6) : 0; };
    return fmax(5 + rounds(time(a), tiles(a), b ? time(*b) : 0, b ? tiles(*b) : 0, PAIRS, 0.7),
                7 + memory_us(a) + (b ? memory_us(*b) : 0)) + join(a) + (b ? join(*b) : 0);
}
double dense_split_us(const DenseArgs &a, const DenseArgs *b) {
    const Job j0 = make_job(a), j1 = b ? make_job(*b) : Job{};
    if (j0.tiles + j1.tiles > 1000000) return 1e30;
    const int places = a.places ? a.places : PLACES;
    const double s = choose_split(j0, b ? &j1 : nullptr, places);
    auto time = [&](const Job &j) { return 3 + 0.04 * j.rows + 0.41 / 32768 * (P_BYTES + j.rows * TK * 2) * ceil(stages_of(j) / s); };
    return fmax(2 + rounds(time(j0), j0.tiles * s, b ? time(j1) : 0, j1.tiles * s, places, 1),
                6 + memory_us(a) + (b ? memory_us(*b) : 0));
}

cudaError_t launch_dense_split(const DenseArgs &a, const DenseArgs *b, cudaStream_t st) {
    switch (a.kind) {
        case DENSE_LINEAR: return launch<LINEAR>(a, nullptr, st);
        case DENSE_GATED: return launch<GATED>(a, nullptr, st);
        default: return launch<BACKWARD>(a, b, st);
    }
}

}  // namespace la
