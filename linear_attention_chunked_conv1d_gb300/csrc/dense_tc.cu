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
//
// A persistent, warp-specialised kernel; two blocks on neighbouring SMs form a pair (cta_group::2) that works on
// one 256 x 256 tile: each holds 128 rows of A and half of B, so that an operand byte in shared memory serves
// twice the multiply-adds of a single block's tile of 128 x 256.
//  - warp 0 streams its block's halves (2 x 16 KB a stage of 64 summed indexes) through a ring of six stages by
//    TMA; both blocks' copies complete on the leader's barrier;
//  - warp 1 of the leader issues tcgen05.mma (M = 256, N = 256, K = 16) into one of two accumulators; GATED takes
//    128 columns of each weight (one from each block), so that gate and up stand side by side in the accumulator;
//  - warps 2-9 turn the other accumulator into the result meanwhile, 32 rows x 64 columns at a time, laid out in
//    shared memory so that whole 128-byte lines go to memory.
// Tiles are walked in bands of sixteen rows of tiles; those of a round that would leave half the pairs without any are cut
// in halves of 128 columns (512 x 4096 x 4096: 24.5 -> 20.5 us, 1024 x 2048 x 2048: 15.9 -> 13.0). DX and DW of one backward pass are one launch, the tiles with
// the longer sums first: two launches would each leave SMs idle in their last round. A long sum of few tiles of DW is cut
// in parts, which go to the workspace in fp32 and are joined in their order.
// 8192 x 8192 x 2048 takes 146 us (1.88 PFLOP/s, tensor pipe 95% in the backward pass, 81% where an epilogue keeps z or gate
// and up); back to back, large products are held at 1.6 to 1.75 PFLOP/s by the power limit.
// Every wait is bounded; on a timeout the blocks raise LA_DEV_TIMEOUT, stop issuing, let what is under way end,
// free TMEM and return. Ragged edges come from TMA's zero fill; stores are guarded.
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

constexpr int TM = 256, TN = 256, TK = 64, STAGES = 6;  // a pair's tile; a block holds half of each operand
constexpr uint32_t HALF_BYTES = 128 * TK * 2, STAGE_BYTES = 2 * HALF_BYTES;
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t OFF_OUT = STAGES * STAGE_BYTES;             // a warp's 32 rows of 128 bytes, for each epilogue warp
constexpr uint32_t OFF_BAR = OFF_OUT + EPI_WARPS * 32 * 128;
constexpr size_t SMEM = OFF_BAR + 256 + 1024;  // barriers, alignment
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr uint32_t SLEEP_NS = 1000000u;
// Tiles of rows that are walked together (gated 16384 x 8192 x 4096: 2 1,410 us, 4 1,332, 8 1,290, 16 1,253, 24 1,264).
constexpr int BAND = 16;

enum { LINEAR = DENSE_LINEAR, GATED = DENSE_GATED, BACKWARD };

// One product of a launch (BACKWARD: up to two).
struct Job {
    int M, N, K, parts;
    bool dw;  // BACKWARD: DW, else DX
    int split;  // DW: parts of a long sum that are units of their own and are joined afterwards
    int64_t mt, nt, tiles;  // tiles: times parts
};

using bf16 = __nv_bfloat16;

// Tile `t` of an output of mt x nt tiles: bands of BAND tiles of rows, column by column, so that the tiles
// under way at one time share few rows and columns and find them in L2.
__device__ __forceinline__ void place_in_bands(int64_t t, int64_t mt, int64_t nt, int &m, int &n) {
    const int64_t band = t / (BAND * nt), r = t - band * BAND * nt;
    const int64_t high = mt - band * BAND < BAND ? mt - band * BAND : BAND;
    n = (int)(r / high);
    m = (int)(band * BAND + (r - n * high));
}

// What a pair works on at one time: a tile, or, of those from tile number `whole` on, half of its columns.
struct Unit {
    bool second;     // of the launch's second product
    int o, m, n;     // output (DW), place of the tile
    int part;        // of the sum
    bool cut;        // half a tile:
    int half;        // the first or the second
};
__device__ __forceinline__ Unit unit_at(int64_t u, int64_t whole, const Job &job0, const Job &job1) {
    Unit q;
    q.cut = u >= whole;
    q.half = q.cut ? (int)((u - whole) & 1) : 0;
    int64_t t = q.cut ? whole + ((u - whole) >> 1) : u;
    q.second = t >= job0.tiles;
    if (q.second) t -= job0.tiles;
    const Job &job = q.second ? job1 : job0;
    q.part = job.split > 1 ? (int)(t % job.split) : 0;
    if (job.split > 1) t /= job.split;
    const int64_t per = job.mt * job.nt;
    q.o = (int)(t / per);
    place_in_bands(t - q.o * per, job.mt, job.nt, q.m, q.n);
    return q;
}

// The stages of 64 summed indexes that a unit adds up (of each of DX's parts), from first to end.
__device__ __forceinline__ void stages_of(const Job &job, const Unit &unit, int &first, int &end) {
    const int64_t all = (job.K + TK - 1) / TK;
    first = (int)(all * unit.part / job.split);
    end = (int)(all * (unit.part + 1) / job.split);
}

// A warp's 32 x 64 values on their way to or from memory: row r's 16-byte piece j lies at place j ^ (r % 8) of its
// 128 bytes, so that neither a lane's own row nor eight lanes' pieces of one row meet in a bank.
__device__ __forceinline__ uint4 &piece(uint4 *buf, int r, int j) { return buf[r * 8 + (j ^ (r & 7))]; }
__device__ __forceinline__ uint4 pack8(const float *v) {
    uint4 p;
    Vec16<bf16>::store(reinterpret_cast<bf16 *>(&p), v);
    return p;
}
template <int V>
__device__ __forceinline__ void put(uint4 *buf, int r, int j, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) piece(buf, r, j + i) = pack8(v + 8 * i);
}
// Rows row0.. (up to M) and columns col.. (up to N) of a matrix from the buffer, in whole lines.
__device__ __forceinline__ void flush(uint4 *buf, bf16 *out, int64_t ld, int64_t row0, int M, int col, int N, int lane) {
    __syncwarp();
    const int j = lane & 7, c = col + j * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (row0 + r < M && c < N) {
            const uint4 v = piece(buf, r, j);
            bf16 *dst = out + (row0 + r) * ld + c;
            if (c + 8 <= N) {
                *reinterpret_cast<uint4 *>(dst) = v;
            } else {
                const bf16 *e = reinterpret_cast<const bf16 *>(&v);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < N) dst[k] = e[k];
            }
        }
    }
    __syncwarp();
}
// The same of a matrix of bytes, from each lane's row.
__device__ __forceinline__ void flush_bytes(uint2 *buf, const uint2 (&mine)[8], uint8_t *out, int64_t ld, int64_t row0, int M, int col, int N, int lane) {
#pragma unroll
    for (int j = 0; j < 8; ++j) buf[lane * 8 + (j ^ (lane & 7))] = mine[j];
    __syncwarp();
    const int j = lane & 7, c = col + j * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (row0 + r < M && c < N) *reinterpret_cast<uint2 *>(out + (row0 + r) * ld + c) = buf[r * 8 + (j ^ (r & 7))];
    }
    __syncwarp();
}
// Rows of 32 floats (whole pieces up to ld, which is a multiple of 8).
__device__ __forceinline__ void flush_floats(uint4 *buf, float *out, int64_t ld, int64_t row0, int M, int col, int lane) {
    __syncwarp();
    const int j = lane & 7, c = col + j * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (row0 + r < M && c < ld) *reinterpret_cast<uint4 *>(out + (row0 + r) * ld + c) = piece(buf, r, j);
    }
    __syncwarp();
}
// The same of an input, first into registers (what lies outside stays as it is), then into the buffer.
__device__ __forceinline__ void fetch(uint4 (&raw)[8], const bf16 *in, int64_t ld, int64_t row0, int M, int col, int N, int lane) {
    const int c = col + (lane & 7) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (row0 + r < M && c < N) {
            const bf16 *src = in + (row0 + r) * ld + c;
            if (c + 8 <= N) {
                raw[i] = *reinterpret_cast<const uint4 *>(src);
            } else {
                bf16 e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = c + k < N ? src[k] : __float2bfloat16_rn(0.f);
                memcpy(&raw[i], e, 16);
            }
        }
    }
}

// The bias of 32 of the warp's columns, from c on, onto v: lane l has those of columns 4 l .. 4 l + 3.
__device__ __forceinline__ void add_bias(float (&v)[32], const uint2 &bias, int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __shfl_sync(0xffffffffu, bias.x, c / 4 + i), b = __shfl_sync(0xffffffffu, bias.y, c / 4 + i);
        v[4 * i] += __uint_as_float(a << 16);
        v[4 * i + 1] += __uint_as_float(a & 0xFFFF0000u);
        v[4 * i + 2] += __uint_as_float(b << 16);
        v[4 * i + 3] += __uint_as_float(b & 0xFFFF0000u);
    }
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1)
dense_kernel(const __grid_constant__ Maps maps0, const __grid_constant__ Maps maps1, const __grid_constant__ Epilogue ep0,
             const __grid_constant__ Epilogue ep1, const __grid_constant__ Job job0, const __grid_constant__ Job job1,
             int64_t whole, int64_t units, int beside, int *status, uint64_t wait_ns, int debug_stall) {
    constexpr int OUT_N = KIND == GATED ? TN / 2 : TN;  // columns of the result a tile holds
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
    if (beside) wait_and_let_beside();  // the call's other kernel, beside this one's last round
    else wait_for_previous();
    const uint32_t tm = *tmem_sh;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
    // Every round but the first goes to the pairs from the last to the first: where the first pairs had the longer sums,
    // the last ones have an incomplete round's.
    auto later = [&](int64_t round) { return round * step + (step - 1 - first); };
    const uint32_t sbase = tc::smem_u32(sm);

    if (warp == 0) {
        if (tc::elect_one()) {
            uint32_t s = 0, ph = 0, used = 0;
            for (int64_t u = first, round = 0; u < units && !*err; u = later(++round)) {
                const Unit unit = unit_at(u, whole, job0, job1);
                const Job &job = KIND == BACKWARD && unit.second ? job1 : job0;
                const Maps &maps = KIND == BACKWARD && unit.second ? maps1 : maps0;
                const int m0 = unit.m * TM + (int)rank * 128, share = unit.cut ? 64 : 128;  // rows of B in a block
                const int n0 = unit.n * OUT_N + unit.half * (OUT_N / 2) + (KIND == GATED ? 0 : (int)rank * share);
                const uint32_t bytes = 2 * (HALF_BYTES + share * TK * 2);
                const CUtensorMap *ma = &maps.a[KIND == BACKWARD && job.dw ? unit.o : 0], *mb = &maps.b[KIND == GATED ? rank : 0];
                int k_first, k_end;
                stages_of(job, unit, k_first, k_end);
                for (int p = 0; p < job.parts && !*err; ++p) {
                    if (KIND == BACKWARD && p) {
                        ma = &maps.a[1];
                        mb = &maps.b[1];
                    }
                    int k0 = k_first * TK;
                    for (int k = k_first; k < k_end; ++k, k0 += TK) {
                        if (!tc::mbar_wait(empty + s, ph ^ 1u, wait_ns, SLEEP_NS) || *err) {
                            *err = 1;
                            break;
                        }
                        const uint32_t da = sbase + s * STAGE_BYTES, db = da + HALF_BYTES;
                        const uint32_t bar = tc::map_to_rank(tc::smem_u32(full + s), 0);
                        if (rank == 0) tc::mbar_expect_tx(full + s, bytes);
                        if (KIND == BACKWARD && job.dw) {
                            tc::tma_load_2d_pair(da, ma, m0, k0, bar);
                            tc::tma_load_2d_pair(da + HALF_BYTES / 2, ma, m0 + 64, k0, bar);
                        } else {
                            tc::tma_load_2d_pair(da, ma, k0, m0, bar);
                        }
                        for (int i = 0; i < share; i += 64)
                            tc::tma_load_2d_pair(db + i * TK * 2, mb, KIND == BACKWARD ? n0 + i : k0, KIND == BACKWARD ? k0 : n0 + i, bar);
                        used |= 1u << s;
                        if (++s == STAGES) s = 0, ph ^= 1u;
                    }
                }
            }
            // Before the blocks exit, each waits until the MMAs have read its last copies: they have landed then, and the
            // leader's arrivals have reached the other block's barriers. Where something went wrong the two may have
            // stopped at different stages; a copy takes microseconds, so each then gives its last ones a millisecond.
            if (*err) {
                const uint64_t t0 = tc::globaltimer_ns();
                while (tc::globaltimer_ns() - t0 < 1000000u) __nanosleep(1000);
            } else {
                for (uint32_t i = 0; i < STAGES; ++i)  // stages before s were last filled in phase ph, the others in the one before
                    if ((used >> i & 1u) && !tc::mbar_wait(empty + i, i < s ? ph : ph ^ 1u, wait_ns, SLEEP_NS)) *err = 1;
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && tc::elect_one()) {
            uint32_t s = 0, ph = 0, tcnt = 0;
            if (debug_stall && !tc::mbar_wait(fin, 0, wait_ns, SLEEP_NS)) *err = 1;
            for (int64_t u = first; u < units && !*err; u = later(++tcnt)) {
                const Unit unit = unit_at(u, whole, job0, job1);
                const Job &job = KIND == BACKWARD && unit.second ? job1 : job0;
                const bool a_mn = KIND == BACKWARD && job.dw;
                constexpr bool b_mn = KIND == BACKWARD;
                const uint32_t id = tc::idesc(TM, unit.cut ? TN / 2 : TN, tc::FMT_BF16, a_mn, b_mn);
                int k_first, k_end;
                stages_of(job, unit, k_first, k_end);
                const int64_t kb = (int64_t)(k_end - k_first) * job.parts;
                const uint32_t acc = tcnt & 1u, aph = (tcnt >> 1) & 1u;
                if (!tc::mbar_wait(acce + acc, aph ^ 1u, wait_ns, SLEEP_NS)) {
                    *err = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t d = tm + acc * TN;
                bool ok = true;
                for (int64_t k = 0; k < kb; ++k) {
                    if (!tc::mbar_wait(full + s, ph, wait_ns, SLEEP_NS) || *err) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t a = sbase + s * STAGE_BYTES, b = a + HALF_BYTES;
#pragma unroll
                    for (uint32_t kk = 0; kk < TK / 16; ++kk)
                        tc::mma_bf16_ss_pair(
                            d, a_mn ? tc::sdesc_sw128_mn(a + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(a + kk * 32u),
                            b_mn ? tc::sdesc_sw128_mn(b + kk * 2048u, 8192u, 1024u) : tc::sdesc_sw128(b + kk * 32u), id,
                            (k | kk) != 0);
                    tc::mma_commit_pair(empty + s, 3);
                    if (++s == STAGES) s = 0, ph ^= 1u;
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
        uint4 *buf = reinterpret_cast<uint4 *>(sm + OFF_OUT) + (warp - 2) * 256;
        uint32_t tcnt = 0;
        for (int64_t u = first; u < units; u = later(++tcnt)) {
            // every decision to stop is made per warp: the TMEM loads below are warp-collective
            if (__any_sync(0xffffffffu, *err != 0)) break;
            const Unit unit = unit_at(u, whole, job0, job1);
            const Job &job = KIND == BACKWARD && unit.second ? job1 : job0;
            const Epilogue &ep = KIND == BACKWARD && unit.second ? ep1 : ep0;
            // A warp has 128 columns of a tile (half a tile, GATED: 64); of half a GATED tile the first four warps have all.
            const int wide = unit.cut ? OUT_N / 2 : OUT_N, cols = wide / 2 < 64 ? (warp < 6 ? 64 : 0) : wide / 2;
            const int c_first = (warp - 2) / 4 * (wide / 2), up_at = unit.cut ? TN / 4 : TN / 2;
            const int M = job.M, N = job.N, o = unit.o, n0 = unit.n * OUT_N + unit.half * (OUT_N / 2) + c_first;
            const int64_t row0 = (int64_t)unit.m * TM + rank * 128 + 32 * q;
            uint4 res[8];  // the residual's next 64 columns
            uint2 bias = make_uint2(0u, 0u);  // the bias of columns 4 lane .. 4 lane + 3 of the warp's
            if (KIND == LINEAR && ep.residual) fetch(res, ep.residual, ep.ldr, row0, M, n0, N, lane);
            if (KIND == LINEAR && ep.bias) {
                const int c = n0 + lane * 4;
                if (c + 4 <= N) {
                    bias = *reinterpret_cast<const uint2 *>(ep.bias + c);
                } else if (c < N) {
                    bf16 e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = c + k < N ? ep.bias[c + k] : __float2bfloat16_rn(0.f);
                    memcpy(&bias, e, 8);
                }
            }
            const uint32_t acc = tcnt & 1u, aph = (tcnt >> 1) & 1u;
            const uint64_t acc_ns = wait_ns + (uint64_t)((job.K + TK - 1) / TK) * job.parts * 1000;  // as long as the sum is
            if (!__all_sync(0xffffffffu, tc::mbar_wait(accf + acc, aph, acc_ns, SLEEP_NS))) {
                *err = 1;
                break;
            }
            tc::fence_after_sync();
            const uint32_t src = tc::tmem_addr(tm + acc * TN, 32 * q, c_first);
            if (KIND == BACKWARD && job.split > 1) {  // a part of the sum, in fp32
                float *part = ep.partial + ((int64_t)o * job.split + unit.part) * M * ep.ldp;
#pragma unroll 1
                for (int c = 0; c < cols; c += 32) {
                    float v[32];
                    tc::tmem_ld16(src + c, v);
                    tc::tmem_ld16(src + c + 16, v + 16);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        piece(buf, lane, j) = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                                         __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
                    flush_floats(buf, part, ep.ldp, row0, M, n0 + c, lane);
                }
            }
#pragma unroll 1
            for (int c = KIND == BACKWARD && job.split > 1 ? cols : 0; c < cols; c += 64) {
                const int col = n0 + c;
                if (KIND == LINEAR) {
                    if (ep.saved) {  // z goes out first, y is made of it in a second look at the accumulator
#pragma unroll 1
                        for (int j = 0; j < 8; j += 4) {
                            float v[32];
                            tc::tmem_ld16(src + c + j * 8, v);
                            tc::tmem_ld16(src + c + j * 8 + 16, v + 16);
                            tc::tmem_wait_ld();
                            if (ep.bias) add_bias(v, bias, c + j * 8);
                            put(buf, lane, j, v);
                        }
                        flush(buf, ep.saved, ep.lds, row0, M, col, N, lane);
                    }
                    if (ep.residual) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) piece(buf, i * 4 + (lane >> 3), lane & 7) = res[i];
                        if (c + 64 < cols) fetch(res, ep.residual, ep.ldr, row0, M, col + 64, N, lane);
                        __syncwarp();
                    }
#pragma unroll 1
                    for (int j = 0; j < 8; j += 4) {
                        float v[32];
                        tc::tmem_ld16(src + c + j * 8, v);
                        tc::tmem_ld16(src + c + j * 8 + 16, v + 16);
                        tc::tmem_wait_ld();
                        if (ep.bias) add_bias(v, bias, c + j * 8);
                        act_values(v, ep.act);
                        if (ep.residual) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float u[8];
                                Vec16<bf16>::load(reinterpret_cast<bf16 *>(&piece(buf, lane, j + i)), u);
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[8 * i + e] += u[e];
                            }
                        }
                        put(buf, lane, j, v);
                    }
                } else if (KIND == GATED) {
                    if (ep.saved) {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            uint2 lower[8];
#pragma unroll
                            for (int j = 0; j < 8; j += 4) {
                                float v[32];
                                tc::tmem_ld16(src + half * up_at + j * 8, v);
                                tc::tmem_ld16(src + half * up_at + j * 8 + 16, v + 16);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    piece(buf, lane, j + i) = upper8(v + 8 * i);
                                    lower[j + i] = lower8(v + 8 * i);
                                }
                            }
                            flush(buf, ep.saved + half * ep.half, ep.lds, row0, M, col, N, lane);
                            flush_bytes(reinterpret_cast<uint2 *>(buf), lower, ep.lower + half * ep.half, ep.lds, row0, M, col, N, lane);
                        }
                    }
#pragma unroll 1
                    for (int j = 0; j < 8; j += 2) {
                        float v[16], u[16];
                        tc::tmem_ld16(src + j * 8, v);
                        tc::tmem_ld16(src + up_at + j * 8, u);
                        tc::tmem_wait_ld();
                        act_values(v, ep.act);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= u[e];
                        put(buf, lane, j, v);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        float v[32];
                        tc::tmem_ld16(src + c + j * 8, v);
                        tc::tmem_ld16(src + c + j * 8 + 16, v + 16);
                        tc::tmem_wait_ld();
                        put(buf, lane, j, v);
                    }
                }
                flush(buf, ep.out[o], ep.ldo[o], row0, M, col, N, lane);
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

// dW from the parts of its sum, [split][M][ldp] fp32, added up in their order.
__global__ void __launch_bounds__(256)
dense_join_kernel(const float *__restrict__ partial, bf16 *__restrict__ out, int M, int N, int split, int64_t ldp, int64_t ldo) {
    wait_for_previous();
    const int c = (blockIdx.x * 32 + threadIdx.x) * 8;
    if (c >= N) return;
    for (int64_t r = blockIdx.y * 8 + threadIdx.y; r < M; r += (int64_t)gridDim.y * 8) {
        float v[8] = {};
#pragma unroll 4
        for (int s = 0; s < split; ++s) {
            const float *p = partial + ((int64_t)s * M + r) * ldp + c;
            float t[8];
            Vec16<float>::load(p, t);
            Vec16<float>::load(p + 4, t + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        store_piece(out + r * ldo, c, N, v);
    }
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

Job make_job(const DenseArgs &a) {
    const int out_n = a.kind == DENSE_GATED ? TN / 2 : TN;
    Job j{a.M, a.N, a.K, a.kind == DENSE_DX ? a.count : 1, a.kind == DENSE_DW, a.split > 1 ? a.split : 1, 0, 0, 0};
    j.mt = (a.M + TM - 1) / TM;
    j.nt = (a.N + out_n - 1) / out_n;
    j.tiles = j.mt * j.nt * (a.kind == DENSE_DW ? a.count : 1) * j.split;
    return j;
}

// One product, or (BACKWARD) two.
template <int KIND>
cudaError_t launch(const DenseArgs &a, const DenseArgs *b, cudaStream_t st) {
    Maps maps[2];
    const bool mn = KIND == BACKWARD;
    if (!make_maps(&maps[0], a, a.kind == DENSE_DW, mn, 128, 64)) return cudaErrorInvalidValue;
    if (b && !make_maps(&maps[1], *b, b->kind == DENSE_DW, mn, 128, 64)) return cudaErrorInvalidValue;
    const Job j0 = make_job(a), j1 = b ? make_job(*b) : Job{0, 0, 0, 1, false, 1, 0, 0, 0};
    // the tiles of an incomplete round are cut in halves where there are pairs for them
    const int64_t tiles = j0.tiles + j1.tiles, pairs = resident_pairs<KIND>(), rest = tiles % pairs;
    const int64_t whole = 2 * rest <= pairs ? tiles - rest : tiles, units = whole + 2 * (tiles - whole);
    const cudaError_t e = launch_overlapped(
        dense_kernel<KIND>, dim3(2 * (int)(units < pairs ? units : pairs)), dim3(THREADS), SMEM, 2, st, maps[0], b ? maps[1] : maps[0],
        make_epilogue(a), make_epilogue(b ? *b : a), j0, j1, whole, units, a.beside, a.status, a.wait_ns ? a.wait_ns : WAIT_NS,
        a.debug_stall);
    const DenseArgs &w = b && b->split > 1 ? *b : a;
    if (e != cudaSuccess || w.split <= 1) return e;
    const Epilogue ep = make_epilogue(w);
    const int cols = (w.N + 255) / 256, runs = (w.M + 7) / 8, most = SMS * 6 / cols < 1 ? 1 : SMS * 6 / cols;
    for (int o = 0; o < w.count; ++o) {
        const cudaError_t j = launch_overlapped(dense_join_kernel, dim3(cols, runs < most ? runs : most), dim3(32, 8), 0, 0, st,
                                                (const float *)(ep.partial + (int64_t)o * w.split * w.M * ep.ldp), ep.out[o], w.M, w.N,
                                                w.split, ep.ldp, ep.ldo[o]);
        if (j != cudaSuccess) return j;
    }
    return cudaSuccess;
}

}  // namespace

namespace {

cudaError_t launch_pairs(const DenseArgs &a, cudaStream_t st) {
    switch (a.kind) {
        case DENSE_LINEAR: return launch<LINEAR>(a, nullptr, st);
        case DENSE_GATED: return launch<GATED>(a, nullptr, st);
        default: return launch<BACKWARD>(a, nullptr, st);
    }
}

// A call's rows from `row` on.
DenseArgs rows_from(const DenseArgs &a, int row) {
    DenseArgs r = a;
    auto on = [&](const void *p, int64_t ld, int size) { return p ? static_cast<const char *>(p) + row * ld * size : nullptr; };
    for (int i = 0; i < 2; ++i) r.a[i] = on(a.a[i], a.lda[i], 2);
    r.out[0] = const_cast<char *>(on(a.out[0], a.ldo[0], 2));
    r.residual = on(a.residual, a.ldr, 2);
    r.saved = const_cast<char *>(on(a.saved, a.lds, 2));
    r.lower = const_cast<char *>(on(a.lower, a.lds, 1));
    r.M = a.M - row;
    return r;
}

}  // namespace

// Parts of dW's long sum. Few tiles of many rows' sums (16384 rows, 1024 x 1024: 16 tiles of 256 stages) would keep few
// pairs busy; parts of them are units of their own, as many as make the model's time the least. (dx and dw of 16384 rows,
// 1024 x 1024: 64.4 us in one part, 52.6 so; 8192 rows, 1000 x 1000: 55.9 and 42.8; dw of 65,536 rows: 115.9 and 83.4.)
namespace {

int choose_dw_split(const DenseArgs &dw, const DenseArgs *dx) {
    DenseArgs q = dw;
    q.split = 1;
    double best = dense_pairs_us(q, dx) - 2;  // worth a second launch
    int s = 1;
    for (int k = 2; k <= 8; ++k) {
        q.split = k;
        if ((q.K + TK - 1) / TK < 8 * k) break;
        const double t = dense_pairs_us(q, dx);
        if (t < best) best = t, s = k;
    }
    return s;
}

}  // namespace

size_t dense_dw_partial_bytes(int rows, int M, int N, int count) {
    DenseArgs dw{}, dx{};
    dw.kind = DENSE_DW; dw.count = count; dw.M = M; dw.N = N; dw.K = rows;
    dx.kind = DENSE_DX; dx.count = count; dx.M = rows; dx.N = N; dx.K = M;
    const int with = choose_dw_split(dw, &dx), alone = choose_dw_split(dw, nullptr), s = with > alone ? with : alone;
    return s > 1 ? (size_t)count * s * M * (((size_t)N + 7) / 8 * 8) * sizeof(float) : 0;
}

cudaError_t launch_dense(const DenseArgs &args, cudaStream_t st) {
    DenseArgs a = args;
    a.split = a.kind == DENSE_DW && a.partial ? choose_dw_split(a, nullptr) : 1;
    const double pairs = dense_pairs_us(a, nullptr), split = dense_split_us(a, nullptr);
    // A few rows past whole tiles would take tiles of their own, and with them part of another round. Where the whole
    // tiles leave pairs without work, the other kernel takes those rows there, beside this one's last round. (777 x 5001 x
    // 2048: 60 tiles on 76 pairs and 9 rows, 22.3 us in 80 tiles, 17.7 so; with bias, GELU and residual 27.0 and 22.2;
    // 1030 x 8192 x 2048: 31.8 and 27.5; where little is to be gained it may be lost: 1040 x 2048 x 2048 16.0 and 19.5.)
    const int rest = a.M % TM;
    if (a.kind != DENSE_DW && a.M > TM && rest && rest <= 64) {
        DenseArgs main = a, other = rows_from(a, a.M - rest);
        main.M = a.M - rest;
        const int64_t last = make_job(main).tiles % PAIRS, idle = last ? PAIRS - (2 * last <= PAIRS ? 2 * last : last) : 0;
        other.places = (int)idle * 4;
        // the other kernel starts some 4 us after this one
        if (idle >= 8 && fmax(dense_pairs_us(main, nullptr) + 1.5, 4 + dense_split_us(other, nullptr)) + 2 < fmin(pairs, split)) {
            main.beside = 1;
            other.beside = 2;
            const cudaError_t e = launch_pairs(main, st);
            return e != cudaSuccess ? e : launch_dense_split(other, nullptr, st);
        }
    }
    return split < pairs ? launch_dense_split(a, nullptr, st) : launch_pairs(a, st);
}

cudaError_t launch_dense_pair(const DenseArgs &dx, const DenseArgs &dw_args, cudaStream_t st) {
    DenseArgs dw = dw_args, alone = dw_args;
    dw.split = dw.partial ? choose_dw_split(dw, &dx) : 1;
    alone.split = dw.partial ? choose_dw_split(dw, nullptr) : 1;
    const double pairs = dense_pairs_us(dw, &dx), split = dense_split_us(dx, &dw);
    const double apart = fmin(dense_pairs_us(dx, nullptr), dense_split_us(dx, nullptr)) + fmin(dense_pairs_us(alone, nullptr), dense_split_us(dw, nullptr));
    if (apart < fmin(pairs, split)) {
        const cudaError_t e = launch_dense(dx, st);
        return e != cudaSuccess ? e : launch_dense(dw_args, st);
    }
    const bool by_split = split < pairs;
    if (by_split) dw.split = 1;
    const bool dx_first = (int64_t)dx.K * dx.count * dw.split >= dw.K;  // the longer sums first
    const DenseArgs &a = dx_first ? dx : dw, &b = dx_first ? dw : dx;
    return by_split ? launch_dense_split(a, &b, st) : launch<BACKWARD>(a, &b, st);
}

}  // namespace la
