// Products of a few rows with 4-bit weights that have a scale for each group of inputs:
//   y[m][n] = sum_k x[m][k] W[n][k],  W[n][k] = scales[n][k / group] (q(n, k) - 8),  q in 0..15.
// The projections of "split_prefill.rs", prefill_phase1_proj_batched, when a layer decodes a few
// tokens: reading the weights is all the time there is, and these take a quarter of bf16's.
//
// Layout of q [N][K / 2] bytes: eight weights of a row to a little-endian 32-bit word, weight 2i in
// bits 4i .. 4i+3 and weight 2i + 1 in bits 16+4i .. 16+4i+3, so that one shift and one mask give a
// pair (2i, 2i + 1) in the two halves of a word.
#include "common.cuh"
#include "launch.h"
#include "overlap.cuh"

namespace la {

namespace {

// Eight weights of one thread: the group's largest magnitude over its lanes, the scale max / 7
// rounded to bf16, and the nearest multiples of that scale (ties to even).
__global__ void w4_quantize_kernel(const W4QuantArgs a, int64_t words) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int per_row = a.K / 8, lanes = a.group / 8;  // 4, 8 or 16 lanes have one group
    const bool active = i < words;                     // whole groups: words is a multiple of lanes
    const int64_t n = active ? i / per_row : 0;
    const int k8 = active ? (int)(i % per_row) : 0;
    float v[8] = {};
    if (active) Vec16<__nv_bfloat16>::load((const __nv_bfloat16 *)a.w + n * a.ldw + k8 * 8, v);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
    for (int off = lanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const __nv_bfloat16 scale = __float2bfloat16_rn(__fdiv_rn(top, 7.f));
    const float sc = to_f(scale);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int q = sc > 0.f ? __float2int_rn(fminf(fmaxf(__fdiv_rn(v[e], sc), -8.f), 7.f)) : 0;
        word |= (uint32_t)(q + 8) << (4 * (e / 2) + 16 * (e % 2));
    }
    if (!active) return;
    ((uint32_t *)a.q)[i] = word;
    if (k8 % lanes == 0) ((__nv_bfloat16 *)a.scales)[n * (a.K / a.group) + k8 / lanes] = scale;
}

// The products: a tile of 128 outputs over a share of the inputs that the blocks of a cluster split.
// 256 inputs at a time go through a ring of asynchronous copies: the tile's weights (16 KB), the rows'
// inputs, laid out so that a lane finds its part of an operand in 16 bytes, and the scales. A warp has
// 32 of the outputs and 128 of the inputs. Weights are the A operand of mma.m16n8k16, 16 outputs by 16
// inputs, as exact bf16 numbers; the rows are B. A lane's word of eight weights serves two mma: which
// inputs meet in one mma is free as long as A and B agree, so word c of 32 inputs goes to the lanes
// with c = lane % 4 as it lies in memory. Products are exact in fp32; a group's sum is scaled by its
// output's scale and added to the others in fp32. In the end every block of the cluster gets the parts of
// its share of the outputs and adds them in a fixed order. (Each warp's sums by themselves, 4 bytes a store,
// took 1.4 us longer at 32 x 16384 x 8192, 3 us at 32 x 4096 x 8192.)
// Measured on the device: 1 x 8192 x 2048 4.3 us (3.2 of it without the products: the launch, one trip to
// HBM, two cluster barriers); 1 x 16384 x 8192 20.1 us, 3.5 TB/s (loads alone 13.7, products alone 14.0: with
// 16 warps on an SM neither hides the other), 32 rows 38 us (21 and 30).
constexpr int kThreads = 256;
constexpr int kTile = 128;           // outputs of a block: four warps of 32
constexpr int kMaxBlocks = 8;        // of a cluster
constexpr int kParts = kTile + kMaxBlocks;  // places for the parts: a share is rounded up
constexpr int kSeg = 256;            // inputs of a stage: two warps of 128
constexpr int kRowBytes = 128 + 16;  // a row's weights of a stage, padded: 8 rows x 4 lanes on 32 banks

// Words that hold an output's scales of a stage: they may start in the middle of one.
template <int G> constexpr int kScaleWords = kSeg / G / 2 + 1;
// A stage: weights, inputs, scales.
template <int NT> constexpr int kInputsAt = kTile * kRowBytes;
template <int NT> constexpr int kScalesAt = kInputsAt<NT> + NT * 8 * kSeg * 2;
template <int NT, int G> constexpr int kStageBytes = kScalesAt<NT> + kTile * kScaleWords<G> * 4;
template <int NT> constexpr int kStages = NT == 1 ? 4 : 3;  // two blocks on an SM

__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same, onto zeros.
__device__ __forceinline__ void mma_bf16_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Pairs of weights (2i, 2i + 1) of a word as bf16, times 2^-6. A nibble in the low half of a bf16 pattern
// is a subnormal (bit 7 is the exponent's last, and the least normal numbers go on in the subnormals'
// steps): q 2^-133 in bits 0-3, q 2^-129 in bits 4-7. One multiply-add makes (q - 8) 2^-6 of either,
// exactly; the sums take the 2^6.
__device__ __forceinline__ uint32_t to_weight(uint32_t v, uint32_t mul) {
    const uint32_t minus = 0xbe00be00u;  // -8 2^-6
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(mul), "r"(minus));
    return r;
}
__device__ __forceinline__ void weights_of(uint32_t word, uint32_t (&v)[4]) {
    constexpr uint32_t lo = 0x7f007f00u, hi = 0x7d007d00u;  // 2^127, 2^123
    const uint32_t up = word >> 8;
    v[0] = to_weight(word & 0x000f000fu, lo);
    v[1] = to_weight(word & 0x00f000f0u, hi);
    v[2] = to_weight(up & 0x000f000fu, lo);
    v[3] = to_weight(up & 0x00f000f0u, hi);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int NT, int G>  // 8 NT rows at most, groups of G inputs
__global__ void __launch_bounds__(kThreads, 2) w4_matvec_kernel(const W4Args a, int segs_each) {
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int t = threadIdx.x, warp = t / 32, lane = t % 32, g = lane / 4, c = lane % 4;
    const int rows_at = warp % 4 * 32, half = warp / 4;
    uint32_t rank, blocks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    const int n0 = blockIdx.x / blocks * kTile;
    const int all = (a.K + kSeg - 1) / kSeg;
    const int first = (int)rank * segs_each, last = min(first + segs_each, all);

    // this thread's copies of a stage: 16 bytes of weights of rows t / 8, + 32, + 64, + 96 (past the last
    // output the last one's: nobody looks at what becomes of them) ..
    int left = a.K - first * kSeg;  // inputs from the stage's first one on
    const unsigned char *qp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        qp[i] = static_cast<const unsigned char *>(a.q) + (int64_t)min(n0 + t / 8 + i * 32, a.N - 1) * (a.K / 2) +
                (first * kSeg + t % 8 * 32) / 2;
    const uint32_t q_to = t / 8 * kRowBytes + t % 8 * 16;
    // .. and of inputs: 8 of them of row t / 32, + 8, .. (rows past the last one stay what they are) ..
    const __nv_bfloat16 *xp = static_cast<const __nv_bfloat16 *>(a.x) + (int64_t)warp * a.ldx + first * kSeg + lane * 8;
    const uint32_t x_to = kInputsAt<NT> + (lane / 4 * 32 + warp * 4 + lane % 4) * 16;
    // .. and of scales, a word at a time
    constexpr int kWords = kScaleWords<G>;
    constexpr int kScaleCopies = (kTile * kWords + kThreads - 1) / kThreads;
    const int per_row = a.K / G;
    const __nv_bfloat16 *sp[kScaleCopies];
    const __nv_bfloat16 *const sp_end = static_cast<const __nv_bfloat16 *>(a.scales) + (int64_t)a.N * per_row;
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i) {
        const int w = t + i * kThreads;
        sp[i] = static_cast<const __nv_bfloat16 *>(a.scales) +
                (((int64_t)(n0 + w / kWords) * per_row + first * (kSeg / G)) & ~int64_t(1)) + w % kWords * 2;
    }
    uint32_t at = sbase;
    const auto fetch = [&](int seg) {
        if (seg < last) {
            // Only a row's last stage may end inside: what lies past K is zeros. (Of the inputs: a weight is
            // finite whatever its bits are.)
            const bool q_there = t % 8 * 32 < left, x_there = lane * 8 < left;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                copy16(at + q_to + i * 32 * kRowBytes, q_there ? qp[i] : a.q, q_there);
                qp[i] += kSeg / 2;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (warp + n * 8 < a.M) copy16(at + x_to + n * 8 * kSeg * 2, x_there ? xp + n * 8 * a.ldx : a.x, x_there);
            xp += kSeg;
#pragma unroll
            for (int i = 0; i < kScaleCopies; ++i) {
                if (kTile * kWords % kThreads && t + i * kThreads >= kTile * kWords) break;
                // an odd last one is half a word
                copy4(at + kScalesAt<NT> + (t + i * kThreads) * 4, sp[i] < sp_end ? sp[i] : a.scales,
                      sp[i] + 1 < sp_end ? 4 : sp[i] < sp_end ? 2 : 0);
                sp[i] += kSeg / G;
            }
            left -= kSeg;
            at = at == sbase + (kStages<NT> - 1) * kStageBytes<NT, G> ? sbase : at + kStageBytes<NT, G>;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // where a stage has the scales of this lane's four outputs
    constexpr int kGroups = 128 / G;
    int scale_at[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = rows_at + g + 8 * r;
        scale_at[r] = row * kWords * 2 + (int)((int64_t)(n0 + row) * per_row & 1) + half * kGroups;
    }

    float acc[2][NT][4] = {};
    wait_for_previous();
#pragma unroll
    for (int s = 0; s < kStages<NT> - 1; ++s) fetch(first + s);
    const unsigned char *st = smem;
    for (int seg = first; seg < last; ++seg) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages<NT> - 2) : "memory");
        __syncthreads();  // this stage is here, and the one before it read by all
        fetch(seg + kStages<NT> - 1);
        const uint32_t *w = reinterpret_cast<const uint32_t *>(st + (rows_at + g) * kRowBytes + half * 64) + c;
        const uint4 *xs = reinterpret_cast<const uint4 *>(st + kInputsAt<NT>) + half * 4 * 32 + lane;
        // Inputs past K are zeros, but their scales are the next output's or nobody's.
        const __nv_bfloat16 *sc = reinterpret_cast<const __nv_bfloat16 *>(st + kScalesAt<NT>);
        const int groups_left = per_row - seg * (kSeg / G) - half * kGroups;
        float part[2][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t A[2][2][4];  // [16 outputs][8 of 32 inputs' pairs]
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t u[4], v[4];
                weights_of(w[r * 16 * (kRowBytes / 4) + j * 4], u);
                weights_of(w[(r * 16 + 8) * (kRowBytes / 4) + j * 4], v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    A[r][h][0] = u[2 * h];
                    A[r][h][1] = v[2 * h];
                    A[r][h][2] = u[2 * h + 1];
                    A[r][h][3] = v[2 * h + 1];
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 b = xs[n * (kSeg / 32 * 32) + j * 32];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (j * 32 % G == 0) mma_bf16_0(part[r][n], A[r][0], b.x, b.y);
                    else mma_bf16(part[r][n], A[r][0], b.x, b.y);
                    mma_bf16(part[r][n], A[r][1], b.z, b.w);
                }
            }
            if ((j + 1) * 32 % G == 0) {
                const int i = j * 32 / G;
                float s[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = i < groups_left ? to_f(sc[scale_at[r] + i]) : 0.f;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][n][e] = fmaf(s[2 * r + e / 2], part[r][n][e], acc[r][n][e]);
            }
        }
        st = st == smem + (kStages<NT> - 1) * kStageBytes<NT, G> ? smem : st + kStageBytes<NT, G>;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // The ring is free. The warps with the second half of a stage's inputs hand their sums to those with the
    // first, these theirs to the block whose share the output is in, 8 bytes a store.
    __syncthreads();
    cluster_arrive();
    constexpr int kPitch = NT * 8 + 2;  // of an output's rows
    float *parts = reinterpret_cast<float *>(smem), *hand = parts + kParts * kPitch + t % 128;
    if (half)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) hand[((r * NT + n) * 4 + e) * 128] = acc[r][n][e];
    __syncthreads();
    cluster_wait();  // every block's ring is
    const int share = (kTile + (int)blocks - 1) / (int)blocks;
    if (!half)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int out = rows_at + r * 16 + g + e / 2 * 8;
                uint32_t to;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(sbase), "r"(out / share));
                to += (((int)rank * share + out % share) * kPitch + 2 * c) * 4;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float *other = hand + ((r * NT + n) * 4 + e) * 128;
                    if (n * 8 + 2 * c < a.M)
                        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + n * 32),
                                     "f"((acc[r][n][e] + other[0]) * 64.f), "f"((acc[r][n][e + 1] + other[128]) * 64.f) : "memory");
                }
            }
    cluster_arrive();
    cluster_wait();
    for (int i = t; i < a.M * share; i += kThreads) {
        const int m = i / share, out = i % share, n = n0 + (int)rank * share + out;
        float v = 0.f;
        for (uint32_t b = 0; b < blocks; ++b) v += parts[((int)b * share + out) * kPitch + m];
        if (n < a.N && (int)rank * share + out < kTile) static_cast<__nv_bfloat16 *>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(v);
    }
}

// Blocks that share a tile's inputs: as few as make their shares as short as they can be while each still
// has two stages and all fit on 152 SMs, two on each less a tenth for clusters that do not fill a group of
// SMs. By N and K alone, and a fixed number of SMs: a row's sums do not depend on the batch or the device.
int cluster_of(int N, int K) {
    const int tiles = (N + kTile - 1) / kTile, segs = (K + kSeg - 1) / kSeg;
    int most = 272 / tiles;
    most = most < 1 ? 1 : most > kMaxBlocks ? kMaxBlocks : most;
    int each = (segs + most - 1) / most;
    each = each < 2 ? 2 : each;
    return (segs + each - 1) / each;
}

template <int NT, int G> cudaError_t launch_t(const W4Args &a, cudaStream_t st) {
    constexpr int smem = kStages<NT> * kStageBytes<NT, G>;
    static_assert(smem >= kParts * (NT * 8 + 2) * 4 + 128 * NT * 8 * 4, "what is handed on takes the ring's place");
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two blocks on an SM");
    cudaError_t e = cudaFuncSetAttribute(w4_matvec_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int blocks = cluster_of(a.N, a.K), segs = (a.K + kSeg - 1) / kSeg;
    return launch_overlapped(w4_matvec_kernel<NT, G>, dim3((a.N + kTile - 1) / kTile * blocks), dim3(kThreads), smem, blocks, st, a,
                             (segs + blocks - 1) / blocks);
}
template <int NT> cudaError_t launch_g(const W4Args &a, cudaStream_t st) {
    return a.group == 32 ? launch_t<NT, 32>(a, st) : a.group == 64 ? launch_t<NT, 64>(a, st) : launch_t<NT, 128>(a, st);
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Args &a, cudaStream_t st) {
    return a.M <= 8 ? launch_g<1>(a, st) : a.M <= 16 ? launch_g<2>(a, st) : launch_g<4>(a, st);
}

cudaError_t launch_w4_quantize(const W4QuantArgs &a, cudaStream_t st) {
    const int64_t words = (int64_t)a.N * (a.K / 8);
    w4_quantize_kernel<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(a, words);
    return cudaGetLastError();
}

}  // namespace la
