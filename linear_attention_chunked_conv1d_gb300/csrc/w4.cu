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

// The products: a tile of 128 outputs, 16 to a warp, over a share of the inputs that the blocks of a
// cluster split. 128 inputs at a time go through a ring of asynchronous copies: the tile's weights (8
// KB) and the rows' inputs, laid out so that a lane finds its part of an operand in 16 bytes. Weights
// are the A operand of mma.m16n8k16, 16 outputs by 16 inputs, as exact bf16 integers -8 .. 7; the rows
// are B. A lane's word of eight weights serves two mma: which inputs meet in one mma is free as long
// as A and B agree, so word c of 32 inputs goes to the lanes with c = lane % 4 as it lies in memory.
// Products and sums within a group are exact integers times bf16 in fp32; each group's sum is scaled
// by its output's scale and added up in fp32. Blocks of a cluster leave their sums in shared memory
// and each adds up a share of the outputs, in order of the blocks.
constexpr int kThreads = 256;
constexpr int kTile = 128;        // outputs of a block
constexpr int kSeg = 128;         // inputs of a stage
constexpr int kRowBytes = 64 + 16;  // a row's weights of a stage, padded: 8 rows x 4 lanes on 32 banks
constexpr int kStages = 5;

__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Weights 2i and 2i + 1 of a word as bf16: 128 + q is exact in bf16 (0x4300 | q), and so is its
// difference to 136.
__device__ __forceinline__ uint32_t weight_pair(uint32_t word, int i) {
    const uint32_t v = (word >> (4 * i) & 0x000f000fu) | 0x43004300u;
    __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __floats2bfloat162_rn(136.f, 136.f));
    return *reinterpret_cast<uint32_t *>(&h);
}

template <int NT> constexpr int kStageBytes = kTile * kRowBytes + NT * 2048;

template <int NT, int G>  // 8 NT rows at most, groups of G inputs
__global__ void __launch_bounds__(kThreads, 2) w4_matvec_kernel(const W4Args a, int segs_each) {
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int t = threadIdx.x, warp = t / 32, lane = t % 32, g = lane / 4, c = lane % 4;
    uint32_t rank, blocks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    const int n0 = blockIdx.x / blocks * kTile;
    const int all = (a.K + kSeg - 1) / kSeg;
    const int first = rank * segs_each, last = min(first + segs_each, all);
    const unsigned char *q = static_cast<const unsigned char *>(a.q);
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x);

    const auto fetch = [&](int seg) {
        if (seg < last) {
            const uint32_t to = sbase + seg % kStages * kStageBytes<NT>;
#pragma unroll
            for (int i = 0; i < kTile * 4 / kThreads; ++i) {
                const int r = (t + i * kThreads) / 4, part = t % 4, k = seg * kSeg + part * 32;
                const bool there = n0 + r < a.N && k < a.K;
                copy16(to + r * kRowBytes + part * 16, there ? q + (int64_t)(n0 + r) * (a.K / 2) + k / 2 : q, there);
            }
#pragma unroll
            for (int i = 0; i < (NT * 128 + kThreads - 1) / kThreads; ++i) {
                const int at = t + i * kThreads, m = at / 16, jc = at % 16, k = seg * kSeg + jc * 8;
                const bool there = m < a.M && k < a.K;
                if (NT * 128 >= kThreads || at < NT * 128)
                    copy16(to + kTile * kRowBytes + ((m / 8 * 4 + jc / 4) * 32 + m % 8 * 4 + jc % 4) * 16,
                           there ? x + m * a.ldx + k : x, there);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the scales of this lane's two outputs in a stage
    constexpr int kGroups = kSeg / G;
    const int row0 = n0 + warp * 16 + g, per_row = a.K / G;
    const __nv_bfloat16 *sc = static_cast<const __nv_bfloat16 *>(a.scales);
    const auto scales = [&](int seg, float (&s)[2][kGroups]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int row = row0 + 8 * h, at = seg * kGroups + i;
                s[h][i] = row < a.N && at < per_row && seg < last ? to_f(sc[(int64_t)row * per_row + at]) : 0.f;
            }
    };

    float acc[NT][4] = {}, next[2][kGroups];
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s);
    scales(first, next);
    for (int seg = first; seg < last; ++seg) {
        float s[2][kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) s[0][i] = next[0][i], s[1][i] = next[1][i];
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();  // this stage is here, and the one before it read by all
        fetch(seg + kStages - 1);
        scales(seg + 1, next);
        const unsigned char *st = smem + seg % kStages * kStageBytes<NT>;
        const uint32_t *w0 = reinterpret_cast<const uint32_t *>(st + (warp * 16 + g) * kRowBytes) + c;
        const uint32_t *w1 = w0 + 8 * kRowBytes / 4;
        const uint4 *xs = reinterpret_cast<const uint4 *>(st + kTile * kRowBytes) + lane;
        float part[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j * 32 % G == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0.f;
            }
            const uint32_t u0 = w0[j * 4], u1 = w1[j * 4];
            const uint32_t A0[4] = {weight_pair(u0, 0), weight_pair(u1, 0), weight_pair(u0, 1), weight_pair(u1, 1)};
            const uint32_t A1[4] = {weight_pair(u0, 2), weight_pair(u1, 2), weight_pair(u0, 3), weight_pair(u1, 3)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 b = xs[(n * 4 + j) * 32];
                mma_bf16(part[n], A0, b.x, b.y);
                mma_bf16(part[n], A1, b.z, b.w);
            }
            if ((j + 1) * 32 % G == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][e] = fmaf(s[e / 2][j * 32 / G], part[n][e], acc[n][e]);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // sums to shared memory: [8 NT rows][128 outputs]
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[(n * 8 + 2 * c + e % 2) * kTile + warp * 16 + g + e / 2 * 8] = acc[n][e];
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // each block adds up a share of the outputs
    const int share = kTile / (int)blocks;
    for (int i = t; i < a.M * share; i += kThreads) {
        const int m = i / share, r = (int)rank * share + i % share;
        float v = 0.f;
        for (uint32_t b = 0; b < blocks; ++b) {
            uint32_t at;
            float u;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sbase + (m * kTile + r) * 4), "r"(b));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(at) : "memory");
            v += u;
        }
        if (n0 + r < a.N) static_cast<__nv_bfloat16 *>(a.y)[m * a.ldy + n0 + r] = __float2bfloat16_rn(v);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Blocks that share a tile's inputs: as many (1, 2, 4 or 8) as it takes for a block and a half on each
// of 152 SMs, while each still has four stages. By N and K alone, and a fixed number of SMs: a row's
// sums do not depend on the batch or the device.
int cluster_of(int N, int K) {
    const int tiles = (N + kTile - 1) / kTile, segs = (K + kSeg - 1) / kSeg;
    int blocks = 1;
    while (blocks < 8 && tiles * blocks < 228 && segs >= 8 * blocks) blocks *= 2;
    return blocks;
}

template <int NT, int G> cudaError_t launch_t(const W4Args &a, cudaStream_t st) {
    constexpr int smem = kStages * kStageBytes<NT>;
    static_assert(smem >= NT * 8 * kTile * 4, "the sums take the ring's place");
    cudaError_t e = cudaFuncSetAttribute(w4_matvec_kernel<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int blocks = cluster_of(a.N, a.K), segs = (a.K + kSeg - 1) / kSeg;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + kTile - 1) / kTile * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4_matvec_kernel<NT, G>, a, (segs + blocks - 1) / blocks);
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
