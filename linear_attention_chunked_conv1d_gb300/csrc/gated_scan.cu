// Gated linear recurrence with one state per channel, over packed streams, and its backward pass:
//   d_t = sigmoid(a_t), beta_t = sigmoid(b_t), h_t = (1 - d_t) h_{t-1} + beta_t x_t, y_t = h_t.
// 1 - d = exp(-softplus(a)) and beta are the gates of la_gate_activations ("split_prefill.rs",
// prefill_phase1_proj_batched) on the same rows a | b; the recurrence is the per-channel counterpart
// of the KDA state update ("glm5next_kda/prefill.rs"), without its key and value dimensions.
//
// Backward: with m the gradient of the state that a token finds (for the last token's successor: the
// gradient of the stream's final state),
//   lam_t = dy_t + m_{t+1},  m_t = (1 - d_t) lam_t,  dh_0 = m at the stream's first token,
//   dx = lam beta,  db = lam x beta (1 - beta),  da = -lam h_{t-1} d (1 - d).
// h_{t-1} is computed again from the states that the forward pass saved.
//
// Both are HBM-bound: 4 activations a (token, channel) forward, 7 backward, a few tens of
// instructions on them. One launch reads every input once, whatever the streams' lengths:
//  - The packed rows are cut into tiles of L tokens x 32 channels, regardless of where streams meet
//    (but for the few sections below).
//    A tile maps the state (or, backward, the gradient m) that reaches it to the one that leaves it:
//    h -> K h + H with K = prod (1 - d). Where a stream starts inside the tile, what comes from before
//    is dropped. K is a product of its factors, right to its own last places however small it gets:
//    what a channel forgets is gone. Of a K above 3/4 the difference from 1, N = K - 1, is kept beside
//    it, for the reason in gated.cuh, and it is what the tiles of a chain pass on (word_of).
//  - Tiles of a channel group are chained along the sequence. A block publishes its tile's (N, H) as
//    soon as it has them, finds the nearest earlier tile whose outgoing state is known, and applies
//    the maps in between to that state, oldest first. The state that leaves a tile is thus the same
//    expression, evaluated in the same order, wherever that search ended: results do not depend on
//    timing. Tiles are handed out in chain order by a counter, so a tile's predecessors are always
//    done or running and no block waits for one that has not started; the waits are bounded.
//  - Narrow, long tiles keep that search short: blocks at work / chains tiles of a chain are in flight
//    at a time, 5 at 2048 channels (128-channel tiles of 64 tokens: 19, and the whole scan was bound by
//    it). Several streams make more chains: the rows are cut into sections where a stream starts, each
//    with tiles and chains of its own, as many as it takes for one tile of a chain in flight.
//  - Blocks are persistent. Tiles come by TMA into a ring in shared memory and are worked on in
//    registers, so a tile's place in the ring is free again, and the next copy under way, while the
//    tile waits for its state.
//  - To keep the instructions few (29 a (token, channel) forward, 65 backward) channels go in packed
//    pairs, and tiles without a start or an end of a stream (all but one in each stream)
//    take a path without tests for them.
// Measured, bf16: 262,144 x 2048 in 64 streams 0.79 ms (5.4 TB/s of what has to move), one stream 65,536 x
// 2048 0.237 ms (4.5 TB/s: it waits for its chains), both passes of 8 x 2048 x 4096 0.348 ms (4.2 TB/s: the
// backward pass waits at its tiles' two barriers, 45% of its issue slots are used).
#include <cuda.h>

#include <type_traits>

#include "gated.cuh"
#include "launch.h"
#include "overlap.cuh"
#include "tc.cuh"

namespace la {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kLoader = 3;   // the warp that takes tiles and starts their copies
constexpr int kWidth = 32;   // channels of a tile: 8 lanes of 4; the other 4 lanes' worth of a warp
constexpr int kRuns = 4 * kWarps;  // is along the tokens, in runs of S
constexpr uint64_t kWaitNs = 2000000000ull;

// Tokens of a run, and the ring's depth. What a thread keeps of a tile across the wait for its state
// is 2 registers a (token, channel) forward and 4.5 (bf16) or 5 (fp32) backward; two blocks on an SM leave
// 128 registers a thread, which these fill: half of these runs takes half again as long. A tile's place
// in the ring is free, and its next copy under way, half way through the tile: backward one place is
// enough (a second one only takes tiles earlier than needed: 8 x 2048 x 4096 bf16, both passes, 2%
// longer), forward two are better by 5%.
template <typename T, bool BWD> struct Shape {
    static constexpr int kIn = BWD ? 4 : 3;                              // x, a, b (, dy)
    static constexpr int S = sizeof(T) == 2 && !BWD ? 8 : 4;
    static constexpr int L = S * kRuns;
    static constexpr int kPlane = L * kWidth * (int)sizeof(T);           // bytes of one input's tile
    static constexpr int kStage = kIn * kPlane;                          // 48 KB; backward 32 (bf16), 64 (fp32)
    static constexpr int kStages = BWD ? 1 : 2;
    static constexpr int kBlocks = 2;                                    // on an SM
    // A slot is read until its tile is done, one tile longer than its copies are.
    static constexpr int kSlots = kStages + 1;
};

// Tokens between two saved states, from the start of a section: the backward tile.
template <typename T> constexpr int kSave = Shape<T, true>::L;

constexpr int kMaxSections = 8;

// Sections of a call: chains enough for the blocks of 152 SMs, and not more than streams. By sizes
// alone, as the saved states follow them.
template <typename T> int sections_of(int B, int total, int channels) {
    if (total <= Shape<T, false>::L) return 1;
    const int groups = (channels + kWidth - 1) / kWidth, wanted = (2 * 152 + groups - 1) / groups;
    const int n = wanted < kMaxSections ? wanted : kMaxSections;
    return n < B ? n : B;
}
// The most tiles (saved states) that total tokens in these sections can have.
inline int64_t tiles_of(int total, int sections, int L) { return (int64_t)total / L + sections; }

// What lies in the workspace before the tiles' words.
struct Ctl {
    int bad;          // an offset of cu_seqlens is out of order: no stream runs
    int abort;        // a wait ran out: every block leaves
    unsigned ticket;  // tiles handed out, of
    unsigned tasks;   // tiles * groups
};

// A tile, by its place in the order of work.
struct alignas(16) Tile {
    int t0, count;  // its tokens
    int id, place;  // in the chains' arrays and in its chain
    int first;      // the stream of its first token; ~: some token is marked (Slot)
    int saved;      // row of the saved state that reaches it
    int pad[2];
};

// A word of the chains that nobody has written. No value is: arithmetic makes no NaN of this pattern.
constexpr uint32_t kUnwritten = 0xffffffffu;

struct Chain {
    Ctl *ctl;
    Tile *tile;          // [tiles]
    float *N, *H, *out;  // [tiles][groups][32]: the tile's map (N: word_of), the state that leaves it
    int tiles, groups, sections;  // tiles: the most there can be
    // All tokens fit in one tile: nothing is chained, and a block for each group does without the
    // kernel that lays the chains out (100 tokens x 768 fp32: 9.7 us on the device with it, 4.4 without).
    bool single;
};

template <typename T, bool BWD> Chain make_chain(void *workspace, int B, int total, int channels) {
    Chain c;
    c.sections = sections_of<T>(B, total, channels);
    c.tiles = (int)tiles_of(total, c.sections, Shape<T, BWD>::L);
    c.groups = (channels + kWidth - 1) / kWidth;
    c.single = total <= Shape<T, BWD>::L;
    const int64_t words = (int64_t)c.tiles * c.groups * kWidth;
    c.ctl = static_cast<Ctl *>(workspace);
    c.tile = reinterpret_cast<Tile *>(c.ctl + 1);
    c.N = reinterpret_cast<float *>(c.tile + c.tiles);
    c.H = c.N + words;
    c.out = c.H + words;
    return c;
}

template <typename T, bool BWD> size_t chain_bytes(int B, int total, int channels) {
    const Chain c = make_chain<T, BWD>(nullptr, B, total, channels);
    return sizeof(Ctl) + c.tiles * sizeof(Tile) + (size_t)c.tiles * c.groups * kWidth * 12;
}

// Where the streams start and end in the packed rows.
struct Streams {
    const int32_t *cu;  // or nullptr: B streams of T_each tokens
    int B, T_each, total;
    __device__ __forceinline__ int start(int s) const { return cu ? cu[s] : s * T_each; }
    // Whether an offset is out of order; every thread of the block looks at its share.
    __device__ __forceinline__ bool bad() const {
        int b = 0;
        if (cu) {
            if (threadIdx.x == 0) b = cu[0] != 0 || cu[B] != total;
            for (int s = threadIdx.x; s < B; s += blockDim.x) b |= cu[s + 1] < cu[s];
        }
        return __syncthreads_or(b);
    }
};

// Clears the chains and lays out the tiles in the order of work: the first of each section's chains
// (the last one's, BWD), then the second ones, ...; block 0 also looks at every offset.
template <bool BWD>
__global__ void chain_init_kernel(Streams st, int L, int save, Chain c, int *status) {
    // sections, longest first: where they start and end, their first tile's id and saved row
    __shared__ int from[kMaxSections + 1], start[kMaxSections], end[kMaxSections], id[kMaxSections], row[kMaxSections];
    const int K = c.sections, tid = threadIdx.x;
    wait_for_previous();
    if (tid <= K) {  // at the first stream that starts at or after an even share
        const int64_t share = (int64_t)st.total * tid / K;
        int lo = 0, hi = st.B;  // it is in [lo, hi]
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (st.start(mid) < share) lo = mid + 1; else hi = mid;
        }
        from[tid] = st.start(lo);
    }
    __syncthreads();
    if (tid == 0) {
        int tiles = 0, rows = 0;
        for (int k = 0; k < K; ++k) {
            const int len = from[k + 1] - from[k];
            int at = k;
            for (; at > 0 && end[at - 1] - start[at - 1] < len; --at)
                start[at] = start[at - 1], end[at] = end[at - 1], id[at] = id[at - 1], row[at] = row[at - 1];
            start[at] = from[k], end[at] = from[k + 1], id[at] = tiles, row[at] = rows;
            tiles += (len + L - 1) / L;
            rows += (len + save - 1) / save;
        }
    }
    __syncthreads();
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + tid, step = (int64_t)gridDim.x * blockDim.x;
    int tasks = 0;
    for (int k = 0; k < K; ++k) tasks += (end[k] - start[k] + L - 1) / L;
    for (int64_t o = t; o < c.tiles && o < tasks; o += step) {
        // order `o`: `place` of section k, where the first j sections still have tiles
        int rest = (int)o, place = 0, k = 0;
        for (int j = K; j > 0; --j) {
            const int upto = (end[j - 1] - start[j - 1] + L - 1) / L;
            if (rest < j * (upto - place)) {
                place += rest / j;
                k = rest % j;
                break;
            }
            rest -= j * (upto - place);
            place = upto;
        }
        const int n = (end[k] - start[k] + L - 1) / L, i = BWD ? n - 1 - place : place;
        Tile v;
        v.t0 = start[k] + i * L;
        v.count = min(L, end[k] - v.t0);
        v.id = id[k] + i;
        v.place = place;
        v.saved = row[k] + i * (L / save);
        int lo = 0, hi = st.B;  // the last stream that starts at or before t0 is in [lo, hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (st.start(mid) <= v.t0) lo = mid; else hi = mid;
        }
        const bool whole = st.start(lo) < v.t0 && st.start(lo + 1) > v.t0 + L;  // inside one stream
        v.first = whole ? lo : ~lo;
        v.pad[0] = v.pad[1] = 0;
        c.tile[o] = v;
    }
    const int64_t quads = (int64_t)c.tiles * c.groups * kWidth * 3 / 4;
    uint4 *p = reinterpret_cast<uint4 *>(c.N);
    for (int64_t i = t; i < quads; i += step) p[i] = make_uint4(kUnwritten, kUnwritten, kUnwritten, kUnwritten);
    if (blockIdx.x) return;
    const bool bad = st.bad();
    if (tid == 0) {
        *c.ctl = Ctl{bad, 0, 0u, (unsigned)tasks * (unsigned)c.groups};
        if (bad) raise_status(status, LA_DEV_BAD_SEQLENS);
    }
}

// A tile in the ring: which one it is, and where in it streams start and end.
template <int L> struct Slot {
    static constexpr int S = L / kRuns;
    int t0, count, id, place, saved;        // as Tile
    int group;                              // of channels; -1: no more
    bool marked;                            // some token is (a section's last one always)
    uint32_t starts[L / 32], ends[L / 32];  // a bit for each token
    // A bit for each run with a start (an end) in it. A start at the tile's first token and an end
    // at its last are apart: there the state (gradient) that reaches the tile is the stream's own.
    uint32_t run_starts, run_ends;
    int start_id[L];                        // the streams of the marked starts
    int run_id[kRuns];                      // the stream of each run's first token

    __device__ __forceinline__ bool first() const { return starts[0] & 1u; }
    __device__ __forceinline__ bool last() const { return ends[L / 32 - 1] >> 31; }
    // the marked tokens of a run, without those two
    __device__ __forceinline__ uint32_t starts_of(int run) const { return bits(starts, run) & (run ? ~0u : ~1u); }
    __device__ __forceinline__ uint32_t ends_of(int run) const {
        return bits(ends, run) & (run < kRuns - 1 ? ~0u : ~(1u << (S - 1)));
    }
    static __device__ __forceinline__ uint32_t bits(const uint32_t *mask, int run) {
        return mask[run * S / 32] >> (run * S % 32) & ((1u << S) - 1u);
    }
    // the stream of a run's token i
    __device__ __forceinline__ int stream(int run, int i) const {
        const uint32_t before = bits(starts, run) & ((2u << i) - 1u);
        return before ? start_id[run * S + 31 - __clz(before)] : run_id[run];
    }
};

// The whole warp marks the tokens t0 .. t0 + count - 1 of a slot; `lo` is the stream of the first one.
template <int L> __device__ void mark_streams(const Streams &st, int lo, int t0, int count, int lane, Slot<L> *slot) {
    if (lane < L / 32) slot->starts[lane] = slot->ends[lane] = 0;
    __syncwarp();
    for (int s0 = lo; s0 < st.B; s0 += 32) {
        const int s = s0 + lane;
        int b = st.total, e = st.total;
        if (s < st.B) {
            b = st.start(s);
            e = st.start(s + 1);
            if (b < e) {  // an empty stream has no tokens to mark
                if (b >= t0 && b < t0 + count) {
                    atomicOr(&slot->starts[(b - t0) >> 5], 1u << ((b - t0) & 31));
                    slot->start_id[b - t0] = s;
                }
                if (e > t0 && e <= t0 + count) atomicOr(&slot->ends[(e - 1 - t0) >> 5], 1u << ((e - 1 - t0) & 31));
            }
        }
        if (__any_sync(0xffffffffu, b >= t0 + count || s >= st.B)) break;
    }
    __syncwarp();
    const unsigned rs = __ballot_sync(0xffffffffu, slot->starts_of(lane) != 0);
    const unsigned re = __ballot_sync(0xffffffffu, slot->ends_of(lane) != 0);
    if (lane == 0) slot->run_starts = rs, slot->run_ends = re;
    static_assert(kRuns == 32, "a lane for each run");
    const int at = lane * (L / kRuns);  // the run's first token: the last start at or before it
    int id = lo;
    for (int w = at / 32; w >= 0; --w) {
        const uint32_t m = slot->starts[w] & (w == at / 32 ? (2u << at % 32) - 1u : ~0u);
        if (m) {
            id = slot->start_id[w * 32 + 31 - __clz(m)];
            break;
        }
    }
    slot->run_id[lane] = id;
    __syncwarp();
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ F4 zero4() { return all4(0.f); }

// h -> K h + H of some tokens.
struct Map {
    F4 K, H;
    __device__ __forceinline__ F4 apply(const F4 &h) const { return fma4(K, h, H); }
    // these tokens after those of `e`
    __device__ __forceinline__ Map after(const Map &e) const { return Map{mul4(K, e.K), apply(e.H)}; }
};
__device__ __forceinline__ Map identity() { return Map{all4(1.f), zero4()}; }

// What a run's tokens leave of a state, K = R or 1 + N: R is rounded at every token, which for slow
// channels goes the same way each time, N's terms all have one sign. N is there only where every decay of
// the run is above 1/2 (decay4), so that it is looked at only where K is well above it.
constexpr float kSlow = 0.75f;
__device__ __forceinline__ F4 left_of_run(const F4 &N, const F4 &R) {
    float n[4], r[4];
    unpack4(N, n);
    unpack4(R, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = r[e] > kSlow ? 1.f + n[e] : r[e];
    return pack4(r);
}
// N of a warp's four runs (ranks), from each lane's: (1 + a)(1 + b) - 1 = a (1 + b) + b.
__device__ __forceinline__ F4 join_ranks(F4 N) {
#pragma unroll
    for (int off = 8; off < 32; off *= 2) {
        float f[4];
        unpack4(N, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __shfl_xor_sync(0xffffffffu, f[e], off);
        const F4 other = pack4(f);
        N = fma4(N, add4(other, all4(1.f)), other);
    }
    return N;
}

// The word by which a tile's K is passed on: N (its sign is set: -0 says that all is kept) where K is above
// kSlow, else K itself (its sign is not).
__device__ __forceinline__ float word_of(float N, float K) { return K > kSlow ? N : K; }
// K h of a word
__device__ __forceinline__ float left_by(float word, float h) { return fmaf(word, h, __float_as_int(word) < 0 ? h : 0.f); }

// The first `last` of n maps (rows at a stride of kStep), joined in order of the tokens, or against it
// (REV: row n - 1 first). A bit in `resets` says that a stream starts among a row's tokens: what comes
// before it is dropped there, not multiplied by 0 (it may be NaN). kMarked: whether there may be any.
template <bool REV, bool kMarked, int n, int kStep>
__device__ __forceinline__ Map join(const float (*K)[kWidth], const float (*H)[kWidth], uint32_t resets, int last, int quad) {
    Map m = identity();
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const int r = REV ? n - 1 - k : k;
        if (k < last) {
            const Map e{load_f4(&K[r * kStep][quad * 4]), load_f4(&H[r * kStep][quad * 4])};
            m = kMarked && (resets >> r & 1u) ? Map{e.after(m).K, e.H} : e.after(m);
        }
    }
    return m;
}
// Whether there is a reset among the first `last` of n rows.
template <bool REV, int n> __device__ __forceinline__ bool reset_before(uint32_t resets, int last) {
    return resets & (REV ? ~0u << (n - last) : (1u << last) - 1u) & ((1u << n) - 1u);
}
// A bit for each warp with a bit among its four runs.
__device__ __forceinline__ uint32_t by_warp(uint32_t runs) {
    uint32_t r = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) r |= (uint32_t)((runs >> 4 * w & 15u) != 0) << w;
    return r;
}

__device__ __forceinline__ void store_relaxed(float *p, float v) {
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ bool written(float v) { return __float_as_uint(v) != kUnwritten; }
__device__ __forceinline__ int load_abort(const Ctl *ctl) {
    int v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(&ctl->abort) : "memory");
    return v;
}

// Passing a tile's state on is the work of one warp, with one channel a lane: few registers, next to
// those that hold its tokens.

// The joined map of all warps of a tile (as join, for one channel), its K as a word.
template <bool REV, bool kMarked, class Sh>
__device__ __forceinline__ void join_all(const Sh *sh, const float (*H)[kWidth], uint32_t resets, int lane, float &word, float &h) {
    float n = -0.f, k = 1.f;
    h = 0.f;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        const int r = REV ? kWarps - 1 - j : j;
        const float en = sh->N[r][lane], ek = sh->K[r * 4 + 3][lane], eh = H[r * 4][lane];
        n = fmaf(n, 1.f + en, en);
        k *= ek;
        h = kMarked && (resets >> r & 1u) ? eh : fmaf(ek, h, eh);
    }
    word = word_of(n, k);
}

// Eight places of a chain in shared memory, `top` and those before it, as one warp finds them in L2.
// The words themselves say whether they have been written, each by itself, so there are no flags and
// no fences, and the copies can start before their answer is needed.
struct Window {
    float N[8][kWidth], H[8][kWidth], out[8][kWidth];

    template <class Cell> __device__ __forceinline__ void fetch(const Chain &c, int top, Cell cell, int lane) {
        const int quad = lane % 8 * 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int n = 4 * u + lane / 8, p = top - n;
            if (p >= 0) {
                const int64_t at = cell(p) * kWidth + quad;
                copy(&out[n][quad], c.out + at);
                copy(&N[n][quad], c.N + at);
                copy(&H[n][quad], c.H + at);
            } else {
                store_f4(&out[n][quad], all4(__uint_as_float(kUnwritten)));
                store_f4(&N[n][quad], all4(__uint_as_float(kUnwritten)));
            }
        }
    }
    static __device__ __forceinline__ void copy(float *to, const float *from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
    }
    // Waits for the copies. Bit n of the answer: place top - n has its state there; bit 8 + n: its map.
    __device__ __forceinline__ unsigned look(int lane) const {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        unsigned there = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (written(out[n][lane])) there |= 1u << n;
            if (written(N[n][lane]) && written(H[n][lane])) there |= 256u << n;
        }
        return __reduce_and_sync(0xffffffffu, there);
    }
    // h through places top - n + 1 .. top
    __device__ __forceinline__ float apply(int n, float h, int lane) const {
        for (int k = n - 1; k >= 0; --k) h = left_by(N[k][lane], h) + H[k][lane];
        return h;
    }
};

// What reaches the tile at place `at` > 0 of its chain. cell(place) is a place's index; `w` has been
// told to fetch the places before `at`. False: the wait ran out (with `stall` it is made to). Every copy
// into the window has been waited for when it returns: such copies have no order among themselves, so one
// of this tile's must not be under way when the next tile's begin.
template <class Cell>
__device__ __forceinline__ bool look_back(Window &w, const Chain &c, int at, Cell cell, int lane, uint64_t wait_ns,
                                          bool stall, float &h) {
    int top = at - 1, n = 0;  // place top - n is the search's result
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        const unsigned seen = w.look(lane), there = stall ? 0u : seen, states = there & 255u, maps = there >> 8;
        const unsigned nearer = states ? (states & -states) - 1 : 255u;
        if ((maps & nearer) == nearer) {
            if (states) {
                n = __ffs(states) - 1;
                break;
            }
            top -= 8;  // place 0 has a state and no map: the search never passes it
        } else if ((i & 15) == 15) {
            const uint64_t now = tc::globaltimer_ns();
            if (!t0) t0 = now;
            if (__any_sync(0xffffffffu, now - t0 > wait_ns || load_abort(c.ctl))) return false;
        }
        __syncwarp();
        w.fetch(c, top, cell, lane);
    }
    h = w.apply(n, w.out[n][lane], lane);
    while (top < at - 1) {  // on to `at` through the windows that the search has seen
        top += 8;
        __syncwarp();
        w.fetch(c, top, cell, lane);
        w.look(lane);
        h = w.apply(8, h, lane);
    }
    return true;
}

// Publishes the map (n: the word of its K, h) of the tile at `place` (`reset`: its h is what leaves it, whatever comes),
// waits for what reaches it (unless `known`: then the window has not been told to fetch anything, as nobody
// would wait for it), publishes what leaves it. False: the wait ran out.
template <class Cell>
__device__ __forceinline__ bool pass_on(Window &w, const Chain &c, int place, Cell cell, int lane, float n, float h,
                                        bool reset, bool known, uint64_t wait_ns, bool stall, float &in) {
    const int64_t own = cell(place) * kWidth + lane;
    if (reset) {
        store_relaxed(c.out + own, h);
    } else if (!known) {
        store_relaxed(c.N + own, n);
        store_relaxed(c.H + own, h);
    }
    if (!known && !look_back(w, c, place, cell, lane, wait_ns, stall, in)) return false;
    if (!reset) store_relaxed(c.out + own, left_by(n, in) + h);
    return true;
}

// Why a block leaves: a warp's wait for the tile ran out, told at the tile's first barrier, or the wait for
// its state, told at the second. Two values, so that a warp that is late to look behind one barrier does
// not take what was written after it for that barrier's answer, and leave while others wait at the next.
enum { kNoTile = 1, kNoState = 2 };

// Shared memory of a block, in front of its ring.
template <int L, int STAGES, bool BWD> struct Shared {
    uint64_t full[STAGES];
    int failed;
    Slot<L> slot[STAGES + 1];
    // the runs' maps: K and H, backward also M with K along the reverse scan; then, in the last row of
    // each warp's four (of M: in the first), the warps'
    alignas(16) float K[kRuns][kWidth], H[kRuns][kWidth], M[BWD ? kRuns : 1][kWidth];
    alignas(16) float N[kWarps][kWidth];  // the warps' K - 1
    alignas(16) float in[kWidth];  // what reaches the tile
    alignas(16) Window window;
};

template <class Sh> __device__ void init_shared(Sh *sh, int stages) {
    for (int s = 0; s < stages; ++s) tc::mbar_init(&sh->full[s], 2);  // the copies and the slot
    sh->failed = 0;
    tc::fence_mbar_init();
}

// What the loading warp does, all its lanes together.
template <typename T, bool BWD, bool kSingle, class Sh> struct Loader {
    using G = Shape<T, BWD>;
    Sh *sh;
    unsigned char *ring;
    const CUtensorMap *x, *a, *b, *dy;
    Streams streams;
    Chain c;
    uint32_t issued;  // tiles put into the ring, the end among them

    unsigned tasks;
    unsigned ticket;  // the tile last taken (lane 0's)

    // Takes the next tile of the chains, in their order: late, for a tile taken early is one that its
    // successors wait for (taken one tile sooner, a 262,144 x 2048 scan without sections takes 4% longer).
    __device__ __forceinline__ void take(int lane) {
        if (lane == 0 && !kSingle) ticket = atomicAdd(&c.ctl->ticket, 1u);
    }
    // The tile last taken into the ring's next place, or the end.
    __device__ void put(int lane) {
        const unsigned t = __shfl_sync(0xffffffffu, ticket, 0);
        if (t < tasks) {
            const int4 *tile = reinterpret_cast<const int4 *>(c.tile + t / c.groups);
            put_tile(tile[0], tile[1], (int)(t % c.groups), lane);
            return;
        }
        if (lane == 0) {
            sh->slot[issued % G::kSlots].group = -1;
            mbar_arrive(&sh->full[issued % G::kStages]);
            mbar_arrive(&sh->full[issued % G::kStages]);
        }
        ++issued;
    }
    // Starts a tile's copies into the ring's next place and fills in its slot. u: t0, count, id, place;
    // v: first, saved.
    __device__ void put_tile(const int4 &u, const int4 &v, int group, int lane) {
        const uint32_t s = issued % G::kStages;
        auto &slot = sh->slot[issued % G::kSlots];
        ++issued;
        if (lane == 0) {
            tc::mbar_expect_tx(&sh->full[s], G::kStage);
            const uint32_t to = tc::smem_u32(ring + s * G::kStage);
            tc::tma_load_2d(to, x, group * kWidth, u.x, &sh->full[s]);
            tc::tma_load_2d(to + G::kPlane, a, group * kWidth, u.x, &sh->full[s]);
            tc::tma_load_2d(to + 2 * G::kPlane, b, group * kWidth, u.x, &sh->full[s]);
            if (BWD) tc::tma_load_2d(to + 3 * G::kPlane, dy, group * kWidth, u.x, &sh->full[s]);
        }
        if (v.x < 0) mark_streams<G::L>(streams, ~v.x, u.x, u.y, lane, &slot);
        if (lane == 0) {
            slot.t0 = u.x;
            slot.count = u.y;
            slot.id = u.z;
            slot.place = u.w;
            slot.saved = v.y;
            slot.group = group;
            slot.marked = v.x < 0;
            mbar_arrive(&sh->full[s]);
        }
    }
    // Fills the ring.
    __device__ void begin(int lane) {
        int n = 0;
        if (kSingle) {  // the first stream that has tokens starts at the first one
            int first = 0;
            while (streams.start(first + 1) == 0) ++first;
            put_tile(make_int4(0, streams.total, 0, 0), make_int4(~first, 0, 0, 0), blockIdx.x, lane);
            n = 1;
        }
        for (; n < G::kStages; ++n) {  // one at a time: a second tile taken with the first is late for its chain
            take(lane);
            put(lane);
        }
    }
    // A block that leaves early waits (with a limit) for the copies it has started; those before number `it`
    // have been waited for.
    __device__ void drain(uint32_t it) {
        for (; it < issued; ++it) tc::mbar_wait(&sh->full[it % G::kStages], (it / G::kStages) & 1u, kWaitNs, 100000u);
    }
};

// A wait ran out (why: kNoTile, kNoState): the status says so, every block leaves.
template <class Sh> __device__ __forceinline__ void give_up(Sh *sh, const Chain &c, int why, int lane, int *status) {
    if (lane == 0) {
        atomicExch(&c.ctl->abort, 1);
        raise_status(status, LA_DEV_TIMEOUT);
    }
    *(volatile int *)&sh->failed = why;
}

template <typename T, bool kSingle>
__global__ void __launch_bounds__(kThreads, Shape<T, false>::kBlocks)
scan_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ CUtensorMap map_b, const GatedScanArgs a, const Chain c) {
    using G = Shape<T, false>;
    using V = Vec4<T>;
    constexpr int S = G::S, L = G::L, kPlane = G::kPlane / (int)sizeof(T);
    using Sh = Shared<L, G::kStages, false>;
    extern __shared__ __align__(128) unsigned char smem[];
    Sh *sh = reinterpret_cast<Sh *>(smem);
    unsigned char *ring = smem + (sizeof(Sh) + 127) / 128 * 128;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, quad = lane % 8, rank = lane / 8, run = warp * 4 + rank;
    if (threadIdx.x == 0) init_shared(sh, G::kStages);
    __syncthreads();
    wait_for_previous();
    const Streams streams{a.cu, a.B, a.T_each, a.total};
    if (kSingle ? streams.bad() : c.ctl->bad != 0) {
        if (kSingle && threadIdx.x == 0) raise_status(a.status, LA_DEV_BAD_SEQLENS);
        return;
    }
    Loader<T, false, kSingle, Sh> loader{sh, ring, &map_x, &map_a, &map_b, nullptr, streams, c, 0, kSingle ? 0u : c.ctl->tasks, 0};
    if (warp == kLoader) loader.begin(lane);
    volatile int *failed = &sh->failed;
    float *saved_initial = a.saved ? a.saved + a.saved_rows * a.channels : nullptr;

    // One tile of the ring, number `it`. False: the block leaves.
    const auto tile_step = [&](auto is_marked, const Slot<L> &slot, uint32_t it) {
        constexpr bool kMarked = decltype(is_marked)::value;
        const int group = slot.group, place = slot.place, chain = slot.id - place;
        const int ch = group * kWidth + quad * 4;
        const bool live = ch < a.channels;
        const uint32_t starts = kMarked ? slot.starts_of(run) : 0u;
        const uint32_t resets = kMarked ? slot.run_starts : 0u;
        const bool first = kMarked && slot.first();
        const auto cell = [&](int p) { return (int64_t)(chain + p) * c.groups + group; };

        // this run's tokens from a state of zero: h, and how much is left of what comes before
        F4 hl[S], A[S];
        const T *in = reinterpret_cast<const T *>(ring + it % G::kStages * G::kStage) + run * S * kWidth + quad * 4;
        Map m = identity();
        F4 N = all4(-0.f);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (kMarked && (starts >> i & 1u)) {
                const int id = slot.start_id[run * S + i];
                m.H = zero4();
                if (a.h_ptrs && live) m.H = load_f4(reinterpret_cast<const float *>(a.h_ptrs[id]) + ch);
                if (a.saved && live) {
                    store_f4(saved_initial + (int64_t)id * a.channels + ch, m.H);
                    if (i == 0 && run * S % kSave<T> == 0)
                        store_f4(a.saved + (int64_t)(slot.saved + run * S / kSave<T>) * a.channels + ch, m.H);
                }
            }
            F4 neg;
            const F4 side = decay4<false>(widen4<T>(V::load_raw(in + i * kWidth + kPlane)), neg), keep = decay_of(side, neg);
            const F4 beta = input4(widen4<T>(V::load_raw(in + i * kWidth + 2 * kPlane)));
            m.H = fma4(beta, widen4<T>(V::load_raw(in + i * kWidth)), mul4(keep, m.H));
            N = fma4(side, m.K, N);
            m.K = mul4(keep, m.K);
            hl[i] = m.H;
            A[i] = m.K;
        }
        m.K = left_of_run(N, m.K);
        if (warp == kWarps - 1 && !first) sh->window.fetch(c, place - 1, cell, lane);  // in good time for look_back
        store_f4(&sh->K[run][quad * 4], m.K);
        store_f4(&sh->H[run][quad * 4], m.H);
        N = join_ranks(N);
        __syncwarp();
        const uint32_t own_resets = resets >> 4 * warp & 15u;
        if (rank == 3) {
            const Map w = m.after(join<false, kMarked, 3, 1>(&sh->K[warp * 4], &sh->H[warp * 4], own_resets, 3, quad));
            store_f4(&sh->N[warp][quad * 4], N);
            store_f4(&sh->K[run][quad * 4], w.K);
            store_f4(&sh->H[run][quad * 4], kMarked && (own_resets & 8u) ? m.H : w.H);
        }
        __syncthreads();
        if (*failed == kNoTile) return false;
        if (warp == kLoader) loader.put(lane);

        const uint32_t warp_resets = kMarked ? by_warp(resets) : 0u;
        if (warp == kWarps - 1) {
            float n, h, v = 0.f;
            join_all<false, kMarked>(sh, &sh->H[3], warp_resets, lane, n, h);
            const int lane_ch = group * kWidth + lane;
            if (first && lane_ch < a.channels) {
                const int id = slot.start_id[0];
                if (a.h_ptrs) v = reinterpret_cast<const float *>(a.h_ptrs[id])[lane_ch];
                if (a.saved) saved_initial[(int64_t)id * a.channels + lane_ch] = v;
            }
            if (!pass_on(sh->window, c, place, cell, lane, n, h, resets != 0, first, a.wait_ns, a.debug_stall == 1, v))
                give_up(sh, c, kNoState, lane, a.status);
            sh->in[lane] = v;
        }
        const Map before_warp = join<false, kMarked, kWarps - 1, 4>(&sh->K[3], &sh->H[3], warp_resets, warp, quad);
        __syncthreads();
        if (*failed == kNoState) return false;

        // the state that reaches this run, then its tokens'
        F4 v = load_f4(&sh->in[quad * 4]);
        v = reset_before<false, kWarps>(warp_resets, warp) ? before_warp.H : before_warp.apply(v);
        const Map before_run = join<false, kMarked, 3, 1>(&sh->K[warp * 4], &sh->H[warp * 4], own_resets, rank, quad);
        v = reset_before<false, 4>(own_resets, rank) ? before_run.H : before_run.apply(v);
        const int count = kMarked ? slot.count - run * S : S;  // tokens of this run (or more)
        if (a.saved && live && run * S % kSave<T> == 0 && (!kMarked || (!(starts & 1u) && count > 0)))
            store_f4(a.saved + (int64_t)(slot.saved + run * S / kSave<T>) * a.channels + ch, v);
        const uint32_t ends = kMarked ? Slot<L>::bits(slot.ends, run) : 0u;
        T *yp = static_cast<T *>(a.y) + (int64_t)(slot.t0 + run * S) * a.y_stride + ch;
        bool fresh = false;  // a stream has started in this run
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (kMarked && (starts >> i & 1u)) fresh = true;
            const F4 y = kMarked && fresh ? hl[i] : fma4(A[i], v, hl[i]);
            if (live && (!kMarked || i < count)) store_act4<T>(yp, y);
            yp += a.y_stride;
            if (kMarked && (ends >> i & 1u) && a.h_ptrs && live)
                store_f4(reinterpret_cast<float *>(a.h_ptrs[slot.stream(run, i)]) + ch, y);
        }
        return true;
    };

    for (uint32_t it = 0;; ++it) {
        if (warp == kLoader) loader.take(lane);  // for the place that this tile leaves
        // one answer for the warp, whose lanes work together from here on
        const bool arrived = __all_sync(0xffffffffu, tc::mbar_wait(&sh->full[it % G::kStages], (it / G::kStages) & 1u,
                                                                   a.wait_ns + kWaitNs) && a.debug_stall != 2);
        const Slot<L> &slot = sh->slot[it % G::kSlots];
        if (arrived && slot.group < 0) break;
        if (!arrived) {  // nothing of the tile is used; the others leave at their first barrier
            give_up(sh, c, kNoTile, lane, a.status);
            __syncthreads();
        }
        const bool ok = !arrived ? false
                        : slot.marked ? tile_step(std::true_type{}, slot, it)
                                      : tile_step(std::false_type{}, slot, it);
        if (!ok) {  // no copy into shared memory, of the ring or of the window, outlives the block
            if (warp == kLoader) loader.drain(arrived ? it + 1 : it);
            asm volatile("cp.async.wait_all;" ::: "memory");
            break;
        }
    }
}

template <typename T, bool kSingle>
__global__ void __launch_bounds__(kThreads, Shape<T, true>::kBlocks)
scan_backward_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_dy,
                     const GatedScanBwdArgs a, const Chain c) {
    using G = Shape<T, true>;
    using V = Vec4<T>;
    constexpr int S = G::S, L = G::L, kPlane = G::kPlane / (int)sizeof(T);
    using Sh = Shared<L, G::kStages, true>;
    extern __shared__ __align__(128) unsigned char smem[];
    Sh *sh = reinterpret_cast<Sh *>(smem);
    unsigned char *ring = smem + (sizeof(Sh) + 127) / 128 * 128;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, quad = lane % 8, rank = lane / 8, run = warp * 4 + rank;
    if (threadIdx.x == 0) init_shared(sh, G::kStages);
    __syncthreads();
    wait_for_previous();
    const Streams streams{a.cu, a.B, a.T_each, a.total};
    if (kSingle ? streams.bad() : c.ctl->bad != 0) {
        if (kSingle && threadIdx.x == 0) raise_status(a.status, LA_DEV_BAD_SEQLENS);
        return;
    }
    Loader<T, true, kSingle, Sh> loader{sh, ring, &map_x, &map_a, &map_b, &map_dy, streams, c, 0, kSingle ? 0u : c.ctl->tasks, 0};
    if (warp == kLoader) loader.begin(lane);
    volatile int *failed = &sh->failed;
    const float *saved_initial = a.saved + (int64_t)c.tiles * a.channels;  // a tile for each saved row
    if (a.cu && a.dh0_ptrs) {  // the gradient passes through an empty stream
        for (int s = blockIdx.x; s < a.B; s += gridDim.x) {
            if (a.cu[s] != a.cu[s + 1]) continue;
            for (int i = threadIdx.x; i < a.channels; i += kThreads)
                reinterpret_cast<float *>(a.dh0_ptrs[s])[i] =
                    a.dh_final_ptrs ? reinterpret_cast<const float *>(a.dh_final_ptrs[s])[i] : 0.f;
        }
    }

    const auto tile_step = [&](auto is_marked, const Slot<L> &slot, uint32_t it) {
        constexpr bool kMarked = decltype(is_marked)::value;
        const int group = slot.group, place = slot.place, chain = slot.id + place;
        const int ch = group * kWidth + quad * 4;
        const bool live = ch < a.channels;
        const auto cell = [&](int p) { return (int64_t)(chain - p) * c.groups + group; };
        F4 h_in = zero4();  // the state that reaches the tile
        if (live) h_in = load_f4(a.saved + (int64_t)slot.id * a.channels + ch);
        const uint32_t starts = kMarked ? slot.starts_of(run) : 0u, ends = kMarked ? slot.ends_of(run) : 0u;
        const uint32_t resets = kMarked ? slot.run_starts : 0u, end_resets = kMarked ? slot.run_ends : 0u;
        // behind a chain's first place there is nothing: a stream ends in it
        const bool last = kMarked && slot.last(), known = last || place == 0;
        const auto initial = [&](int i) {  // state of the stream that starts at this run's token i
            return live ? load_f4(saved_initial + (int64_t)slot.start_id[run * S + i] * a.channels + ch) : zero4();
        };
        const auto final_gradient = [&](int i) {  // of the stream that ends at this run's token i
            return a.dh_final_ptrs && live ? load_f4(reinterpret_cast<const float *>(a.dh_final_ptrs[slot.stream(run, i)]) + ch)
                                           : zero4();
        };

        // the decays' sides (past the second barrier: the decays), e^-b, and what enters, beta x
        F4 gate[S], input[S], u[S];
        typename V::Raw dyr[S];
        const T *in = reinterpret_cast<const T *>(ring + it % G::kStages * G::kStage) + run * S * kWidth + quad * 4;
        Map h = identity();  // of this run, forward; with m in place of h.H, along the reverse scan
        F4 N = all4(-0.f), m = zero4(), keep[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            F4 neg;
            gate[i] = decay4<true>(widen4<T>(V::load_raw(in + i * kWidth + kPlane)), neg);
            input[i] = input_exp4(widen4<T>(V::load_raw(in + i * kWidth + 2 * kPlane)));
            keep[i] = decay_of(gate[i], neg);
            if (kMarked && (starts >> i & 1u)) h.H = initial(i);
            u[i] = mul4(input_of(input[i]), widen4<T>(V::load_raw(in + i * kWidth)));
            h.H = fma4(keep[i], h.H, u[i]);
            N = fma4(gate[i], h.K, N);
            h.K = mul4(keep[i], h.K);
        }
        h.K = left_of_run(N, h.K);
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
            dyr[i] = V::load_raw(in + i * kWidth + 3 * kPlane);
            if (kMarked && (ends >> i & 1u)) m = final_gradient(i);
            m = mul4(keep[i], add4(widen4<T>(dyr[i]), m));
        }
        if (warp == 0 && !known) sh->window.fetch(c, place - 1, cell, lane);  // in good time for look_back
        store_f4(&sh->K[run][quad * 4], h.K);
        store_f4(&sh->H[run][quad * 4], h.H);
        store_f4(&sh->M[run][quad * 4], m);
        N = join_ranks(N);
        __syncwarp();
        const uint32_t own_resets = resets >> 4 * warp & 15u, own_ends = end_resets >> 4 * warp & 15u;
        const Map h_run = join<false, kMarked, 4, 1>(&sh->K[warp * 4], &sh->H[warp * 4], own_resets, rank, quad);
        const Map m_run = join<true, kMarked, 4, 1>(&sh->K[warp * 4], &sh->M[warp * 4], own_ends, 3 - rank, quad);
        __syncwarp();
        if (rank == 3) {
            const Map w = h.after(h_run);
            store_f4(&sh->N[warp][quad * 4], N);
            store_f4(&sh->K[run][quad * 4], w.K);
            store_f4(&sh->H[run][quad * 4], kMarked && (own_resets & 8u) ? h.H : w.H);
        }
        if (rank == 0) store_f4(&sh->M[run][quad * 4], kMarked && (own_ends & 1u) ? m : Map{h.K, m}.apply(m_run.H));
        __syncthreads();
        if (*failed == kNoTile) return false;
        if (warp == kLoader) loader.put(lane);

        const uint32_t warp_resets = kMarked ? by_warp(resets) : 0u, warp_ends = kMarked ? by_warp(end_resets) : 0u;
        if (warp == 0) {
            float n, h, v = 0.f;
            join_all<true, kMarked>(sh, &sh->M[0], warp_ends, lane, n, h);
            const int lane_ch = group * kWidth + lane;
            if (last && a.dh_final_ptrs && lane_ch < a.channels)
                v = reinterpret_cast<const float *>(a.dh_final_ptrs[slot.stream(kRuns - 1, S - 1)])[lane_ch];
            if (!pass_on(sh->window, c, place, cell, lane, n, h, end_resets != 0, known, a.wait_ns, a.debug_stall == 1, v))
                give_up(sh, c, kNoState, lane, a.status);
            sh->in[lane] = v;
        }
        // meanwhile the others (and warp 0 after it) have the states before their tokens
        const Map h_warp = join<false, kMarked, kWarps - 1, 4>(&sh->K[3], &sh->H[3], warp_resets, warp, quad);
        F4 hd[S];  // what a token finds and forgets, -d h_{t-1}
        {
            F4 v = reset_before<false, kWarps>(warp_resets, warp) ? h_warp.H : h_warp.apply(h_in);
            v = reset_before<false, 4>(own_resets, rank) ? h_run.H : h_run.apply(v);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (kMarked && (starts >> i & 1u)) v = initial(i);
                const F4 neg = neg_of(gate[i]), side = gate[i];
                hd[i] = mul4(v, minus_d_of(side, neg));
                gate[i] = decay_of(side, neg);
                v = fma4(gate[i], v, u[i]);
            }
        }
        // what the tokens after this run make of the gradient that reaches the tile
        Map after_run = m_run;
        bool ended = reset_before<true, 4>(own_ends, 3 - rank);
        if (!ended) {
            after_run = m_run.after(join<true, kMarked, kWarps - 1, 4>(&sh->K[3 + 4], &sh->M[4], warp_ends >> 1, kWarps - 1 - warp, quad));
            ended = reset_before<true, kWarps>(warp_ends, kWarps - 1 - warp);
        }
        __syncthreads();
        if (*failed == kNoState) return false;

        // beta comes from e^-b anew: kept since its first use, it would be 4 S registers more, and spills (362 us
        // instead of 347 for both passes of 8 x 2048 x 4096 bf16)
#pragma unroll
        for (int i = 0; i < S; ++i) asm volatile("" : "+l"(input[i].p[0]), "+l"(input[i].p[1]));
        F4 v = load_f4(&sh->in[quad * 4]);
        v = ended ? after_run.H : after_run.apply(v);
        const uint32_t all_starts = kMarked ? Slot<L>::bits(slot.starts, run) : 0u;
        const int count = kMarked ? slot.count - run * S : S;
        T *dxp = static_cast<T *>(a.dx) + (int64_t)(slot.t0 + run * S + S - 1) * a.dx_stride + ch;
        T *dap = static_cast<T *>(a.dab) + (int64_t)(slot.t0 + run * S + S - 1) * a.dab_stride + ch;
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
            if (kMarked && (ends >> i & 1u)) v = final_gradient(i);
            const F4 lam = add4(widen4<T>(dyr[i]), v), beta = input_of(input[i]), dx = mul4(lam, beta);
            v = mul4(gate[i], lam);
            if (live && (!kMarked || i < count)) {
                store_act4<T>(dxp, dx);
                store_act4<T>(dap, mul4(v, hd[i]));
                store_act4<T>(dap + a.channels, mul4(mul4(lam, u[i]), mul4(input[i], beta)));
            }
            dxp -= a.dx_stride;
            dap -= a.dab_stride;
            if (kMarked && (all_starts >> i & 1u) && a.dh0_ptrs && live)
                store_f4(reinterpret_cast<float *>(a.dh0_ptrs[slot.start_id[run * S + i]]) + ch, v);
        }
        return true;
    };

    for (uint32_t it = 0;; ++it) {
        if (warp == kLoader) loader.take(lane);  // for the place that this tile leaves
        // one answer for the warp, whose lanes work together from here on
        const bool arrived = __all_sync(0xffffffffu, tc::mbar_wait(&sh->full[it % G::kStages], (it / G::kStages) & 1u,
                                                                   a.wait_ns + kWaitNs) && a.debug_stall != 2);
        const Slot<L> &slot = sh->slot[it % G::kSlots];
        if (arrived && slot.group < 0) break;
        if (!arrived) {  // nothing of the tile is used; the others leave at their first barrier
            give_up(sh, c, kNoTile, lane, a.status);
            __syncthreads();
        }
        const bool ok = !arrived ? false
                        : slot.marked ? tile_step(std::true_type{}, slot, it)
                                      : tile_step(std::false_type{}, slot, it);
        if (!ok) {  // no copy into shared memory, of the ring or of the window, outlives the block
            if (warp == kLoader) loader.drain(arrived ? it + 1 : it);
            asm volatile("cp.async.wait_all;" ::: "memory");
            break;
        }
    }
}

int device_sms() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Tensor map of one input's tiles, from its first channel.
template <typename T, bool BWD>
bool tile_map(CUtensorMap *map, const void *base, int total, int channels, int64_t ld) {
    return make_map_2d(map, base, sizeof(T) == 2 ? LA_BF16 : LA_F32, total, channels, ld, kWidth, Shape<T, BWD>::L, false);
}

// Clears the chain, then starts as many blocks as fit (or as there are tiles).
template <typename T, bool BWD, class Kernel, class Launch>
cudaError_t start(Kernel kernel, const Streams &streams, const Chain &c, int *status, cudaStream_t st,
                  Launch launch) {
    using G = Shape<T, BWD>;
    constexpr size_t smem = (sizeof(Shared<G::L, G::kStages, BWD>) + 127) / 128 * 128 + G::kStages * G::kStage;
    static_assert(G::kBlocks * (smem + 1024) <= 228 * 1024, "the blocks of an SM share its 228 KB, 1 KB of it each their own");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (c.single) return launch(c.groups, smem);
    const int64_t cells = (int64_t)c.tiles * c.groups, clear = (cells * kWidth * 3 / 4 + 1023) / 1024;
    const int sms = device_sms();
    e = launch_overlapped(chain_init_kernel<BWD>, dim3((int)(clear < sms ? clear : sms)), dim3(1024), 0, 0, st, streams, G::L, kSave<T>,
                          c, status);
    if (e != cudaSuccess) return e;
    const int room = G::kBlocks * sms;
    return launch((int)(cells < room ? cells : room), smem);
}

template <typename T> cudaError_t scan(GatedScanArgs a, cudaStream_t st) {
    CUtensorMap x, ga, gb;
    const T *ab = static_cast<const T *>(a.ab);
    if (!tile_map<T, false>(&x, a.x, a.total, a.channels, a.x_stride) ||
        !tile_map<T, false>(&ga, ab, a.total, a.channels, a.ab_stride) ||
        !tile_map<T, false>(&gb, ab + a.channels, a.total, a.channels, a.ab_stride))
        return cudaErrorInvalidValue;
    a.saved_rows = tiles_of(a.total, sections_of<T>(a.B, a.total, a.channels), kSave<T>);
    const Chain c = make_chain<T, false>(a.workspace, a.B, a.total, a.channels);
    const auto kernel = c.single ? scan_kernel<T, true> : scan_kernel<T, false>;
    return start<T, false>(kernel, Streams{a.cu, a.B, a.T_each, a.total}, c, a.status, st, [&](int grid, size_t smem) {
        return launch_overlapped(kernel, dim3(grid), dim3(kThreads), smem, 0, st, x, ga, gb, a, c);
    });
}

template <typename T> cudaError_t backward(const GatedScanBwdArgs &a, cudaStream_t st) {
    CUtensorMap x, ga, gb, dy;
    const T *ab = static_cast<const T *>(a.ab);
    if (!tile_map<T, true>(&x, a.x, a.total, a.channels, a.x_stride) ||
        !tile_map<T, true>(&ga, ab, a.total, a.channels, a.ab_stride) ||
        !tile_map<T, true>(&gb, ab + a.channels, a.total, a.channels, a.ab_stride) ||
        !tile_map<T, true>(&dy, a.dy, a.total, a.channels, a.dy_stride))
        return cudaErrorInvalidValue;
    const Chain c = make_chain<T, true>(a.workspace, a.B, a.total, a.channels);
    const auto kernel = c.single ? scan_backward_kernel<T, true> : scan_backward_kernel<T, false>;
    return start<T, true>(kernel, Streams{a.cu, a.B, a.T_each, a.total}, c, a.status, st, [&](int grid, size_t smem) {
        return launch_overlapped(kernel, dim3(grid), dim3(kThreads), smem, 0, st, x, ga, gb, dy, a, c);
    });
}

}  // namespace

size_t gated_scan_workspace_bytes(int B, int total, int channels, int dtype) {  // of either pass
    return dtype == LA_BF16 ? chain_bytes<__nv_bfloat16, true>(B, total, channels)
                            : chain_bytes<float, true>(B, total, channels);
}

size_t gated_scan_saved_bytes(int B, int total, int channels, int dtype) {
    const int64_t rows = dtype == LA_BF16
                             ? tiles_of(total, sections_of<__nv_bfloat16>(B, total, channels), kSave<__nv_bfloat16>)
                             : tiles_of(total, sections_of<float>(B, total, channels), kSave<float>);
    return ((size_t)rows + B) * channels * sizeof(float);
}

cudaError_t launch_gated_scan(const GatedScanArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? scan<__nv_bfloat16>(a, st) : scan<float>(a, st);
}

cudaError_t launch_gated_scan_backward(const GatedScanBwdArgs &a, cudaStream_t st) {
    return a.dtype == LA_BF16 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
}

}  // namespace la
