// The gated recurrence over packed sequences: kernels and host side of
// lce_recurrence_forward / _backward.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "lce_host.h"
#include "row_ring.cuh"

using namespace lce;

namespace {

constexpr int kEvery = 128;   // tokens between kept states

struct ScanArgs {
    const int32_t *cu;
    int B, T, len, d;   // len: of every sequence, without offsets
    const void *x, *g, *dh;
    const float *state, *dfinal;
    float *kept, *final, *dstate;
    void *h, *dx, *dg;
    int64_t ld_x, ld_g, ld_h, ld_dh, ld_dx, ld_dg;
    int *status;
    // first token of sequence b (b <= B), within [0, T] whatever the offsets hold
    __device__ __forceinline__ int start(int b) const { return cu ? min(max(cu[b], 0), T) : b * len; }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The state of a channel pair (bf16) or a channel (fp32), the 4 bytes of a row
// that a thread takes.
template <typename T>
struct Lane;
template <>
struct Lane<__nv_bfloat16> {
    struct F {
        float a, b;
    };
    static constexpr int kCh = 2;
    static __device__ __forceinline__ F get(uint32_t w) { return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}; }
    static __device__ __forceinline__ uint32_t put(F v) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.a, v.b);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    static __device__ __forceinline__ F all(float v) { return {v, v}; }
    static __device__ __forceinline__ F fma(F a, F b, F c) { return {fmaf(a.a, b.a, c.a), fmaf(a.b, b.b, c.b)}; }
    static __device__ __forceinline__ F mul(F a, F b) { return {a.a * b.a, a.b * b.b}; }
    static __device__ __forceinline__ F add(F a, F b) { return {a.a + b.a, a.b + b.b}; }
    static __device__ __forceinline__ float first(F v) { return v.a; }
    template <typename G>
    static __device__ __forceinline__ F each(F v, G g) { return {g(v.a), g(v.b)}; }
    static __device__ __forceinline__ F load(const float *p) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        return {v.x, v.y};
    }
    static __device__ __forceinline__ void save(float *p, F v) { *reinterpret_cast<float2 *>(p) = make_float2(v.a, v.b); }
};
template <>
struct Lane<float> {
    using F = float;
    static constexpr int kCh = 1;
    static __device__ __forceinline__ F get(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t put(F v) { return __float_as_uint(v); }
    static __device__ __forceinline__ F all(float v) { return v; }
    static __device__ __forceinline__ F fma(F a, F b, F c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ F mul(F a, F b) { return a * b; }
    static __device__ __forceinline__ F add(F a, F b) { return a + b; }
    static __device__ __forceinline__ float first(F v) { return v; }
    template <typename G>
    static __device__ __forceinline__ F each(F v, G g) { return g(v); }
    static __device__ __forceinline__ F load(const float *p) { return *p; }
    static __device__ __forceinline__ void save(float *p, F v) { *p = v; }
};

// exp(-g) = 2^z, z = -g log2(e), bounded so that neither 1 + it nor its reciprocal leaves fp32 (a NaN stays one). z's own
// rounding is off by up to |z| 2^-24, which is that share of the exponential. kExact (fp32 tensors) takes it up, with what
// log2(e) has beyond fp32, by the first term of 2^r: 5 units of 2^-24 whatever the logit, where it was 17 at logits up to 16
// and 64 up to 87; 8192 tokens of 4096 channels 67 us either way. bf16 tensors, whose results are rounded to 2^-8, do without
// (16384 tokens of 4096 channels 81 us, 92 with it; backward 138, 163).
template <typename L, bool kExact>
__device__ __forceinline__ typename L::F gate_exp(typename L::F g) {
    return L::each(g, [](float g) {
        constexpr float kHigh = 1.4426950408889634, kLow = 1.4426950408889634 - kHigh, kLn2 = 0.6931471805599453;
        if constexpr (kExact) {
            asm("max.NaN.f32 %0, %0, 0fC2AEAC4F;\n\tmin.NaN.f32 %0, %0, 0f43000000;" : "+f"(g));   // -87.33654, 128 (so r is finite)
            const float z = g * -kHigh, r = fmaf(g, -kLow, fmaf(g, -kHigh, -z)), e = ex2(z);
            return fmaf(e, r * kLn2, e);
        } else {
            float z = g * -kHigh;
            asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(z));   // 126
            return ex2(z);
        }
    });
}
// The gate and its complement
template <typename L, bool kExact>
__device__ __forceinline__ void gate(typename L::F g, typename L::F &a, typename L::F &rest) {
    const typename L::F e = gate_exp<L, kExact>(g);
    a = L::each(L::add(e, L::all(1.f)), rcp);
    rest = L::mul(e, a);
}

// What a run of tokens does to the state before it: s -> A s + H, or, where a
// sequence begins among them, just H: A is kReset then, which no product of
// gates is, so that nothing of the state before gets through, NaN or infinite.
constexpr float kReset = -1.f;
template <typename L>
struct Step {
    typename L::F A, H;
};
template <typename L>
__device__ __forceinline__ typename L::F apply(const Step<L> &s, typename L::F before) {
    return L::first(s.A) < 0.f ? s.H : L::fma(s.A, before, s.H);
}

// A product of gates, which are never zero, that ran out of fp32: its smallest value, so that an infinite state stays one
// (0 would make it a NaN). A finite state adds 2^-21 at most by it, where it is fp32's largest.
__device__ __forceinline__ float never_zero(float a) { return __uint_as_float(max(__float_as_uint(a), 1u)); }   // kReset stays, NaN too

// Work is split over channels and over time. A slice is the channels of 128
// bytes of a row; a cluster of CTAs takes a slice through the tokens, each CTA a
// tile of 128 tokens in every group of as many tiles, and 8 warps 16 tokens each
// of a tile. A warp forms its gates once, into registers, and from them what its
// tokens do to the state (a Step); the tile's Step goes to every CTA of the
// cluster through distributed shared memory, each folds those before its own
// into the state that the group began with, and the tokens are gone through once
// more from their true state. Tiles come ahead through a ring of TMA copies, with
// the places where sequences begin and end in them, which the copying warp looks
// up. The backward forms h of a tile again from the state kept before it, which
// needs no other tile, and goes through the tiles from the last.
//
// What bounds it in bf16 is a tile's way through its CTA: about 5000 cycles, of
// which the gates are 1000, the joins with their barriers and the exchange 2000,
// the asking warp's work 800 and the tokens' second time 700, and two CTAs share
// an SM: 16384 tokens of 4096 channels in 81 us (5.0 TB/s, 73% of the copy rate),
// backward 139 us (4.8 TB/s); fp32, half the channels a byte, 65 us for 8192
// tokens (6.2 TB/s, 91%). Neither its arithmetic nor its stores: without
// exponentials and reciprocals, or without stores, it takes as long. Tried: lanes
// along time, joined by shuffles alone (copies of 2 KB, partial lines: 112 us
// where this stood at 90); one reciprocal for two gates (+8%: the case of a NaN is
// a branch); pairs of channels in packed arithmetic (the same).
constexpr int kTok = kEvery, kWarps = 8, kPer = kTok / kWarps, kScanThreads = kWarps * 32;
constexpr int kTileBytes = kTok * 128, kMaxCluster = 16, kMaxStages = 3;
constexpr long long kScanWaitCycles = 2000000000LL;   // ~1 s: far above any legitimate wait

struct TileSeqs {
    uint32_t begin[kTok / 32], end[kTok / 32], dead[kTok / 32];   // bits: first tokens, last tokens, tokens of no sequence
    int seq[kTok];                                                // of the first and last tokens
};
struct ScanBars {
    uint64_t full[kMaxStages], done[kMaxStages], steps[2];
    uint32_t flags[kTok];
    TileSeqs seqs[kMaxStages + 1];   // one more than tiles: the forward gives up a tile before its sequences
};
// Steps of a warp's channels; 32 bytes apart, so that the lanes that join two warps each meet in no more banks than they must.
constexpr int kStepBytes = 32 * 16, kWarpStepBytes = kStepBytes + 32;

struct ScanMaps {
    CUtensorMap x, g, dh;
};
struct ScanGeo {
    int tiles, cluster, groups, stages;   // groups: of `cluster` tiles
};

// Steps in memory: A and H of one channel after the other
template <typename L>
__device__ __forceinline__ void save_step(uint8_t *p, const Step<L> &s) {
    if constexpr (L::kCh == 2) {
        *reinterpret_cast<float4 *>(p) = make_float4(s.A.a, s.H.a, s.A.b, s.H.b);
    } else {
        *reinterpret_cast<float2 *>(p) = make_float2(s.A, s.H);
    }
}
template <typename L>
__device__ __forceinline__ Step<L> load_step(const uint8_t *p) {
    if constexpr (L::kCh == 2) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        return Step<L>{{v.x, v.z}, {v.y, v.w}};
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        return Step<L>{v.x, v.y};
    }
}

// A channel's Steps of the warps joined in order (kDown: from the last warp), by
// the group of 8 / N neighbouring lanes that take it, N warps each: in a warp's
// place the Step of those before it; the tile's Step is returned to all of them.
template <int N, bool kDown>
__device__ __forceinline__ Step<Lane<float>> join_warps(uint8_t *at, int stride, int lane) {
    using L = Lane<float>;
    constexpr int kLanes = kWarps / N;
    auto then = [](const Step<L> &a, const Step<L> &b) {   // a, then b
        return Step<L>{b.A < 0.f ? b.A : a.A < 0.f ? a.A : never_zero(a.A * b.A), apply(b, a.H)};
    };
    const int q = kDown ? kLanes - 1 - lane % kLanes : lane % kLanes;   // place in order
    Step<L> own[N], sum;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        own[i] = load_step<L>(at + (kDown ? kWarps - 1 - (q * N + i) : q * N + i) * stride);
        sum = i == 0 ? own[0] : then(sum, own[i]);
    }
    auto from = [&](const Step<L> &s, int off) {   // of the lane `off` places before
        return kDown ? Step<L>{__shfl_down_sync(0xffffffffu, s.A, off, kLanes), __shfl_down_sync(0xffffffffu, s.H, off, kLanes)}
                     : Step<L>{__shfl_up_sync(0xffffffffu, s.A, off, kLanes), __shfl_up_sync(0xffffffffu, s.H, off, kLanes)};
    };
#pragma unroll
    for (int off = 1; off < kLanes; off *= 2) {
        const Step<L> b = from(sum, off);
        if (q >= off) sum = then(b, sum);
    }
    Step<L> before = from(sum, 1);
    if (q == 0) before = Step<L>{1.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        save_step<L>(at + (kDown ? kWarps - 1 - (q * N + i) : q * N + i) * stride, before);
        if (i + 1 < N) before = then(before, own[i]);
    }
    const int last = kDown ? 0 : kLanes - 1;
    return Step<L>{__shfl_sync(0xffffffffu, sum.A, last, kLanes), __shfl_sync(0xffffffffu, sum.H, last, kLanes)};
}

// 8 bytes to the shared memory of a CTA of the cluster, counted on a barrier there
__device__ __forceinline__ void store_remote(uint32_t addr, float a, float b, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(a), "f"(b), "r"(bar)
                 : "memory");
}

// A bounded wait of a warp; after one that gave up the warp makes no other and
// goes through the rest with whatever is there, in step with the others.
__device__ __forceinline__ void scan_wait(uint64_t *bar, uint32_t parity, bool &lost, int *status) {
    if (lost) return;
    const uint32_t at = smem_u32(bar);
    if (!mbar_try_wait(at, parity)) {
        const long long t0 = clock64();
        while (!lost && !mbar_try_wait(at, parity)) lost = clock64() - t0 > kScanWaitCycles;
        if (lost) atomicOr(status, LCE_DEV_TIMEOUT);
    }
    lost = __any_sync(0xffffffffu, lost);
}

// Where sequences begin and end in a tile, by one warp, which keeps the ends of
// 32 sequences in its registers: tiles come in order, so that it seldom has to
// look for others.
struct SeqFinder {
    const ScanArgs &a;
    uint32_t *flags;
    int live;                 // tokens of all sequences
    int lo = -1, s = 0, e = 0;   // first token of sequence lo + lane, and the one behind its last
    __device__ __forceinline__ SeqFinder(const ScanArgs &a_, uint32_t *f) : a(a_), flags(f), live(a_.cu ? a_.start(a_.B) : a_.T) {}

    __device__ __forceinline__ void take(int from) {
        const int mine = from + (threadIdx.x & 31);
        s = mine < a.B ? a.start(mine) : a.T, e = mine < a.B ? a.start(mine + 1) : a.T;
    }
    __device__ __forceinline__ bool holds(int t0) const {   // all sequences with tokens in the tile
        return lo >= 0 && __shfl_sync(0xffffffffu, s, 0) <= t0 && (lo + 32 >= a.B || __shfl_sync(0xffffffffu, e, 31) >= t0 + kTok);
    }
    __device__ __forceinline__ void mark(int from, int t0, TileSeqs &out) const {
        const int mine = from + (threadIdx.x & 31);
        if (mine >= a.B || e <= s) return;
        if (s >= t0 && s < t0 + kTok) out.seq[s - t0] = mine, atomicOr(&flags[s - t0], 1u);
        if (e > t0 && e <= t0 + kTok) out.seq[e - 1 - t0] = mine, atomicOr(&flags[e - 1 - t0], 2u);
    }
    // The last sequence that does not begin after t, among 32 probes a round
    __device__ __forceinline__ int last_at(int t) const {
        const int lane = threadIdx.x & 31;
        int b = 0, n = a.B + 1;
        while (n > 1) {
            const int step = (n + 31) / 32, off = lane * step;
            const uint32_t mask = __ballot_sync(0xffffffffu, off < n && a.start(b + off) <= t);
            const int hit = mask ? 31 - __clz(mask) : 0;   // offsets that do not ascend may leave holes
            b += hit * step;
            n = min(step, n - hit * step);
        }
        return b;
    }
    // The ends of the tile from t0 on. Most tiles have none, and all warps wait
    // for the one that looks: that is settled first (16384 tokens of 4096 channels
    // bf16: 84 us with the full account of every tile, 81 this way).
    template <bool kBack>
    __device__ __forceinline__ void operator()(int t0, TileSeqs &out) {
        const int lane = threadIdx.x & 31;
        bool plain;   // within one sequence, neither its first token nor its last among them
        if (a.cu) {
            plain = holds(t0) && t0 + kTok <= live &&
                    !__any_sync(0xffffffffu, e > s && ((s >= t0 && s < t0 + kTok) || (e > t0 && e <= t0 + kTok)));
        } else {
            const int at = t0 % a.len;
            plain = at > 0 && at + kTok < a.len;
        }
        if (plain) {
            if (lane < kTok / 32) out.begin[lane] = out.end[lane] = out.dead[lane] = 0;
            return;
        }
        if (!a.cu) {
#pragma unroll
            for (int k = 0; k < kTok / 32; ++k) {
                const int t = t0 + 32 * k + lane;
                const bool live = t < a.T;
                const int b = live ? t / a.len : 0, at = t - b * a.len;
                const uint32_t begin = __ballot_sync(0xffffffffu, live && at == 0), end = __ballot_sync(0xffffffffu, live && at == a.len - 1),
                               dead = __ballot_sync(0xffffffffu, !live);
                out.seq[32 * k + lane] = b;
                if (lane == 0) out.begin[k] = begin, out.end[k] = end, out.dead[k] = dead;
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < kTok / 32; ++k) flags[32 * k + lane] = 0;
        __syncwarp();
        if (holds(t0)) {
            mark(lo, t0, out);
        } else {
            int b = last_at(t0);
            lo = kBack ? max(0, b - 15) : b;   // the tiles to come are on that side
            take(lo);
            if (holds(t0)) {
                mark(lo, t0, out);
            } else {
                lo = -1;
                while (b < a.B) {
                    take(b);
                    mark(b, t0, out);
                    if (__any_sync(0xffffffffu, s >= t0 + kTok)) break;
                    // where all are empty there may be millions, and the other warps wait: on to the last that begins there
                    const bool some = __any_sync(0xffffffffu, e > s);
                    const int here = __shfl_sync(0xffffffffu, s, 0);
                    b += 32;
                    if (!some) b = max(b, last_at(here));
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kTok / 32; ++k) {
            const uint32_t f = flags[32 * k + lane];
            const uint32_t begin = __ballot_sync(0xffffffffu, f & 1), end = __ballot_sync(0xffffffffu, f & 2),
                           dead = __ballot_sync(0xffffffffu, t0 + 32 * k + lane >= live);
            if (lane == 0) out.begin[k] = begin & ~dead, out.end[k] = end & ~dead, out.dead[k] = dead;
        }
    }
};

// The states of empty sequences pass through; a warp of every CTA takes its share of the sequences.
template <typename L>
__device__ __forceinline__ void empty_seqs(const ScanArgs &a, int rank, int cluster, int ch0, const float *from, float *to) {
    if (!to || (!a.cu && a.len > 0)) return;
    const int lane = threadIdx.x & 31, ch = ch0 + lane * L::kCh;
    for (int b = rank * 32; b < a.B; b += cluster * 32) {
        const int mine = b + lane;
        uint32_t mask = __ballot_sync(0xffffffffu, mine < a.B && a.start(mine + 1) <= a.start(mine));
        for (; mask; mask &= mask - 1) {
            const int64_t at = static_cast<int64_t>(b + __ffs(mask) - 1) * a.d + ch;
            if (ch < a.d) L::save(to + at, from ? L::load(from + at) : L::all(0.f));
        }
    }
}

__device__ __forceinline__ void check_offsets(const ScanArgs &a) {   // one warp
    if (!a.cu) return;
    bool bad = false;
    for (int b = threadIdx.x & 31; b <= a.B; b += 32) bad |= b == 0 ? a.cu[0] != 0 : a.cu[b] < a.cu[b - 1] || a.cu[b] > a.T;
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) atomicOr(a.status, LCE_DEV_SEQLENS);
}

template <typename T, bool kBack>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan(const ScanArgs a, const ScanGeo geo, const __grid_constant__ ScanMaps maps) {
    using L = Lane<T>;
    using F = typename L::F;
    constexpr bool kExact = sizeof(T) == 4;
    constexpr int kStageBytes = (kBack ? 3 : 2) * kTileBytes, kSlice = 32 * L::kCh;
    extern __shared__ __align__(128) uint8_t ring[];   // tiles of x, g (and dh); the warps' steps; the cluster's
    __shared__ ScanBars sm;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    const int rank = geo.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int ch0 = static_cast<int>(blockIdx.x) / geo.cluster * kSlice;
    if (threadIdx.x == 0) {
        for (int i = 0; i < geo.stages; ++i) mbar_init(&sm.full[i], 2), mbar_init(&sm.done[i], kWarps);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.steps[i], 1);
        fence_mbar_init();
    }
    if (geo.cluster > 1) cluster_sync_all();
    else __syncthreads();
    bool lost = false;
    // the tile of a group, or none (in the last group); tiles are asked for by the warp that has the least to do else
    auto tile_of = [&](int group) {
        const int i = group * geo.cluster + rank;
        return i >= geo.tiles ? -1 : kBack ? geo.tiles - 1 - i : i;
    };
    const bool asks = warp == (kBack ? kWarps - 1 : 0);
    SeqFinder find(a, sm.flags);
    int asked = 0, ask_stage = 0, ask_slot = 0;
    auto ask = [&]() {
        const int tile = asked < geo.groups ? tile_of(asked) : -1;
        if (tile < 0) return;
        if (lane == 0) {
            uint8_t *dst = ring + ask_stage * kStageBytes;
            uint64_t *bar = &sm.full[ask_stage];
            mbar_arrive_expect_tx(bar, kStageBytes);
            tma_load_2d(dst, &maps.x, bar, ch0, tile * kTok);
            tma_load_2d(dst + kTileBytes, &maps.g, bar, ch0, tile * kTok);
            if (kBack) tma_load_2d(dst + 2 * kTileBytes, &maps.dh, bar, ch0, tile * kTok);
        }
        find.template operator()<kBack>(tile * kTok, sm.seqs[ask_slot]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[ask_stage]);
        ++asked;
        if (++ask_stage == geo.stages) ask_stage = 0;
        if (++ask_slot > geo.stages) ask_slot = 0;
    };
    if (asks)
        for (int i = 0; i < geo.stages; ++i) ask();
    uint8_t *steps = ring + geo.stages * kStageBytes, *steps_b = steps + kWarps * kWarpStepBytes;   // of the warps; (backward) the gradient's
    uint8_t *tile_steps = steps + (kBack ? 2 : 1) * kWarps * kWarpStepBytes;                          // of the cluster's tiles, [parity][rank]
    const int ch = ch0 + lane * L::kCh;
    const uint32_t lane_bytes = ch * sizeof(T);
    const bool in = ch < a.d;
    F carry = L::all(0.f);   // the state before the group, or (backward) the gradient that comes from behind it
    int s = 0, slot = 0;
    uint32_t phase = 0;
    for (int group = 0; group < geo.groups; ++group) {
        const int tile = tile_of(group), par = group & 1;
        const bool have = tile >= 0;
        const uint8_t *xs = ring + s * kStageBytes + warp * kPer * 128 + lane * 4, *gs = xs + kTileBytes, *ds = gs + kTileBytes;
        auto word = [](const uint8_t *p, int i) { return *reinterpret_cast<const uint32_t *>(p + i * 128); };
        const TileSeqs &seqs = sm.seqs[slot];
        const int *seq = seqs.seq + warp * kPer;
        uint32_t begin = 0, end = 0, dead = 0;
        F av[kPer], v[kPer];   // gates; what a token adds to the state, in the backward later h_{t-1} - x_t
        Step<L> fwd{L::all(1.f), L::all(0.f)}, bwd{L::all(1.f), L::all(0.f)};
        F before = L::all(0.f);   // (backward) the state before the tile
        auto state = [&](const float *p, int i) {
            return p && in ? L::load(p + static_cast<int64_t>(seq[i]) * a.d + ch) : L::all(0.f);
        };
        // what to do at a token, for a warp with and without the ends of sequences among its tokens
        auto at = [](uint32_t bits, int i) { return (bits >> i & 1u) != 0; };
        auto gates = [&](auto special) {
            constexpr bool kSpecial = decltype(special)::value;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                F rest;
                gate<L, kExact>(L::get(word(gs, i)), av[i], rest);
                v[i] = L::mul(rest, L::get(word(xs, i)));
                if (kSpecial && at(dead, i)) av[i] = v[i] = L::all(0.f);
                if (kSpecial && at(begin, i)) v[i] = L::fma(av[i], state(a.state, i), v[i]);
                if (kSpecial && at(begin | dead, i)) fwd.A = L::all(kReset), fwd.H = v[i];
                else {
                    fwd.H = L::fma(av[i], fwd.H, v[i]);
                    if (!kSpecial || !(L::first(fwd.A) < 0.f)) fwd.A = L::mul(fwd.A, av[i]);
                }
            }
            if constexpr (kBack) {
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i) {
                    F l = L::get(word(ds, i));
                    if (kSpecial && at(dead, i)) l = L::all(0.f);
                    if (kSpecial && at(end, i)) l = L::add(l, state(a.dfinal, i));
                    if (kSpecial && at(end | dead, i)) bwd.A = L::all(kReset), bwd.H = L::mul(av[i], l);
                    else {
                        bwd.H = L::mul(av[i], L::add(l, bwd.H));
                        if (!kSpecial || !(L::first(bwd.A) < 0.f)) bwd.A = L::mul(bwd.A, av[i]);
                    }
                }
            }
        };
        if (have) {
            if (kBack && in) before = L::load(a.kept + static_cast<int64_t>(tile) * a.d + ch);
            scan_wait(&sm.full[s], phase, lost, a.status);
            const int sh = warp % 2 * kPer;
            begin = seqs.begin[warp / 2] >> sh & 0xffffu;
            end = seqs.end[warp / 2] >> sh & 0xffffu;
            dead = seqs.dead[warp / 2] >> sh & 0xffffu;
            if (begin | end | dead) gates(std::true_type());
            else gates(std::false_type());
        }
        constexpr int kLaneStep = L::kCh * 8;
        fwd.A = L::each(fwd.A, never_zero);
        save_step(steps + warp * kWarpStepBytes + lane * kLaneStep, fwd);
        if (kBack) bwd.A = L::each(bwd.A, never_zero), save_step(steps_b + warp * kWarpStepBytes + lane * kLaneStep, bwd);
        __syncthreads();
        uint8_t *theirs = tile_steps + par * geo.cluster * kStepBytes;
        {
            constexpr int kLanes = 8 / L::kCh;   // that take a channel
            const int at = threadIdx.x / kLanes * 8;
            Step<Lane<float>> all = join_warps<L::kCh, false>(steps + at, kWarpStepBytes, lane);
            if (kBack) all = join_warps<L::kCh, true>(steps_b + at, kWarpStepBytes, lane);
            if (geo.cluster > 1) {
                uint64_t *bar = &sm.steps[par];
                if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, geo.cluster * 32 * kLaneStep);
                for (int to = lane % kLanes; to < geo.cluster; to += kLanes)
                    store_remote(map_to_cta(smem_u32(theirs + rank * kStepBytes + at), to), all.A, all.H, map_to_cta(smem_u32(bar), to));
            } else if (lane % kLanes == 0) {
                save_step<Lane<float>>(theirs + at, all);
            }
        }
        __syncthreads();
        if (kBack && have) {   // h again, from the state before the tile
            F h = apply(load_step<L>(steps + warp * kWarpStepBytes + lane * kLaneStep), before);
            auto again = [&](auto special) {
                constexpr bool kSpecial = decltype(special)::value;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const F from = kSpecial && at(begin, i) ? state(a.state, i) : h;
                    h = kSpecial && at(begin | dead, i) ? v[i] : L::fma(av[i], h, v[i]);
                    v[i] = L::fma(L::get(word(xs, i)), L::all(-1.f), from);
                }
            };
            if (begin | dead) again(std::true_type());
            else again(std::false_type());
        }
        // (forward: every warp has its gates and is through with the group before)
        if (!kBack && asks && !lost) ask();
        F c = carry;
        if (geo.cluster > 1) scan_wait(&sm.steps[par], group >> 1 & 1, lost, a.status);
        for (int r = 0; r < geo.cluster; ++r) {
            if (r == rank) c = carry;
            carry = apply(load_step<L>(theirs + r * kStepBytes + lane * kLaneStep), carry);
        }
        if (!kBack && a.kept && have && warp == 0 && in) L::save(a.kept + static_cast<int64_t>(tile) * a.d + ch, c);
        c = apply(load_step<L>((kBack ? steps_b : steps) + warp * kWarpStepBytes + lane * kLaneStep), c);
        if (!have) continue;
        const int t0 = tile * kTok + warp * kPer;
        auto rows = [&](void *p, int64_t ld) { return static_cast<uint8_t *>(p) + t0 * ld * sizeof(T); };
        auto put = [&](uint8_t *p, F value) { *reinterpret_cast<uint32_t *>(p + lane_bytes) = L::put(value); };
        auto out = [&](auto special) {
            constexpr bool kSpecial = decltype(special)::value;
            if (!kBack) {
                uint8_t *h = rows(a.h, a.ld_h);
#pragma unroll
                for (int i = 0; i < kPer; ++i, h += a.ld_h * sizeof(T)) {
                    c = kSpecial && at(begin | dead, i) ? v[i] : L::fma(av[i], c, v[i]);
                    if (!kSpecial || t0 + i < a.T) put(h, c);
                    if (kSpecial && at(end, i) && a.final) L::save(a.final + static_cast<int64_t>(seq[i]) * a.d + ch, c);
                }
            } else {
                uint8_t *x = rows(a.dx, a.ld_dx) + (kPer - 1) * a.ld_dx * sizeof(T), *g = rows(a.dg, a.ld_dg) + (kPer - 1) * a.ld_dg * sizeof(T);
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i, x -= a.ld_dx * sizeof(T), g -= a.ld_dg * sizeof(T)) {
                    const F rest = L::mul(gate_exp<L, kExact>(L::get(word(gs, i))), av[i]);
                    F l = L::get(word(ds, i));
                    l = L::add(l, kSpecial && at(end, i) ? state(a.dfinal, i) : c);
                    F dx = L::mul(rest, l), dg = L::mul(L::mul(l, v[i]), L::mul(av[i], rest));
                    c = L::mul(av[i], l);
                    if (kSpecial && at(dead, i)) dx = dg = c = L::all(0.f);
                    if (!kSpecial || t0 + i < a.T) put(x, dx), put(g, dg);
                    if (kSpecial && at(begin, i) && a.dstate) L::save(a.dstate + static_cast<int64_t>(seq[i]) * a.d + ch, c);
                }
            }
        };
        if (in) {
            if (begin | end | dead) out(std::true_type());
            else out(std::false_type());
        }
        if (kBack) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.done[s]);
            if (asks) {
                scan_wait(&sm.done[s], phase, lost, a.status);
                if (!lost) ask();
            }
        }
        if (++s == geo.stages) s = 0, phase ^= 1;
        if (++slot > geo.stages) slot = 0;
    }
    if (asks) {
        empty_seqs<L>(a, rank, geo.cluster, ch0, kBack ? a.dfinal : a.state, kBack ? a.dstate : a.final);
        if (blockIdx.x == 0) check_offsets(a);
        // copies in flight have to land before the CTA gives up its memory (all have, unless a wait gave up)
        for (int i = min(asked, geo.stages); lost && i > 0; --i) {
            const int k = asked - i;   // the group asked for, in stage k % stages, in its (k / stages)th use
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(&sm.full[k % geo.stages]), k / geo.stages & 1) && clock64() - t0 < kScanWaitCycles / 10) {}
        }
    }
    if (geo.cluster > 1) cluster_sync_all();   // no CTA leaves while another may write to its shared memory
}

// One token of every sequence: no scan. A thread takes 8 channels of a sequence.
template <typename T>
__global__ void __launch_bounds__(256) k_scan_step(const ScanArgs a) {
    const int per = a.d / kVec, id = blockIdx.x * 256 + threadIdx.x;
    const int64_t b = id / per;
    const int ch = (id - static_cast<int>(b) * per) * kVec;
    if (b >= a.B) return;
    float g[kVec], x[kVec], h[kVec];
    load_pack(static_cast<const T *>(a.g) + b * a.ld_g + ch).get(g);
    load_pack(static_cast<const T *>(a.x) + b * a.ld_x + ch).get(x);
#pragma unroll
    for (int i = 0; i < kVec; ++i) h[i] = 0.f;
    if (a.state) load_pack(a.state + b * a.d + ch).get(h);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        float f, rest;
        gate<Lane<float>, sizeof(T) == 4>(g[i], f, rest);
        h[i] = fmaf(f, h[i], rest * x[i]);
    }
    store_pack(static_cast<T *>(a.h) + b * a.ld_h + ch, h);
    if (a.final) store_pack(a.final + b * a.d + ch, h);
    if (!a.kept) return;
    if ((b + 1) % kEvery == 0 && b + 1 < a.T) store_pack(a.kept + (b + 1) / kEvery * a.d + ch, h);
    if (b == 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[i] = 0.f;
        store_pack(a.kept + ch, h);
    }
}

lce_status_t check_rows(const void *p, int64_t ld, int64_t d, int elt) {
    if (!p) return LCE_ERR_NULL;
    if (ld < 0 || ld >= (int64_t(1) << 36) || (ld && ld < d)) return LCE_ERR_SHAPE;
    return host_misaligned(p) || (ld * elt) % 16 ? LCE_ERR_ALIGN : LCE_OK;
}

lce_status_t check_scan(const lce_recurrence_t *a, bool backward) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->T < 0 || a->T >= (int64_t(1) << 30) || a->B < 1 || a->B >= (int64_t(1) << 30) || a->d < 8 || a->d >= (1 << 24)) return LCE_ERR_SHAPE;
    if (a->d % 8) return LCE_ERR_ALIGN;
    if (!a->cu && a->T % a->B) return LCE_ERR_SHAPE;
    for (const float *p : {a->state, static_cast<const float *>(a->kept), static_cast<const float *>(a->final), a->dfinal,
                           static_cast<const float *>(a->dstate)})
        if (host_misaligned(p)) return LCE_ERR_ALIGN;
    if (a->T == 0) return LCE_OK;
    if (backward && !a->kept) return LCE_ERR_NULL;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    const struct { const void *p; int64_t ld; bool used; } all[] = {{a->x, a->ld_x, true}, {a->g, a->ld_g, true}, {a->h, a->ld_h, !backward},
        {a->dh, a->ld_dh, backward}, {a->dx, a->ld_dx, backward}, {a->dg, a->ld_dg, backward}};
    for (const auto &t : all) {
        if (!t.used) continue;
        const lce_status_t s = check_rows(t.p, t.ld, a->d, elt);
        if (s != LCE_OK) return s;
    }
    return LCE_OK;
}

ScanArgs make_args(const lce_recurrence_t *a, const HostDev &dev) {
    ScanArgs r{};
    auto ld = [&](int64_t v) { return v ? v : a->d; };
    r.cu = a->cu, r.B = static_cast<int>(a->B), r.T = static_cast<int>(a->T), r.len = static_cast<int>(a->T / a->B);
    r.d = static_cast<int>(a->d);
    r.x = a->x, r.g = a->g, r.dh = a->dh, r.state = a->state, r.dfinal = a->dfinal;
    r.kept = a->kept, r.final = a->final, r.dstate = a->dstate, r.h = a->h, r.dx = a->dx, r.dg = a->dg;
    r.ld_x = ld(a->ld_x), r.ld_g = ld(a->ld_g), r.ld_h = ld(a->ld_h), r.ld_dh = ld(a->ld_dh), r.ld_dx = ld(a->ld_dx), r.ld_dg = ld(a->ld_dg);
    r.status = dev.status;
    return r;
}

lce_status_t encode(CUtensorMap *m, const HostDev &dev, const void *p, bool bf16, int64_t T, int64_t d, int64_t ld) {
    const int elt = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * elt};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elt), static_cast<cuuint32_t>(kTok)}, es[2] = {1, 1};
    const CUresult r = dev.encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(p), dims,
                                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? LCE_OK : LCE_ERR_SHAPE;
}

// Two CTAs an SM; the ring takes what the steps leave of half its shared memory.
constexpr int kScanBytes = 112 * 1024;
constexpr int kMostScanBytes = 200 * 1024;   // two stages and the steps of the largest cluster

template <typename T, bool kBack>
lce_status_t launch_scan(const ScanArgs &r, const HostDev &dev, cudaStream_t st) {
    constexpr bool kBf16 = sizeof(T) == 2;
    constexpr int kStageBytes = (kBack ? 3 : 2) * kTileBytes, kSlice = 128 / sizeof(T);
    ScanMaps maps{};
    lce_status_t s = LCE_OK;
    if (r.T > 0) {
        s = encode(&maps.x, dev, r.x, kBf16, r.T, r.d, r.ld_x);
        if (s == LCE_OK) s = encode(&maps.g, dev, r.g, kBf16, r.T, r.d, r.ld_g);
        if (s == LCE_OK && kBack) s = encode(&maps.dh, dev, r.dh, kBf16, r.T, r.d, r.ld_dh);
        if (s != LCE_OK) return s;
    }
    ScanGeo geo;
    geo.tiles = (r.T + kTok - 1) / kTok;
    const int slices = (r.d + kSlice - 1) / kSlice;
    // As many CTAs as find room at once, two on an SM where their memory allows it. The most of a group's time is the way of
    // a tile through its CTA, so more of them at once pay until they contend; clusters of 16 have more to wait for and pay
    // only where they leave SMs free (bf16: 16384 tokens of 4096 channels, clusters of 2, 4 and 8: 121, 85 and 97 us; 8192 of
    // 2048: 64, 35 and 28, of 16: 46; 4096 of 1024, of 8 and 16: 16 and 21; 65536 of 1024: 168 and 161).
    auto step_bytes = [](int cluster) { return (kBack ? 2 : 1) * kWarps * kWarpStepBytes + 2 * cluster * kStepBytes; };
    auto stages = [&](int cluster) { return (kScanBytes - static_cast<int>(sizeof(ScanBars)) - step_bytes(cluster)) / kStageBytes; };
    geo.cluster = 1;
    while (geo.cluster < kMaxCluster && geo.cluster < geo.tiles &&
           slices * geo.cluster * 2 <= (geo.cluster == 8 || stages(geo.cluster * 2) < 2 ? 1 : 2) * dev.sms)
        geo.cluster *= 2;
    geo.groups = (geo.tiles + geo.cluster - 1) / geo.cluster;
    const int steps = step_bytes(geo.cluster);
    geo.stages = std::max(2, std::min(kMaxStages, stages(geo.cluster)));
    const int smem = geo.stages * kStageBytes + steps;
    constexpr auto kernel = k_scan<T, kBack>;
    if ((s = host_smem<kernel>(dev, kMostScanBytes)) != LCE_OK) return s;
    if (geo.cluster > 8) {
        static std::atomic<uint64_t> done{0};
        const uint64_t bit = uint64_t(1) << dev.index;
        if (!(done.load(std::memory_order_relaxed) & bit)) {
            s = host_cuda(cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
            if (s != LCE_OK) return s;
            done.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(geo.cluster), attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(slices * geo.cluster));
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    s = host_cuda(cudaLaunchKernelEx(&cfg, kernel, r, geo, maps));
    return s != LCE_OK ? s : host_launched();
}

template <typename T>
lce_status_t forward(const ScanArgs &r, const HostDev &dev, cudaStream_t st) {
    if (!r.cu && r.len == 1 && static_cast<int64_t>(r.B) * r.d <= (int64_t(1) << 30)) {
        k_scan_step<T><<<static_cast<unsigned>((static_cast<int64_t>(r.B) * (r.d / kVec) + 255) / 256), 256, 0, st>>>(r);
        return host_launched();
    }
    return launch_scan<T, false>(r, dev, st);
}

}  // namespace

extern "C" {

lce_status_t lce_recurrence_forward(const lce_recurrence_t *a) {
    lce_status_t s = check_scan(a, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    const ScanArgs r = make_args(a, dev);
    return a->dtype == LCE_BF16 ? forward<__nv_bfloat16>(r, dev, st) : forward<float>(r, dev, st);
}

lce_status_t lce_recurrence_backward(const lce_recurrence_t *a) {
    lce_status_t s = check_scan(a, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    const ScanArgs r = make_args(a, dev);
    return a->dtype == LCE_BF16 ? launch_scan<__nv_bfloat16, true>(r, dev, st) : launch_scan<float, true>(r, dev, st);
}

}  // extern "C"
