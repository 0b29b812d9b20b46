// Attention over packed sequences: what every kernel of it shares. Arguments,
// the map from a tile slot to its sequence, and the backward's row statistics.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "tc_ptx.cuh"

namespace lce {

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr int kDevSeqlens = 4;   // LCE_DEV_SEQLENS
constexpr int kDevTimeout = 2;   // LCE_DEV_TIMEOUT

// Token ranges of the sequences of one side. Without offsets every sequence
// has `len` tokens. Sequence number B is the tail: the tokens after cu[B],
// which belong to no sequence and see an empty other side.
struct SeqMap {
    const int *cu;
    int B, T, len;
    __device__ __forceinline__ int raw(int b) const { return cu ? cu[b] : b * len; }
    // first token of sequence b (b <= B), within [0, T] whatever the offsets hold
    __device__ __forceinline__ int start(int b) const { return min(max(raw(b), 0), T); }
};

// Tile t of sequence b has the slot start(b)/TILE + b + t. Slots of different
// sequences never meet (a sequence of L tokens from s on has at most
// (s+L)/TILE - s/TILE + 1 tiles), so a tile finds its sequence by searching
// one ascending function of the offsets and no tile list has to be built
// first; at most B+1 slots are empty.
__host__ __device__ inline int64_t seq_slots(int64_t T, int64_t B, int tile) { return T / tile + B + 1; }
template <int TILE>
__device__ __forceinline__ int slot_base(const SeqMap &m, int b) {
    return m.start(b) / TILE + b;
}

struct AttnArgs {
    const void *q, *k, *v, *o_in, *dO;
    void *o, *dq, *dk, *dv;
    float *lse;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs, dO_ts, dO_hs, dq_ts, dq_hs, dk_ts, dk_hs, dv_ts, dv_hs;
    SeqMap sq, sk;
    int Hq, Hk, group, D;
    int causal, pair_heads;    // pair_heads (tensor-core forward): a piece of work is two heads of a key head, else two tiles of rows
    float scale, scale_log2;   // scale, scale * log2(e)
    // backward: per query slot row, -lse * log2(e) (-inf where the row takes no
    // part) and -delta, both negative so that they are added; [Hq][slots * TILE]
    float *nlse2, *ndelta;
    int64_t stat_stride;       // slots * TILE
    // tensor-core kernels. Backward: a key head's query heads in `split` shares, whose sums of dV and dK go to
    // part[share][2][Tk][Hk][D]. Forward: a row's keys in `split` ranges, whose o goes to part[range][Tq][Hq][D] and
    // whose lse lies after them, [range][Hq][Tq].
    int split;
    float *part;
    int *status;
};

// One tile of one side: its sequence, its row range on both sides.
struct TileInfo {
    int b;             // sequence
    int s0, len;       // first token and length of the sequence on the tile's own side
    int t0;            // first row of the tile within the sequence
    int o0, olen;      // first token and length of the sequence on the other side (tail: empty)
};

// Starts of the sequences lo + lane of both sides (the last token past B): what
// the last step of a search needs.
struct SeqStarts {
    int lo, n;        // sequences lo .. lo + n - 1 may be the one, n <= 31
    int own, other;
};
__device__ __forceinline__ SeqStarts load_starts(const SeqMap &own, const SeqMap &other, int lo, int n) {
    const int lane = threadIdx.x & 31, b = lo + lane;
    const bool in = lane <= n && b <= own.B;
    return SeqStarts{lo, n, in ? own.start(b) : own.T, in ? other.start(b) : other.T};
}

// The tile of `slot` among the sequences of `st`: the largest b with
// slot_base(b) <= slot. No memory is read.
template <int TILE>
__device__ __forceinline__ TileInfo tile_among(const SeqMap &own, const SeqMap &other, const SeqStarts &st, int slot) {
    const int lane = threadIdx.x & 31, b = st.lo + lane;
    const unsigned mask = __ballot_sync(0xffffffffu, lane < st.n && b <= own.B && st.own / TILE + b <= slot);
    const int hit = mask ? 31 - __clz(mask) : 0;
    TileInfo t;
    t.b = st.lo + hit;
    t.s0 = __shfl_sync(0xffffffffu, st.own, hit);
    t.o0 = __shfl_sync(0xffffffffu, st.other, hit);
    // the end: the next sequence's start, or (the tail) the last token
    const int e = __shfl_sync(0xffffffffu, st.own, (hit + 1) & 31), oe = __shfl_sync(0xffffffffu, st.other, (hit + 1) & 31);
    const bool tail = t.b >= own.B;
    t.len = (tail ? own.T : max(e, t.s0)) - t.s0;
    t.olen = tail ? 0 : max(oe, t.o0) - t.o0;
    t.t0 = (slot - (t.s0 / TILE + t.b)) * TILE;
    return t;
}

constexpr int kFewSeqs = 30;   // sequences whose starts, and the tail's, fit one load by a warp

// The tile of `slot`: its sequence is the largest b in [0, B] with
// slot_base(b) <= slot. All 32 lanes take part, each probing one of 32 points
// of what is left, so 1024 sequences take two rounds of loads; the last 31
// sequences' starts then say everything.
template <int TILE>
__device__ __forceinline__ TileInfo tile_info(const SeqMap &own, const SeqMap &other, int slot) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = own.B + 1;
    while (n > kFewSeqs + 1) {
        const int step = (n + 31) / 32;
        const int off = lane * step;
        const bool le = off < n && slot_base<TILE>(own, lo + off) <= slot;
        const unsigned mask = __ballot_sync(0xffffffffu, le);
        // offsets that do not ascend may leave holes; the highest hit is still inside [lo, lo + n)
        const int hit = mask ? 31 - __clz(mask) : 0;
        lo += hit * step;
        n = min(step, n - hit * step);
        if (step == 1) break;
    }
    return tile_among<TILE>(own, other, load_starts(own, other, lo, n), slot);
}

// The same for a warp that looks for many tiles: a few sequences' starts are
// kept in its registers.
template <int TILE>
struct TileFinder {
    const SeqMap &q, &k;
    SeqStarts st;
    __device__ __forceinline__ TileFinder(const SeqMap &q_, const SeqMap &k_) : q(q_), k(k_), st(load_starts(q_, k_, 0, min(q_.B, kFewSeqs) + 1)) {}
    __device__ __forceinline__ TileInfo of_q(int slot) const {
        return q.B <= kFewSeqs ? tile_among<TILE>(q, k, st, slot) : tile_info<TILE>(q, k, slot);
    }
    __device__ __forceinline__ TileInfo of_k(int slot) const {
        return q.B <= kFewSeqs ? tile_among<TILE>(k, q, SeqStarts{0, st.n, st.other, st.own}, slot) : tile_info<TILE>(k, q, slot);
    }
};

// Offsets must ascend from 0 within the tokens; one warp of one block looks.
__device__ __forceinline__ void check_offsets(const SeqMap &m, int *status) {
    if (!m.cu) return;
    bool bad = false;
    for (int b = threadIdx.x & 31; b <= m.B; b += 32) {
        const int v = m.cu[b];
        bad |= b == 0 ? v != 0 : v < m.cu[b - 1];
        bad |= v > m.T;
    }
    if (bad) atomicOr(status, kDevSeqlens);
}

// dot product of 16 bytes of each
__device__ __forceinline__ float dot16(const float4 &a, const float4 &b) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}
__device__ __forceinline__ float dot16(const uint4 &a, const uint4 &b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
        s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
    }
    return s;
}

constexpr int kJoinThreads = 256;

// dV (blockIdx.y = 0) and dK from the shares' sums, added in order: 16 threads
// a row of a head. Bounded by latency (the sums lie in L2).
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const AttnArgs a) {
    griddep_wait();   // launched early
    const unsigned i = blockIdx.x * kJoinThreads + threadIdx.x, row = i / 16, c = i % 16 * 8;
    const unsigned tok = row / a.Hk, h = row % a.Hk;
    if (tok >= static_cast<unsigned>(a.sk.T) || c >= static_cast<unsigned>(a.D)) return;
    const int64_t each = static_cast<int64_t>(a.sk.T) * a.Hk * a.D;
    const float *p = a.part + blockIdx.y * each + static_cast<int64_t>(row) * a.D + c;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < a.split; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(p + k * 2 * each), y = *reinterpret_cast<const float4 *>(p + k * 2 * each + 4);
        s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
    }
    __nv_bfloat162 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __floats2bfloat162_rn(s[2 * k], s[2 * k + 1]);
    __nv_bfloat16 *out = blockIdx.y ? static_cast<__nv_bfloat16 *>(a.dk) + tok * a.dk_ts + h * a.dk_hs
                                    : static_cast<__nv_bfloat16 *>(a.dv) + tok * a.dv_ts + h * a.dv_hs;
    *reinterpret_cast<uint4 *>(out + c) = *reinterpret_cast<const uint4 *>(v);
}

// The forward's o and lse from its ranges': with lse = log sum exp(lse_k),
// o = sum exp(lse_k - lse) o_k, added in order. 16 threads a row of a head.
__global__ void __launch_bounds__(kJoinThreads) k_attn_merge(const AttnArgs a) {
    griddep_wait();   // launched early
    const int64_t row = (static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x) / 16, tok = row / a.Hq;
    const int h = static_cast<int>(row % a.Hq), c = threadIdx.x % 16 * 8;
    if (tok >= a.sq.T || c >= a.D) return;
    const int64_t each = static_cast<int64_t>(a.sq.T) * a.Hq;
    const float *p = a.part + row * a.D + c, *l = a.part + a.split * each * a.D + h * static_cast<int64_t>(a.sq.T) + tok;
    float m = -INFINITY, sum = 0.f;
    for (int k = 0; k < a.split; ++k) m = fmaxf(m, l[k * each]);   // passes a NaN by, which its weight brings back
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < a.split; ++k) {
        const float v = l[k * each];
        if (v == -INFINITY) continue;   // nothing was written
        const float w = exp2f((v - m) * kAttnLog2e);
        const float4 x = *reinterpret_cast<const float4 *>(p + k * each * a.D), y = *reinterpret_cast<const float4 *>(p + k * each * a.D + 4);
        const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        sum += w;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(w, z[i], s[i]);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;   // a row without keys: zeros
    __nv_bfloat162 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __floats2bfloat162_rn(s[2 * k] * inv, s[2 * k + 1] * inv);
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + tok * a.o_ts + h * a.o_hs + c) = *reinterpret_cast<const uint4 *>(v);
    if (c == 0) a.lse[h * static_cast<int64_t>(a.sq.T) + tok] = sum != 0.f ? m + logf(sum) : -INFINITY;
}

constexpr int kStatThreads = 256;

// Row statistics of the backward, by slot: delta_i = dO_i . o_i in fp32 and
// lse_i in base 2, both negated, so that the gradient kernels read aligned rows
// of TILE values and add them. Rows without an allowed key (lse = -inf) and rows
// past a sequence's end get -inf: their probabilities come out as 2^-inf = 0.
// LPR lanes take a row, 16 bytes each; a thread asks for all its rows before it
// adds any up, since the kernel is nothing but waits for memory.
template <typename T, int TILE, int LPR>
__global__ void __launch_bounds__(kStatThreads) k_attn_stats(const AttnArgs a) {
    using V = typename std::conditional<sizeof(T) == 4, float4, uint4>::type;
    constexpr int kRows = kStatThreads / LPR;   // rows at once
    constexpr int kTurns = TILE / kRows;
    const int h = blockIdx.x % a.Hq;
    const int slot = blockIdx.x / a.Hq;
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        check_offsets(a.sq, a.status);
        check_offsets(a.sk, a.status);
    }
    const TileInfo t = tile_info<TILE>(a.sq, a.sk, slot);
    const int r0 = threadIdx.x / LPR, piece = threadIdx.x % LPR;
    constexpr int kPer = 16 / sizeof(T);
    const bool mine = piece * kPer < a.D;
    const T *o = static_cast<const T *>(a.o_in) + h * a.o_hs + piece * kPer;
    const T *g = static_cast<const T *>(a.dO) + h * a.dO_hs + piece * kPer;
    V x[kTurns], y[kTurns];
    float l[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int i = t.t0 + r0 + k * kRows;
        x[k] = y[k] = V{};
        l[k] = -INFINITY;
        if (i >= 0 && i < t.len && t.olen > 0) {
            const int64_t tok = t.s0 + i;
            l[k] = a.lse[static_cast<int64_t>(h) * a.sq.T + tok];
            if (mine) {
                x[k] = *reinterpret_cast<const V *>(o + tok * a.o_ts);
                y[k] = *reinterpret_cast<const V *>(g + tok * a.dO_ts);
            }
        }
    }
    const int64_t at = h * a.stat_stride + static_cast<int64_t>(slot) * TILE;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        float delta = dot16(x[k], y[k]);
#pragma unroll
        for (int m = LPR / 2; m; m >>= 1) delta += __shfl_xor_sync(0xffffffffu, delta, m);
        if (piece == 0) {
            const bool out = l[k] == -INFINITY;
            a.nlse2[at + r0 + k * kRows] = out ? -INFINITY : -l[k] * kAttnLog2e;
            a.ndelta[at + r0 + k * kRows] = out ? 0.f : -delta;
        }
    }
}

}  // namespace lce
