// Attention forward on the tensor cores (bf16).
//
// A tile is 128 query rows of one head, against all the keys they see in tiles
// of 128, with a running maximum and sum per row (two threads a row, 64 keys
// each, that exchange their maxima).
//   S = Q K^T        128 x 128 fp32 in TMEM
//   P = 2^(S - m)    bf16, written over S in TMEM, the A operand of
//   O += P V         fp32 in TMEM
// The maximum a row's exponents refer to moves only when it grows by more than
// 2^8 (kLazy): until then P stays below 256 and O needs no rescaling, which
// costs a round trip of O through registers. The last reference divides out.
// kTwo: what rounding took from P goes in as a second bf16 operand, a product
// more.
//
// What bounds it is shared memory: a product of 128 x 128 x 128 takes the
// tensor core 512 cycles and reads 64 KB (S) or 32 KB (P V) there, at 128 bytes
// a cycle, and K and V have to be written first. So a CTA takes two tiles, the
// sides A and B, that share every K and V: two query heads of one key head
// where they come in pairs, else two tiles of rows. Per tile and key tile that
// is 1024 cycles of each instead of 1280 (with a CTA for each, two on an SM).
// One side's softmax runs beside the other's MMAs. Measured with 32 query and 8
// key heads of 128 channels, causal: one sequence of 8192 tokens 309 us (1.8
// PFLOP/s of the products that the mask leaves), eleven of 750 on average 72
// (850 TFLOP/s; with a CTA for each tile 83). There the tile that the mask cuts
// and the start and output of each piece count for most. Pairs of heads, not
// of tiles, where there is a choice: the sides then have the same keys
// (8192 tokens in sequences of 1024: 67 us against 72, of 128: 46 against 62).
//
// 576 threads: warps 0-7 softmax of A, 8-15 of B, warp 16 loads, warp 17 MMA
// issue. A CTA takes one piece of work after another: warp 16 asks the hardware
// for the next block of the grid that has not started, finds its sequence and
// starts its loads while the piece before is still at work. (With a block for
// every piece, starting, finding the sequence and waiting for the first loads
// took 8500 of 22000 cycles at four key tiles a block.)
#pragma once

#include <stddef.h>

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kFwdThreads = 576;
constexpr float kLazy = 8.f;

template <int KS>
struct FwdSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kK = 2 * kTile, kV = 4 * kTile;  // after the two Q: two slots of K, two of V
    static constexpr int kMax = 6 * kTile;
    static constexpr int kBars = kMax + 8 * kTcTile * 4;  // row maxima: of each side two buffers of two halves
    static constexpr int kBytes = kBars + 512;
};

// One side's tile.
struct FwdSide {
    int head;
    int rows;       // query rows (0: nothing to do)
    int n;          // key tiles (0: no row sees a key)
    int tok;        // first query token
    int last;       // causal: last key of the first row (position in the sequence)
};
// A piece of work as warp 16 hands it to the others.
struct FwdWork {
    FwdSide side[2];   // n of the first is at most n of the second
    int hk;         // key head; -1: no more work
    int first;      // first key tile
    int range;
    int keys;       // keys of the sequence
    int ktok;       // first key token
};

struct FwdBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // loads of K and V tiles
    uint64_t q_full, q_empty;                    // loads of both Q
    uint64_t s_full[2], o_done[2];               // by side: S, an O step done
    uint64_t p_full[2][2];                       // by side: P, each thread's first and second 32 keys
    uint64_t o_free[2];                          // by side: O read
    uint64_t staged[2][2];                       // by side: its output gone out through the last K (A) or V (B) slot (in turn)
    uint64_t work_full[2], work_empty[2];
    uint64_t clc, dead;
    uint4 answer;
    FwdWork work[2];
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(FwdBars) <= 512, "room after the maxima");

// kRanges: a piece takes one of `split` ranges of its keys and leaves its o, in
// fp32, and lse for k_attn_merge.
template <int KS, bool kTwo, bool kRanges>
__global__ void __launch_bounds__(kFwdThreads, 1) k_attn_fwd(const __grid_constant__ AttnArgs a,
                                                             const __grid_constant__ AttnMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // swizzled tiles need it; a launch has no other way to say so
        if (threadIdx.x == 0) atomicOr(a.status, kDevTimeout);
        return;
    }
    using L = FwdSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *sq = smem, *sk = smem + L::kK, *sv = smem + L::kV;
    FwdBars &bar = *reinterpret_cast<FwdBars *>(smem + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        uint64_t *all = bar.k_full;
        for (int i = 0; i < static_cast<int>(offsetof(FwdBars, answer) / 8); ++i) mbar_init(&all[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.p_full[i][0], 8);
            mbar_init(&bar.p_full[i][1], 8);
            mbar_init(&bar.o_free[i], 8);
            mbar_init(&bar.staged[i][0], 8);
            mbar_init(&bar.staged[i][1], 8);
            mbar_init(&bar.work_empty[i], 17);
        }
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 512) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, bar.tmem, 0);   // columns: S of A and B, O of A and B
    const TcWaits wait{&bar.abort_flag, a.status};

    if (warp == 16) {
        const TileFinder<kTcTile> finder(a.sq, a.sk);
        const TileFinder<2 * kTcTile> finder2(a.sq, a.sk);
        // longest rows first: under a causal mask the last tiles have the most keys
        auto find = [&](int block) {
            if (block == 0) {
                check_offsets(a.sq, a.status);
                check_offsets(a.sk, a.status);
            }
            FwdWork w{};
            const int ranges = kRanges ? a.split : 1;
            w.range = kRanges ? block % ranges : 0;
            if (kRanges) block /= ranges;
            const int heads = a.pair_heads ? a.Hq / 2 : a.Hq;
            const int slot = gridDim.x / (heads * ranges) - 1 - block / heads, h = block % heads;
            const TileInfo t = a.pair_heads ? finder.of_q(slot) : finder2.of_q(slot);
            const int off = t.olen - t.len;   // causal: row i sees keys [0, i + off]
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                FwdSide &s = w.side[i];
                const int t0 = a.pair_heads ? t.t0 : t.t0 + i * kTcTile;
                s.head = a.pair_heads ? 2 * h + i : h;
                s.rows = t.t0 < 0 ? 0 : max(0, min(kTcTile, t.len - t0));
                const int kend = a.causal ? min(t.olen, t0 + s.rows + off) : t.olen;
                s.n = s.rows > 0 && kend > 0 ? (kend + kTcTile - 1) / kTcTile : 0;
                s.tok = t.s0 + t0;
                s.last = t0 + off;
            }
            if (w.side[1].rows == 0 && w.side[0].rows > 0) {   // the longer side is the second
                const FwdSide s = w.side[0];
                w.side[0] = w.side[1];
                w.side[1] = s;
            }
            if (kRanges) {   // the second side's keys in equal ranges
                const int each = (w.side[1].n + ranges - 1) / ranges;
                w.first = w.range * each;
#pragma unroll
                for (int i = 0; i < 2; ++i) w.side[i].n = max(0, min(w.side[i].n - w.first, each));
            }
            w.hk = w.side[1].head / a.group;
            w.keys = t.olen;
            w.ktok = t.o0;
            return w;
        };
        bool ok = true;
        int pieces = 0, nq = 0, kv = 0;         // handed over, Q loads, K/V pairs of loads so far
        int kl = 0, vl = 0;                     // loads issued
        int outs[2] = {0, 0}, staged[2] = {0, 0};          // by side: outputs so far, and known to have gone out
        int need_k[2] = {0, 0}, need_v[2] = {0, 0};        // of A's (B's) outputs, how many must have, by ring slot
        auto publish = [&](const FwdWork &w) {
            if (!(ok = wait.all(&bar.work_empty[pieces & 1], ((pieces >> 1) & 1) ^ 1))) return;
            if (lane == 0) {
                bar.work[pieces & 1] = w;
                mbar_arrive(&bar.work_full[pieces & 1]);
            }
            __syncwarp();
            ++pieces;
        };
        auto await_staged = [&](int side, int count) {
            int &seen = staged[side];
            for (; ok && seen < count; ++seen) ok = wait.all(&bar.staged[side][seen & 1], (seen >> 1) & 1);
            return ok;
        };
        bool asked = false;   // a request for the next block is in flight
        int answers = 0;
        auto request = [&] {
            if (lane == 0) {
                fence_proxy_async_smem();   // the last answer has been read
                clc_request(&bar.answer, &bar.clc);
            }
            __syncwarp();
            asked = true;
        };
        FwdWork cur = find(blockIdx.x);
        publish(cur);
        while (ok && cur.hk >= 0) {
            const int n = cur.side[1].n;
            if (n > 0) {
                // seeing every output go out in turn, at most two pieces late, keeps the barriers' phases apart
                if (!await_staged(0, outs[0] - 1) || !await_staged(1, outs[1] - 1)) break;
                if (!(ok = wait.all(&bar.q_empty, (nq & 1) ^ 1))) break;
                if (lane == 0) {
                    // a side without work loads the other's tile: nothing reads it
                    mbar_arrive_expect_tx(&bar.q_full, 2 * L::kTile);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const FwdSide &s = cur.side[cur.side[i].n > 0 ? i : 1];
                        tc_load_tile<NB>(sq + i * L::kTile, &maps.q, &bar.q_full, s.head, s.tok);
                    }
                }
                ++nq;
            }
            FwdWork next{};
            const int steps = max(n, 1);
            for (int j = 0; j < steps; ++j) {
                // the next piece is asked for when this one's last loads but one are due: late enough not to hold work
                // that an idle CTA could start, early enough for it to be found
                if (j == max(0, n - 2)) request();
                if (j < n) {
                    const int at = cur.ktok + (kRanges ? cur.first + j : j) * kTcTile, i = kv & 1;
                    const uint32_t phase = (kv >> 1) & 1;
                    if (!await_staged(0, need_k[i])) break;
                    if (!(ok = wait.all(&bar.k_empty[i], phase ^ 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.k_full[i], L::kTile);
                        tc_load_tile<NB>(sk + i * L::kTile, &maps.k, &bar.k_full[i], cur.hk, at);
                    }
                    ++kl;
                    if (!await_staged(1, need_v[i]) || !(ok = wait.all(&bar.v_empty[i], phase ^ 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.v_full[i], L::kTile);
                        tc_load_tile<NB>(sv + i * L::kTile, &maps.v, &bar.v_full[i], cur.hk, at);
                    }
                    ++vl;
                    ++kv;
                }
                if (j + 1 == steps) {
                    for (;;) {
                        if (!(ok = wait.all(&bar.clc, answers & 1))) break;
                        ++answers;
                        asked = false;
                        const int block = __shfl_sync(0xffffffffu, clc_answer(&bar.answer), 0);
                        if (block >= 0) next = find(block);
                        else next.hk = -1;
                        if (next.hk < 0 || next.side[1].rows > 0) break;
                        request();   // an empty slot: one more
                    }
                    if (ok) publish(next);
                    if (!ok) break;
                }
            }
            if (!ok) break;
            // A's output goes out through the slot of the last K, B's through that of the last V
            if (cur.side[0].n > 0) need_k[(kv - 1) & 1] = ++outs[0];
            if (n > 0) need_v[(kv - 1) & 1] = ++outs[1];
            cur = next;
        }
        if (!ok && lane == 0) {   // what is in flight lands before the CTA gives up its memory
            if (nq) tc_drain(&bar.q_full, (nq - 1) & 1);
            for (int i = max(0, kl - 2); i < kl; ++i) tc_drain(&bar.k_full[i & 1], (i >> 1) & 1);
            for (int i = max(0, vl - 2); i < vl; ++i) tc_drain(&bar.v_full[i & 1], (i >> 1) & 1);
            if (asked) tc_drain(&bar.clc, answers & 1);
        }
        __syncwarp();
    } else if (warp == 17) {
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false) | (a.scale < 0.f ? kIdescNegA : 0);
        const uint32_t idO = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint64_t dq = tc_desc_k(sq), dk = tc_desc_k(sk), dv = tc_desc_mn(sv);
        constexpr uint32_t kStep = L::kTile >> 4;   // from slot to slot in a descriptor
        bool ok = true;
        int nq = 0, kv = 0;             // pieces, K/V tiles so far
        uint32_t np[2] = {0, 0};        // tiles of P so far, by side
        int no[2] = {0, 0};             // pieces with O so far, by side
        for (int pieces = 0; ok; ++pieces) {
            if (!(ok = wait.all(&bar.work_full[pieces & 1], (pieces >> 1) & 1))) break;
            const FwdWork &w = bar.work[pieces & 1];
            const int hk = __shfl_sync(0xffffffffu, w.hk, 0), na = __shfl_sync(0xffffffffu, w.side[0].n, 0),
                      nb = __shfl_sync(0xffffffffu, w.side[1].n, 0), keys = __shfl_sync(0xffffffffu, kRanges ? w.keys - w.first * kTcTile : w.keys, 0);
            if (lane == 0) mbar_arrive(&bar.work_empty[pieces & 1]);
            if (hk < 0) break;
            if (nb == 0) continue;
            if (!(ok = wait.all(&bar.q_full, nq & 1))) break;
            // S of side i for key tile kv + j (its K has arrived)
            auto scores = [&](int i, int j, bool done, bool last) {
                const int slot = (kv + j) & 1;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_scores<KS>(tm + i * 128, dq + i * kStep, dk + slot * kStep, idS);
                    umma_commit(&bar.s_full[i]);
                    if (done) umma_commit(&bar.k_empty[slot]);
                    if (last) umma_commit(&bar.q_empty);
                }
                __syncwarp();
            };
            auto await_k = [&](int j) { return wait.all(&bar.k_full[(kv + j) & 1], ((kv + j) >> 1) & 1); };
            // O += P V of side i for key tile kv + j
            auto mix = [&](int i, int j, bool done) {
                const int slot = (kv + j) & 1;
                const uint32_t parity = np[i]++ & 1;
                if (j == 0) {   // the O before has been read
                    if (no[i] > 0 && !wait.all(&bar.o_free[i], (no[i] - 1) & 1)) return false;
                    ++no[i];
                }
                if (!wait.all(&bar.p_full[i][0], parity)) return false;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_tokens_chunk<0>(tm + 256 + i * 128, tm + i * 128, dv + slot * kStep, idO, j > 0);
                }
                __syncwarp();
                if (!wait.all(&bar.p_full[i][1], parity)) return false;
                if (elect_one()) {
                    tc_fence_after();
                    if constexpr (kTwo) {
                        tc_mma_tokens_chunk<0>(tm + 256 + i * 128, tm + i * 128 + 32, dv + slot * kStep, idO, true);
                        tc_mma_tokens_chunk<1>(tm + 256 + i * 128, tm + i * 128 + 32, dv + slot * kStep, idO, true);
                    }
                    tc_mma_tokens_chunk<1>(tm + 256 + i * 128, tm + i * 128, dv + slot * kStep, idO, true);
                    umma_commit(&bar.o_done[i]);
                    if (done) umma_commit(&bar.v_empty[slot]);
                }
                __syncwarp();
                return true;
            };
            if (!(ok = await_k(0))) break;
            if (na > 0) scores(0, 0, false, false);
            scores(1, 0, true, nb == 1);
            int left = keys;
            for (int j = 0; j < nb; ++j, left -= kTcTile) {
                const int slot = (kv + j) & 1;
                if (!(ok = wait.all(&bar.v_full[slot], ((kv + j) >> 1) & 1))) break;
                if (left < kTcTile) tc_zero_rows<NB>(sv + slot * L::kTile, left);
                const bool more = j + 1 < nb;
                if (j < na && !(ok = mix(0, j, false))) break;
                if (more && !(ok = await_k(j + 1))) break;
                if (j + 1 < na) scores(0, j + 1, false, false);
                if (!(ok = mix(1, j, true))) break;
                if (more) scores(1, j + 1, true, j + 2 == nb);
            }
            kv += nb;
            ++nq;
        }
        if (!ok && elect_one()) {   // let the MMAs issued so far finish
            umma_commit(&bar.dead);
            tc_drain(&bar.dead, 0);
        }
        __syncwarp();
    } else {
        const int side = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;   // keys [64*half, +64) of a tile
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = quarter * 32 + lane;
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);   // never 0: a masked -inf stays -inf
        const uint32_t tSh = tm + side * 128 + lane_base + half * 64, tO = tm + 256 + side * 128 + lane_base;
        float *maxima = reinterpret_cast<float *>(smem + L::kMax) + side * 4 * kTcTile;
        const int pair = side * 4 + quarter + 1;   // barrier of the two warps that share rows
        int turn = 0;   // of the two buffers of maxima
        // what the row's other thread has to say
        auto exchange = [&](float v) {
            float *at = maxima + turn * 2 * kTcTile;
            turn ^= 1;
            at[half * kTcTile + row] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            return at[(half ^ 1) * kTcTile + row];
        };
        // a warp that gives up before an exchange must not leave its partner waiting in it; in all later
        // waits the partner gives up too, since this warp's share of P never comes
        auto leave = [&] { asm volatile("bar.arrive %0, 64;" ::"r"(pair) : "memory"); };
        bool ok = true;
        uint32_t ns = 0;        // tiles of this side so far
        int outs = 0, kv = 0;   // this side's outputs, K/V tiles so far
        for (int pieces = 0; ok; ++pieces) {
            if (!(ok = wait.all(&bar.work_full[pieces & 1], (pieces >> 1) & 1))) {
                leave();
                break;
            }
            const FwdWork &shared = bar.work[pieces & 1];
            const FwdSide w = shared.side[side];
            const int hk = shared.hk, all_keys = shared.keys, tiles = shared.side[1].n, first = kRanges ? shared.first : 0, range = kRanges ? shared.range : 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.work_empty[pieces & 1]);
            if (hk < 0) break;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + static_cast<int64_t>(w.tok) * a.o_ts + w.head * a.o_hs;
            float *lse = a.lse + static_cast<int64_t>(w.head) * a.sq.T + w.tok + row;
            // of a range: o in [range][Tq][Hq][D], then lse in [range][Hq][Tq]
            const int64_t part_ts = static_cast<int64_t>(a.Hq) * a.D;
            float *part_o = nullptr;
            if (kRanges) {
                part_o = a.part + (range * static_cast<int64_t>(a.sq.T) + w.tok) * part_ts + w.head * a.D;
                lse = a.part + a.split * (a.sq.T * part_ts) + (range * static_cast<int64_t>(a.Hq) + w.head) * a.sq.T + w.tok + row;
            }
            const bool live = row < w.rows;
            if (w.n == 0) {   // no row of the tile sees a key (or there are no rows)
                if (live) {
                    if (!kRanges)   // (the merge gives it no weight)
                        for (int c = half * 8; c < a.D; c += 16) *reinterpret_cast<uint4 *>(o + row * a.o_ts + c) = make_uint4(0, 0, 0, 0);
                    if (half == 0) *lse = -INFINITY;
                }
                kv += tiles;   // of the other side
                continue;
            }
            const int last = w.last + row;             // causal: last key of the row
            float m = -INFINITY;                       // reference maximum (of S, unscaled)
            f32x2 l2 = both(0.f);                      // sum, of this thread's keys
            for (int j = 0; j < w.n; ++j, ++ns) {
                if (!(ok = wait.all(&bar.s_full[side], ns & 1))) {
                    leave();
                    break;
                }
                tc_fence_after();
                const int k0 = (first + j) * kTcTile;
                const int keys = min(kTcTile, all_keys - k0);
                // the warp's first row is its tightest
                const bool cut = keys < kTcTile || (a.causal && k0 + kTcTile - 1 > w.last + quarter * 32);
                const int lim = (a.causal ? min(keys, last + 1 - k0) : keys) - half * 64;
                uint32_t s[2][32];
                auto load = [&] {
                    tmem_ld32(tSh, s[0]);
                    tmem_ld32(tSh + 32, s[1]);
                    tmem_ld_wait();
                    if (cut) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i >= lim) s[i / 32][i % 32] = 0xff800000u;   // -inf
                    }
                };
                load();
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i / 32][i % 32]));
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                top = fmaxf(top, exchange(top));
                const bool grow = (top - m) * sc > kLazy || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grow)) {
                    const float next = grow ? top : m;
                    if (j > 0) {
                        const float fix = grow ? ex2((m - next) * sc) : 1.f;   // m = -inf: 2^-inf = 0 on an O of zeros
                        l2 = mul2(l2, both(fix));
                        if (!(ok = wait.all(&bar.o_done[side], (ns - 1) & 1))) break;
                        tc_fence_after();
                        // this half's share of O; its scores are fetched again after it, to leave it their registers
                        using C = Chunks<KS>;
#pragma unroll 1
                        for (int c = half ? C::kFirst : 0; c < (half ? C::kAll : C::kFirst); ++c) {
                            uint32_t v[32];
                            tmem_ld32(tO + c * 32, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fix);
                            tmem_st32(tO + c * 32, v);
                        }
                        load();
                    }
                    m = next;
                }
                const f32x2 base = both(m == -INFINITY ? 0.f : -m * sc), sc2 = both(sc);
                // P in two steps, so that the first half of O's step runs under the second half of the exponents
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[16], rest[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x, y;
                        unpack2(fma2(pack2u(s[c][2 * i], s[c][2 * i + 1]), sc2, base), x, y);
                        x = ex2(x), y = ex2(y);
                        l2 = add2(l2, pack2(x, y));
                        p[i] = pack_bf16(x, y);
                        if constexpr (kTwo) rest[i] = pack_bf16(x - __uint_as_float(p[i] << 16), y - __uint_as_float(p[i] & 0xffff0000u));
                    }
                    tmem_st16(tSh + c * 16, p);
                    if constexpr (kTwo) tmem_st16(tSh + 32 + c * 16, rest);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[side][c]);
                }
            }
            if (!ok) break;
            kv += tiles;
            // the slots that the output goes out through are the other side's too, until it is done with its last tile
            if (!(ok = wait.all(&bar.o_done[side], (ns - 1) & 1)) || !(ok = wait.all(side ? &bar.v_empty[(kv - 1) & 1] : &bar.k_empty[(kv - 1) & 1], ((kv - 1) >> 1) & 1))) {
                leave();
                break;
            }
            tc_fence_after();
            const float part = hsum2(l2), l = part + exchange(part);
            const float inv = l != 0.f ? 1.f / l : 0.f;   // l of an empty row is 0; NaN stays
            if (half == 0 && live) *lse = l == 0.f ? -INFINITY : (m * sc + log2f(l)) * (1.f / kAttnLog2e);
            uint8_t *tile = (side ? sv : sk) + ((kv - 1) & 1) * L::kTile;
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free[side]);
            };
            if (kRanges) tc_store_fp32<KS>(half, tile, tO, inv, quarter * 32, w.rows, part_o, part_ts, a.D, release);
            else tc_store_half<KS>(half, tile, tO, inv, quarter * 32, w.rows, o, a.o_ts, a.D, release);
            fence_proxy_async_smem();   // the slot goes back to the loads
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.staged[side][outs & 1]);
            ++outs;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

}  // namespace lce
