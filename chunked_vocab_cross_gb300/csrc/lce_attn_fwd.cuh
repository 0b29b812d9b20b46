// Attention forward on the tensor cores (bf16).
//
// A tile of work is 128 query rows of one head, against all the keys they see
// in tiles of 128, with a running maximum and sum per row (two threads a row,
// 64 keys each, that exchange their maxima).
//   S = Q K^T        128 x 128 fp32 in TMEM
//   P = 2^(S - m)    bf16, written over S in TMEM, the A operand of
//   O += P V         fp32 in TMEM
// The maximum a row's exponents refer to moves only when it grows by more than
// 2^8 (kLazy): until then P stays below 256 and O needs no rescaling, which
// costs a round trip of O through registers. The last reference divides out.
//
// Two CTAs share an SM, so that one's softmax runs beside the other's MMAs.
// 320 threads: warps 0-7 softmax, warp 8 loads, warp 9 MMA issue. A CTA takes
// one tile after another: warp 8 asks the hardware for the next block of the
// grid that has not started, finds its sequence and starts its loads while the
// tile before is still at work. (A block of its own for every tile spent 8500
// of 22000 cycles on starting, finding its sequence and waiting for its first
// loads, at four key tiles a block.)
#pragma once

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kFwdThreads = 320;
constexpr float kLazy = 8.f;

template <int KS>
struct FwdSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kMax = 3 * kTile;               // Q, one slot of K and of V
    static constexpr int kBars = kMax + 4 * kTcTile * 4; // row maxima: two buffers of two halves
    static constexpr int kBytes = kBars + 256 + 1024;    // alignment slack
};

// A tile of work as warp 8 hands it to the others.
struct FwdWork {
    int h;          // query head; -1: no more work
    int rows;       // query rows (0: nothing to do)
    int n;          // key tiles (0: no row sees a key)
    int tok;        // first query token
    int last;       // causal: last key of the first row (position in the sequence)
    int keys;       // keys of the sequence
    int ktok;       // first key token
    int pad;
};

struct FwdBars {
    uint64_t k_full, k_empty, v_full, v_empty;   // loads of K and V tiles (v_empty: of all but a work tile's last)
    uint64_t staged;                             // O has gone out through V's slot
    uint64_t q_full, q_empty;                    // loads of Q
    uint64_t s_full, p_full[2];                  // S; P, each thread's first and second 32 keys
    uint64_t o_done, o_free;                     // an O step done, O read
    uint64_t work_full[2], work_empty[2];
    uint64_t clc, fin;
    uint4 answer;
    FwdWork work[2];
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(FwdBars) <= 256, "room after the maxima");

template <int KS>
__global__ void __launch_bounds__(kFwdThreads, 2) k_attn_fwd(const __grid_constant__ AttnArgs a,
                                                             const __grid_constant__ AttnMaps maps) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    using L = FwdSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *sq = smem, *sk = smem + L::kTile, *sv = smem + 2 * L::kTile;
    FwdBars &bar = *reinterpret_cast<FwdBars *>(smem + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        uint64_t *one[] = {&bar.k_full, &bar.k_empty, &bar.v_full, &bar.v_empty, &bar.q_full, &bar.q_empty, &bar.s_full,
                           &bar.o_done, &bar.work_full[0], &bar.work_full[1], &bar.clc, &bar.fin};
        for (uint64_t *b : one) mbar_init(b, 1);
        mbar_init(&bar.p_full[0], 8);
        mbar_init(&bar.p_full[1], 8);
        mbar_init(&bar.o_free, 8);
        mbar_init(&bar.staged, 8);
        for (int i = 0; i < 2; ++i) mbar_init(&bar.work_empty[i], 9);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bar.tmem, 256);
        tmem_relinquish();
    }
    if (threadIdx.x == 256) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
    const uint32_t tS = tmem, tO = tmem + 128;
    const TcWaits wait{&bar.abort_flag, a.status};

    if (warp == 8) {
        const TileFinder<kTcTile> finder(a.sq, a.sk);
        // longest rows first: under a causal mask the last tiles have the most keys
        auto find = [&](int block) {
            if (block == 0) {
                check_offsets(a.sq, a.status);
                check_offsets(a.sk, a.status);
            }
            FwdWork w{};
            w.h = block % a.Hq;
            const TileInfo t = finder.of_q(gridDim.x / a.Hq - 1 - block / a.Hq);
            const int off = t.olen - t.len;   // causal: row i sees keys [0, i + off]
            w.rows = t.t0 < 0 ? 0 : max(0, min(kTcTile, t.len - t.t0));
            const int kend = a.causal ? min(t.olen, t.t0 + w.rows + off) : t.olen;
            w.n = w.rows > 0 && kend > 0 ? (kend + kTcTile - 1) / kTcTile : 0;
            w.tok = t.s0 + t.t0;
            w.last = t.t0 + off;
            w.keys = t.olen;
            w.ktok = t.o0;
            return w;
        };
        bool ok = true;
        int tiles = 0, qs = 0, kv = 0, ve = 0;   // tiles handed over, Q loads, K/V pairs of loads, waits on v_empty so far
        auto publish = [&](const FwdWork &w) {
            if (!(ok = wait.all(&bar.work_empty[tiles & 1], ((tiles >> 1) & 1) ^ 1))) return;
            if (lane == 0) {
                bar.work[tiles & 1] = w;
                mbar_arrive(&bar.work_full[tiles & 1]);
            }
            __syncwarp();
            ++tiles;
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
        int kl = 0, vl = 0;   // loads issued
        while (ok && cur.h >= 0) {
            const int hk = cur.h / a.group;
            if (cur.n > 0) {
                if (!(ok = wait.all(&bar.q_empty, (qs & 1) ^ 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.q_full, L::kTile);
                    tc_load_tile<NB>(sq, &maps.q, &bar.q_full, cur.h, cur.tok);
                }
                ++qs;
            }
            FwdWork next{};
            const int steps = max(cur.n, 1);
            for (int j = 0; j < steps; ++j) {
                // the next tile is asked for when this one's last loads but one are due: late enough not to hold work
                // that an idle CTA could start, early enough for it to be found
                if (j == max(0, cur.n - 2)) request();
                if (j < cur.n) {
                    const int at = cur.ktok + j * kTcTile;
                    if (!(ok = wait.all(&bar.k_empty, (kv & 1) ^ 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.k_full, L::kTile);
                        tc_load_tile<NB>(sk, &maps.k, &bar.k_full, hk, at);
                    }
                    ++kl;
                    // a tile's first V waits for the output before it, the others for the MMAs that read V
                    if (j == 0 ? qs > 1 && !(ok = wait.all(&bar.staged, qs & 1)) : !(ok = wait.all(&bar.v_empty, ve++ & 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.v_full, L::kTile);
                        tc_load_tile<NB>(sv, &maps.v, &bar.v_full, hk, at);
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
                        else next.h = -1;
                        if (next.h < 0 || next.rows > 0) break;
                        request();   // an empty slot: one more
                    }
                    if (ok) publish(next);
                    if (!ok) break;
                }
            }
            cur = next;
        }
        if (!ok && lane == 0) {   // what is in flight lands before the CTA gives up its memory
            if (qs) tc_drain(&bar.q_full, (qs - 1) & 1);
            if (kl) tc_drain(&bar.k_full, (kl - 1) & 1);
            if (vl) tc_drain(&bar.v_full, (vl - 1) & 1);
            if (asked) tc_drain(&bar.clc, answers & 1);
        }
        __syncwarp();
    } else if (warp == 9) {
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false) | (a.scale < 0.f ? kIdescNegA : 0);
        const uint32_t idO = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint64_t dq = tc_desc_k(sq), dk = tc_desc_k(sk), dv = tc_desc_mn(sv);
        bool ok = true;
        int qs = 0, kv = 0;
        for (int tiles = 0; ok; ++tiles) {
            if (!(ok = wait.all(&bar.work_full[tiles & 1], (tiles >> 1) & 1))) break;
            const FwdWork &w = bar.work[tiles & 1];
            const int h = __shfl_sync(0xffffffffu, w.h, 0), n = __shfl_sync(0xffffffffu, w.n, 0),
                      left = __shfl_sync(0xffffffffu, w.keys, 0);
            if (lane == 0) mbar_arrive(&bar.work_empty[tiles & 1]);
            if (h < 0) break;
            if (n == 0) continue;
            if (!(ok = wait.all(&bar.q_full, qs & 1))) break;
            for (int j = 0; j < n; ++j, ++kv) {
                if (!(ok = wait.all(&bar.k_full, kv & 1))) break;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_scores<KS>(tS, dq, dk, idS);
                    umma_commit(&bar.k_empty);
                    if (j + 1 == n) umma_commit(&bar.q_empty);
                    umma_commit(&bar.s_full);
                }
                __syncwarp();
                if (!(ok = wait.all(&bar.v_full, kv & 1))) break;
                const int keys = min(kTcTile, left - j * kTcTile);
                if (keys < kTcTile) tc_zero_rows<NB>(sv, keys);
                if (j == 0 && !(ok = wait.all(&bar.o_free, (qs & 1) ^ 1))) break;   // the O before has been read
                if (!(ok = wait.all(&bar.p_full[0], kv & 1))) break;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_tokens_chunk<0>(tO, tS, dv, idO, j > 0);
                }
                __syncwarp();
                if (!(ok = wait.all(&bar.p_full[1], kv & 1))) break;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_tokens_chunk<1>(tO, tS, dv, idO, true);
                    if (j + 1 < n) umma_commit(&bar.v_empty);
                    umma_commit(&bar.o_done);
                }
                __syncwarp();
            }
            ++qs;
        }
        if (!ok && elect_one()) {   // let the MMAs issued so far finish
            umma_commit(&bar.fin);
            tc_drain(&bar.fin, 0);
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;   // keys [64*half, +64) of a tile
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = quarter * 32 + lane;
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);   // never 0: a masked -inf stays -inf
        const uint32_t tSh = tS + lane_base + half * 64;
        float *maxima = reinterpret_cast<float *>(smem + L::kMax);
        int turn = 0;   // of the two buffers of maxima
        // what the row's other thread has to say
        auto exchange = [&](float v) {
            float *at = maxima + turn * 2 * kTcTile;
            turn ^= 1;
            at[half * kTcTile + row] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory");
            return at[(half ^ 1) * kTcTile + row];
        };
        // a warp that gives up before an exchange must not leave its partner waiting in it; in all later
        // waits the partner gives up too, since this warp's share of P never comes
        auto leave = [&] { asm volatile("bar.arrive %0, 64;" ::"r"(quarter + 1) : "memory"); };
        bool ok = true;
        int kv = 0;
        for (int tiles = 0; ok; ++tiles) {
            if (!(ok = wait.all(&bar.work_full[tiles & 1], (tiles >> 1) & 1))) {
                leave();
                break;
            }
            const FwdWork w = bar.work[tiles & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.work_empty[tiles & 1]);
            if (w.h < 0) break;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + static_cast<int64_t>(w.tok) * a.o_ts + w.h * a.o_hs;
            float *lse = a.lse + static_cast<int64_t>(w.h) * a.sq.T + w.tok + row;
            const bool live = row < w.rows;
            if (w.n == 0) {   // no row of the tile sees a key (or there are no rows)
                if (live) {
                    for (int c = half * 8; c < a.D; c += 16) *reinterpret_cast<uint4 *>(o + row * a.o_ts + c) = make_uint4(0, 0, 0, 0);
                    if (half == 0) *lse = -INFINITY;
                }
                continue;
            }
            const int last = w.last + row;             // causal: last key of the row
            float m = -INFINITY;                       // reference maximum (of S, unscaled)
            f32x2 l2 = both(0.f);                      // sum, of this thread's keys
            for (int j = 0; j < w.n; ++j, ++kv) {
                if (!(ok = wait.all(&bar.s_full, kv & 1))) {
                    leave();
                    break;
                }
                tc_fence_after();
                const int k0 = j * kTcTile;
                const int keys = min(kTcTile, w.keys - k0);
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
                        if (!(ok = wait.all(&bar.o_done, (kv - 1) & 1))) break;
                        tc_fence_after();
                        // this half's share of O; its scores are fetched again after it, to leave it their registers
                        using C = Chunks<KS>;
#pragma unroll 1
                        for (int c = half ? C::kFirst : 0; c < (half ? C::kAll : C::kFirst); ++c) {
                            uint32_t v[32];
                            tmem_ld32(tO + lane_base + c * 32, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fix);
                            tmem_st32(tO + lane_base + c * 32, v);
                        }
                        load();
                    }
                    m = next;
                }
                const f32x2 base = both(m == -INFINITY ? 0.f : -m * sc), sc2 = both(sc);
                // P in two steps, so that the first half of O's step runs under the second half of the exponents
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x, y;
                        unpack2(fma2(pack2u(s[c][2 * i], s[c][2 * i + 1]), sc2, base), x, y);
                        x = ex2(x), y = ex2(y);
                        l2 = add2(l2, pack2(x, y));
                        p[i] = pack_bf16(x, y);
                    }
                    tmem_st16(tSh + c * 16, p);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[c]);
                }
            }
            if (!ok) break;
            if (!(ok = wait.all(&bar.o_done, (kv - 1) & 1))) {
                leave();
                break;
            }
            tc_fence_after();
            const float part = hsum2(l2), l = part + exchange(part);
            const float inv = l != 0.f ? 1.f / l : 0.f;   // l of an empty row is 0; NaN stays
            if (half == 0 && live) *lse = l == 0.f ? -INFINITY : (m * sc + log2f(l)) * (1.f / kAttnLog2e);
            tc_store_half<KS>(half, sv, tO + lane_base, inv, quarter * 32, w.rows, o, a.o_ts, a.D, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free);
            });
            fence_proxy_async_smem();   // V's slot goes back to the loads
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.staged);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

}  // namespace lce
