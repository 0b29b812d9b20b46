// Attention backward on the tensor cores (bf16): two kinds of work, so that
// every gradient is summed in TMEM by one CTA in a fixed order, without atomics
// and without a gradient buffer of partial sums. The probabilities are
// recomputed in both (7 products of tiles instead of 5).
//
// dQ: 128 query rows, walking the keys.
//   S = Q K^T, dP = dO V^T (128 x 128 fp32 in TMEM, rows = queries)
//   dS = 2^(S - lse) (dP - delta), bf16 over S in TMEM;  dQ += dS K
// dK/dV: 128 keys of one key head, walking the queries of its query heads.
//   S^T = K Q^T, dP^T = V dO^T (rows = keys)
//   P^T over S^T: dV += P^T dO;  dS^T over dP^T: dK += dS^T Q
// P and dS go back to TMEM as the A operands, so they never touch shared
// memory. They are rounded to bf16 for that, which adds as much to the error of
// a gradient as rounding the gradient does (0.0024 instead of 0.0017 of its
// norm). kTwo: what the rounding took goes in as a second bf16 operand, a
// product more for each sum.
//
// What bounds it is the chain from a product over the elementwise part to the
// next product: the tensor core takes 512 cycles for 128 x 128 x 128, 400 more
// when it starts from idle. So whatever can is issued ahead of its turn: P and
// dS are handed over 32 columns at a time, the sums' first steps running under
// the rest; dQ pieces ask for the next dP as soon as the last has been read;
// and where TMEM has the room (S twice, dP and both sums: up to 64 channels)
// dK/dV pieces ask for the next S before P is there.
//
// 320 threads: warps 0-7 the elementwise part (two threads a row, 64 columns
// each), warp 8 loads, warp 9 MMA issue. One CTA an SM: dK/dV fills the 512
// columns of TMEM, and the tiles fill the shared memory: two that stay for a
// piece of work (`fixed`: Q and dO, or K and V), a ring of three (`a`: K, or Q)
// and one of two (`b`: V, or dO). A CTA takes one piece of work after another
// by cluster launch control, as in the forward; the loads and the first
// products of the next run under the last sums and the output of the one
// before. Both kinds are one grid, the longer dK/dV pieces first. Where a key
// head's query heads would make them too long for the few there are, a piece
// takes a share of the heads, and k_attn_join adds up the shares.
//
// Measured with 32 query and 8 key heads of 128 channels, causal, row statistics
// included: one sequence of 8192 tokens 1.09 ms (1.26 PFLOP/s of the five
// products that the mask leaves, 1.8 of the seven taken; 1.19 ms in long runs,
// where power holds the clock near 1.5 GHz), sequences of 1024 211 us, of 128
// 132 us; 32 heads of 64 channels over 3482 ragged tokens 80 us. Sixteen warps for the elementwise
// part, four threads a row, gained 2 us there and lost 40 on 8192 tokens.
#pragma once

#include <stddef.h>

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kBwdThreads = 320;

template <int KS>
struct BwdSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kAs = 3, kBs = 2;                             // ring slots
    static constexpr int kA = 2 * kTile, kB = kA + kAs * kTile;        // after the fixed tiles
    static constexpr int kStat = 2 * kTcTile * 4;                      // nlse2 and ndelta of a Q tile; two slots
    static constexpr int kStats = kB + kBs * kTile;
    static constexpr int kBars = kStats + 2 * kStat;
    static constexpr int kBytes = kBars + 512;   // no room for alignment slack: the kernel checks the base it gets
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

enum BwdKind : int { BWD_NONE = -1, BWD_DKV = 0, BWD_DQ = 1 };

// A piece of work as warp 8 hands it to the others.
struct BwdWork {
    int kind;
    int head;       // query head (dQ) or key head; kShares: and, from bit 16 on, the share of its query heads
    int rows;       // rows of the own tile (0: nothing to do)
    int n;          // tiles of the other side, over all heads (0: zero gradients)
    int tok;        // first token of the own tile
    int t0;         // its position in the sequence
    int off;        // Lk - Lq: under a causal mask query i sees keys [0, i + off]
    int o0, olen;   // the other side: first token, length
    int first, per; // dK/dV: first query tile, query tiles a head
    int slot;       // dQ: the own tile's slot; dK/dV: the sequence's first query slot
};

struct BwdBars {
    uint64_t a_full[3], a_empty[3], b_full[2], b_empty[2], f_full, f_empty;
    uint64_t st_full[2];                          // row statistics (dK/dV)
    uint64_t s_full[2], dp_full, dp_read;         // S and dP of a tile; dP fetched (dQ)
    // P and dS, each thread's first and second 32 columns. Two sets, for tiles in turn: a warp may hand over a tile
    // while a slower one still has the tile before to hand over (never two: see where the next S and dP are asked for).
    uint64_t p_full[2][2], ds_full[2][2];
    uint64_t fin, acc_free;                       // a piece's sums done, read
    uint64_t staged[2];                           // its output gone out through the staging slot (pieces in turn)
    uint64_t work_full[2], work_empty[2];
    uint64_t clc, dead;
    uint4 answer;
    BwdWork work[2];
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(BwdBars) <= 512, "room after the statistics");

// kShares: as above. Known when the kernel is compiled, like kTwo: the code alone costs the other calls 7%.
template <int KS, bool kTwo, bool kShares>
__global__ void __launch_bounds__(kBwdThreads, 1) k_attn_bwd(const __grid_constant__ AttnArgs a,
                                                             const __grid_constant__ AttnMaps maps, int dkv_blocks) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // swizzled tiles need it; a launch has no other way to say so
        if (threadIdx.x == 0) atomicOr(a.status, kDevTimeout);
        return;
    }
    using L = BwdSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *f0 = smem, *f1 = smem + L::kTile, *sa = smem + L::kA, *sb = smem + L::kB;
    float *stats = reinterpret_cast<float *>(smem + L::kStats);
    BwdBars &bar = *reinterpret_cast<BwdBars *>(smem + L::kBars);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        uint64_t *all = bar.a_full;
        for (int i = 0; i < static_cast<int>(offsetof(BwdBars, answer) / 8); ++i) mbar_init(&all[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bar.p_full[i >> 1][i & 1], 8), mbar_init(&bar.ds_full[i >> 1][i & 1], 8);
        for (uint64_t *b : {&bar.dp_read, &bar.acc_free, &bar.staged[0], &bar.staged[1]}) mbar_init(b, 8);
        for (int i = 0; i < 2; ++i) mbar_init(&bar.work_empty[i], 9);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 256) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        tma_prefetch_map(&maps.dO);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // TMEM columns: S (or two), dP, dV, dK; two S, dP, dQ
    constexpr bool kTwoS = 3 * kTcTile + 2 * KS * 16 <= 512;   // room for two S beside dV and dK
    constexpr uint32_t cP = kTwoS ? 256 : 128, cV = cP + 128, cK = kTwoS ? cV + KS * 16 : 384;   // dK/dV
    constexpr uint32_t cP2 = 256, cQ = 384;                                                      // dQ
    const uint32_t tm = __shfl_sync(0xffffffffu, bar.tmem, 0);
    const TcWaits wait{&bar.abort_flag, a.status};

    if (warp == 8) {
        const TileFinder<kTcTile> finder(a.sq, a.sk);
        auto find = [&](int block) {
            BwdWork w{};
            if (block < dkv_blocks) {   // under a causal mask the first key tiles have the most queries
                const int split = kShares ? a.split : 1, shares = a.Hk * split;
                const TileInfo t = finder.of_k(block / shares);
                w.kind = BWD_DKV;
                w.head = block % shares / split + (kShares ? block % split << 16 : 0);
                w.rows = t.t0 < 0 ? 0 : max(0, min(kTcTile, t.len - t.t0));
                w.off = t.len - t.olen;
                w.first = a.causal ? max(0, t.t0 - w.off) / kTcTile : 0;   // the first that sees the tile's first key
                w.per = max(0, (t.olen + kTcTile - 1) / kTcTile - w.first);
                w.n = w.rows > 0 ? w.per * (kShares ? a.group / a.split : a.group) : 0;
                w.slot = t.o0 / kTcTile + t.b;
                w.tok = t.s0 + t.t0, w.t0 = t.t0, w.o0 = t.o0, w.olen = t.olen;
            } else {                    // ... and the last query tiles the most keys
                block -= dkv_blocks;
                const int slot = (gridDim.x - dkv_blocks) / a.Hq - 1 - block / a.Hq;
                const TileInfo t = finder.of_q(slot);
                w.kind = BWD_DQ;
                w.head = block % a.Hq;
                w.rows = t.t0 < 0 ? 0 : max(0, min(kTcTile, t.len - t.t0));
                w.off = t.olen - t.len;
                const int kend = a.causal ? min(t.olen, t.t0 + w.rows + w.off) : t.olen;
                w.n = w.rows > 0 && kend > 0 ? (kend + kTcTile - 1) / kTcTile : 0;
                w.slot = slot;
                w.tok = t.s0 + t.t0, w.t0 = t.t0, w.o0 = t.o0, w.olen = t.olen;
            }
            return w;
        };
        bool ok = true;
        int pieces = 0;                       // handed over
        int na = 0, nb = 0, nf = 0, ns = 0;   // loads of each kind so far
        int stat0 = -1, stat1 = -1;           // the ring tile that each slot of statistics was last for
        int staged = 0, need[3] = {0, 0, 0};  // outputs known to have gone out; how many must have, by ring slot
        auto publish = [&](const BwdWork &w) {
            if (!(ok = wait.all(&bar.work_empty[pieces & 1], ((pieces >> 1) & 1) ^ 1))) return;
            if (lane == 0) {
                bar.work[pieces & 1] = w;
                mbar_arrive(&bar.work_full[pieces & 1]);
            }
            __syncwarp();
            ++pieces;
        };
        auto await_staged = [&](int count) {
            for (; ok && staged < count; ++staged) ok = wait.all(&bar.staged[staged & 1], (staged >> 1) & 1);
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
        BwdWork cur = find(blockIdx.x);
        publish(cur);
        while (ok && cur.kind != BWD_NONE) {
            const bool dkv = cur.kind == BWD_DKV;
            const int own = kShares ? cur.head & 0xffff : cur.head;
            if (cur.n > 0) {
                // seeing every output go out in turn, at most two pieces late, keeps the barriers' phases apart
                if (!await_staged(nf - 1)) break;
                if (!(ok = wait.all(&bar.f_empty, (nf & 1) ^ 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.f_full, 2 * L::kTile);
                    tc_load_tile<NB>(f0, dkv ? &maps.k : &maps.q, &bar.f_full, own, cur.tok);
                    tc_load_tile<NB>(f1, dkv ? &maps.v : &maps.dO, &bar.f_full, own, cur.tok);
                }
                ++nf;
            }
            BwdWork next{};
            int h = dkv ? own * a.group + (kShares ? (cur.head >> 16) * (a.group / a.split) : 0) : own / a.group, tile = cur.first;   // of the other side
            const int steps = max(cur.n, 1);
            for (int j = 0; j < steps; ++j) {
                // The next piece is asked for when this one's last loads but one are due: late, so that a CTA with
                // a long piece does not hold another that an idle one could start (asked for at the start, a
                // backward of 250 pieces on 152 SMs took 47 us instead of 35), and early enough for it to be found.
                if (j == max(0, cur.n - 2)) request();
                if (j < cur.n) {
                    const int ai = na % L::kAs, bi = nb % L::kBs, at = cur.o0 + tile * kTcTile;
                    if (!await_staged(need[ai])) break;
                    if (!(ok = wait.all(&bar.a_empty[ai], ((na / L::kAs) & 1) ^ 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.a_full[ai], L::kTile);
                        tc_load_tile<NB>(sa + ai * L::kTile, dkv ? &maps.q : &maps.k, &bar.a_full[ai], h, at);
                    }
                    ++na;
                    if (!(ok = wait.all(&bar.b_empty[bi], ((nb / L::kBs) & 1) ^ 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.b_full[bi], L::kTile);
                        tc_load_tile<NB>(sb + bi * L::kTile, dkv ? &maps.dO : &maps.v, &bar.b_full[bi], h, at);
                    }
                    ++nb;
                    if (dkv) {
                        // a slot of statistics is free once the tile it was for has left its ring slot (its dK sum
                        // follows the last use of them); one three loads back has, or this tile's slot were not free
                        const int c = na - 1, p = (ns & 1) ? stat1 : stat0;
                        if (p >= 0 && p > c - L::kAs && !(ok = wait.all(&bar.a_empty[p % L::kAs], (p / L::kAs) & 1))) break;
                        ((ns & 1) ? stat1 : stat0) = c;
                        if (lane == 0) {
                            griddep_wait();   // the statistics come from the launch before
                            const int64_t st = h * a.stat_stride + static_cast<int64_t>(cur.slot + tile) * kTcTile;
                            float *dst = stats + (ns & 1) * 2 * kTcTile;
                            mbar_arrive_expect_tx(&bar.st_full[ns & 1], L::kStat);
                            bulk_load(dst, a.nlse2 + st, kTcTile * 4, &bar.st_full[ns & 1]);
                            bulk_load(dst + kTcTile, a.ndelta + st, kTcTile * 4, &bar.st_full[ns & 1]);
                        }
                        ++ns;
                    }
                    ++tile;
                    if (dkv && tile == cur.first + cur.per) tile = cur.first, ++h;
                }
                if (j + 1 == steps) {
                    for (;;) {
                        if (!(ok = wait.all(&bar.clc, answers & 1))) break;
                        ++answers;
                        asked = false;
                        const int block = __shfl_sync(0xffffffffu, clc_answer(&bar.answer), 0);
                        if (block >= 0) next = find(block);
                        else next.kind = BWD_NONE;
                        if (next.kind == BWD_NONE || next.rows > 0) break;
                        request();   // an empty slot: one more
                    }
                    if (ok) publish(next);
                    if (!ok) break;
                }
            }
            if (!ok) break;
            // the output goes out through the ring slot of the piece's last tile, which is loaded last again
            if (cur.n > 0) need[(na - 1) % L::kAs] = nf;
            cur = next;
        }
        if (!ok && lane == 0) {   // what is in flight lands before the CTA gives up its memory
            if (nf) tc_drain(&bar.f_full, (nf - 1) & 1);
            for (int i = max(0, na - L::kAs); i < na; ++i) tc_drain(&bar.a_full[i % L::kAs], (i / L::kAs) & 1);
            for (int i = max(0, nb - L::kBs); i < nb; ++i) tc_drain(&bar.b_full[i % L::kBs], (i / L::kBs) & 1);
            for (int i = max(0, ns - 2); i < ns; ++i) tc_drain(&bar.st_full[i & 1], (i >> 1) & 1);
            if (asked) tc_drain(&bar.clc, answers & 1);
        }
        __syncwarp();
    } else if (warp == 9) {
        // One warp feeds the tensor core, and what it does between two products is on the chain that bounds the kernel:
        // ring positions, phases and tokens left are counted along, descriptors are a base and a multiple.
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false), idG = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint32_t idSn = idS | (a.scale < 0.f ? kIdescNegA : 0);
        const uint64_t d0 = tc_desc_k(f0), d1 = tc_desc_k(f1);
        const uint64_t aK = tc_desc_k(sa), aM = tc_desc_mn(sa), bK = tc_desc_k(sb), bM = tc_desc_mn(sb);
        constexpr uint32_t kStep = L::kTile >> 4;   // from slot to slot in a descriptor
        bool ok = true;
        // Place in a ring and the phase of its barriers there.
        struct Pos {
            int i = 0;
            uint32_t phase = 0;
            __device__ __forceinline__ void next(int size) {
                if (++i == size) i = 0, phase ^= 1;
            }
        };
        Pos ra, rb, ua, ub;                     // next tile of the rings to multiply, and to sum over
        uint32_t np = 0, pq = 0, nd = 0;        // tiles of P so far, phase of dP read, tiles of dS so far
        int nf = 0;                             // pieces so far
        int kind = BWD_NONE;                    // of the piece before
        for (int pieces = 0; ok; ++pieces) {
            if (!(ok = wait.all(&bar.work_full[pieces & 1], (pieces >> 1) & 1))) break;
            const BwdWork &w = bar.work[pieces & 1];
            const int k = __shfl_sync(0xffffffffu, w.kind, 0), n = __shfl_sync(0xffffffffu, w.n, 0),
                      olen = __shfl_sync(0xffffffffu, w.olen, 0), first = __shfl_sync(0xffffffffu, w.first, 0),
                      per = __shfl_sync(0xffffffffu, w.kind == BWD_DKV ? w.per : w.n, 0);
            if (lane == 0) mbar_arrive(&bar.work_empty[pieces & 1]);
            if (k == BWD_NONE) break;
            if (n == 0) continue;
            const bool dkv = k == BWD_DKV;
            // The sums of the piece before have been read: needed before this piece's first sum, and before its first
            // products where the kinds have their sums in different columns.
            if (kind != k && nf > 0 && !(ok = wait.all(&bar.acc_free, (nf - 1) & 1))) break;
            bool free = kind != k || nf == 0;
            kind = k;
            if (!(ok = wait.all(&bar.f_full, nf & 1))) break;
            const uint32_t tP = tm + (dkv ? cP : cP2);
            const bool two = kTwoS || !dkv;     // S buffers
            const int left0 = olen - first * kTcTile;
            int sl = left0, sj = 0, dl = left0, dj = 0;   // tokens left in the head and tiles of it done, of S and of dP
            int sbuf = 0, di = 0;                         // S buffer to write; dP tiles done
            auto scores = [&] {
                if (!wait.all(&bar.a_full[ra.i], ra.phase)) return false;
                if (sl < kTcTile) tc_zero_rows<NB>(sa + ra.i * L::kTile, sl);   // summed over below
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_scores<KS>(tm + sbuf * 128, d0, aK + ra.i * kStep, idSn);
                    umma_commit(&bar.s_full[sbuf]);
                }
                __syncwarp();
                ra.next(L::kAs);
                sl -= kTcTile;
                if (++sj == per) sj = 0, sl = left0;
                sbuf ^= two;
                return true;
            };
            auto dprobs = [&] {
                if (!wait.all(&bar.b_full[rb.i], rb.phase)) return false;
                if (dl < kTcTile) tc_zero_rows<NB>(sb + rb.i * L::kTile, dl);
                ++di;
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_scores<KS>(tP, d1, bK + rb.i * kStep, idS);
                    umma_commit(&bar.dp_full);
                    if (!dkv) umma_commit(&bar.b_empty[rb.i]);
                    if (di == n) umma_commit(&bar.f_empty);   // the last use of the fixed tiles
                }
                __syncwarp();
                rb.next(L::kBs);
                dl -= kTcTile;
                if (++dj == per) dj = 0, dl = left0;
                return true;
            };
            // acc (+)= A . tile over the tile's tokens, A as it is handed over in two steps
            auto sum = [&](uint32_t acc, uint32_t A, uint64_t tile, uint64_t (&sets)[2][2], uint32_t number, int j,
                           uint64_t *release, bool last) {
                uint64_t *full = sets[number & 1];
                const uint32_t parity = (number >> 1) & 1;
                if (!wait.all(&full[0], parity)) return false;
                if (!free) {
                    if (!wait.all(&bar.acc_free, (nf - 1) & 1)) return false;
                    free = true;
                }
                if (elect_one()) {
                    tc_fence_after();
                    tc_mma_tokens_chunk<0>(acc, A, tile, idG, j > 0);
                }
                __syncwarp();
                if (!wait.all(&full[1], parity)) return false;
                if (elect_one()) {
                    tc_fence_after();
                    if constexpr (kTwo) {
                        tc_mma_tokens_chunk<0>(acc, A + 32, tile, idG, true);
                        tc_mma_tokens_chunk<1>(acc, A + 32, tile, idG, true);
                    }
                    tc_mma_tokens_chunk<1>(acc, A, tile, idG, true);
                    umma_commit(release);
                    if (last) umma_commit(&bar.fin);
                }
                __syncwarp();
                return true;
            };
            ok = scores() && dprobs();
            if (dkv) {
                for (int j = 0; ok && j < n; ++j) {
                    const bool more = j + 1 < n;
                    if (kTwoS && more && !(ok = scores())) break;
                    if (!(ok = sum(tm + cV, tm + (kTwoS ? (j & 1) * 128 : 0), bM + ub.i * kStep, bar.p_full, np, j, &bar.b_empty[ub.i], false))) break;
                    ub.next(L::kBs), ++np;
                    if (!kTwoS && more && !(ok = scores())) break;
                    if (!(ok = sum(tm + cK, tP, aM + ua.i * kStep, bar.ds_full, nd, j, &bar.a_empty[ua.i], !more))) break;
                    ua.next(L::kAs), ++nd;
                    if (more && !(ok = dprobs())) break;
                }
            } else {
                for (int j = 0; ok && j < n; ++j) {
                    const bool more = j + 1 < n;
                    if (more && !(ok = scores())) break;
                    if (!(ok = wait.all(&bar.dp_read, pq))) break;
                    pq ^= 1;
                    tc_fence_after();
                    if (more && !(ok = dprobs())) break;
                    if (!(ok = sum(tm + cQ, tm + (j & 1) * 128, aM + ua.i * kStep, bar.ds_full, nd, j, &bar.a_empty[ua.i], !more))) break;
                    ua.next(L::kAs), ++nd;
                }
                ub = rb;   // V is not summed over
            }
            ++nf;
        }
        if (!ok && elect_one()) {   // let the MMAs issued so far finish
            umma_commit(&bar.dead);
            tc_drain(&bar.dead, 0);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, half = warp >> 2;   // columns [64*half, +64) of a tile
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = quarter * 32 + lane;
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);
        const f32x2 sc2 = both(sc);
        // 32 columns of P or dS to the MMAs; kTwo: with what rounding took from them, 32 columns on
        auto hand_over = [&](uint32_t at, const float (&x)[32], uint64_t *full) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            tmem_st16(at, v);
            if constexpr (kTwo) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {   // a value that is not finite leaves a NaN
                    float e, f;
                    unpack2(fma2(pack2u(v[i] << 16, v[i] & 0xffff0000u), both(-1.f), pack2(x[2 * i], x[2 * i + 1])), e, f);
                    v[i] = pack_bf16(e, f);
                }
                tmem_st16(at + 32, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        };
        bool ok = true;
        int na = 0, nf = 0, nd = 0, ns = 0, s0 = 0, s1 = 0;   // ring tiles, pieces, dS, statistics, S by buffer so far
        int pieces = 0;
        BwdWork w, next;
        f32x2 nl2 = both(0.f), nd2 = both(0.f);               // dQ: the row's statistics
        // The next piece, and its row's statistics: fetched before the output of the one before goes out.
        auto fetch = [&] {
            if (!wait.all(&bar.work_full[pieces & 1], (pieces >> 1) & 1)) return false;
            next = bar.work[pieces & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.work_empty[pieces & 1]);
            ++pieces;
            if (next.kind == BWD_DQ) {
                griddep_wait();   // the statistics come from the launch before
                const int64_t at = next.head * a.stat_stride + static_cast<int64_t>(next.slot) * kTcTile + row;
                nl2 = both(a.nlse2[at]), nd2 = both(a.ndelta[at]);
            }
            return true;
        };
        ok = fetch();
        while (ok) {
            w = next;
            if (w.kind == BWD_NONE) break;
            const bool dkv = w.kind == BWD_DKV;
            __nv_bfloat16 *out0, *out1 = nullptr;   // dQ, or dV and dK
            int64_t ts0, ts1 = 0;
            if (dkv) {
                ts0 = a.dv_ts, ts1 = a.dk_ts;
                out0 = static_cast<__nv_bfloat16 *>(a.dv) + w.tok * ts0 + w.head * a.dv_hs;
                out1 = static_cast<__nv_bfloat16 *>(a.dk) + w.tok * ts1 + w.head * a.dk_hs;
            } else {
                ts0 = a.dq_ts;
                out0 = static_cast<__nv_bfloat16 *>(a.dq) + w.tok * ts0 + w.head * a.dq_hs;
            }
            float *part0 = nullptr, *part1 = nullptr;   // a share's dV and dK
            const int64_t part_ts = static_cast<int64_t>(a.Hk) * a.D;
            if (kShares && dkv) {
                part0 = a.part + ((w.head >> 16) * 2 * static_cast<int64_t>(a.sk.T) + w.tok) * part_ts + (w.head & 0xffff) * a.D;
                part1 = part0 + a.sk.T * part_ts;
            }
            if (kShares && w.n == 0 && dkv) {
                if (row < w.rows)
                    for (int c = half * 4; c < a.D; c += 8) {
                        *reinterpret_cast<uint4 *>(part0 + row * part_ts + c) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(part1 + row * part_ts + c) = make_uint4(0, 0, 0, 0);
                    }
                ok = fetch();
                continue;
            }
            if (w.n == 0) {   // nothing on the other side
                if (row < w.rows)
                    for (int c = half * 8; c < a.D; c += 16) {
                        *reinterpret_cast<uint4 *>(out0 + row * ts0 + c) = make_uint4(0, 0, 0, 0);
                        if (dkv) *reinterpret_cast<uint4 *>(out1 + row * ts1 + c) = make_uint4(0, 0, 0, 0);
                    }
                ok = fetch();
                continue;
            }
            if (dkv) {
                const uint32_t tPh = tm + cP + lane_base + half * 64;
                const int key = w.t0 + row;
                int qt = w.first;
                for (int j = 0; j < w.n; ++j, ++nd, ++ns) {
                    const ulonglong2 *nlse2 = reinterpret_cast<const ulonglong2 *>(stats + (ns & 1) * 2 * kTcTile + half * 64);
                    const ulonglong2 *ndelta = nlse2 + kTcTile / 4;   // packed pairs of fp32, as they lie
                    const int buf = kTwoS ? j & 1 : 0;
                    const uint32_t tSh = tm + buf * 128 + lane_base + half * 64;
                    int &sn = buf ? s1 : s0;
                    if (!(ok = wait.all(&bar.st_full[ns & 1], (ns >> 1) & 1))) break;
                    if (!(ok = wait.all(&bar.s_full[buf], sn & 1))) break;
                    ++sn;
                    tc_fence_after();
                    uint32_t s[2][32];
                    tmem_ld32(tSh, s[0]);
                    tmem_ld32(tSh + 32, s[1]);
                    tmem_ld_wait();
                    float p[2][32];
                    // causal: query i sees the key from i = key - off on; the warp's last key is its tightest
                    const bool cut = a.causal && qt * kTcTile < w.t0 + quarter * 32 + 31 - w.off;
                    const int lim = key - w.off - qt * kTcTile - half * 64;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const ulonglong2 l = nlse2[c * 8 + i];
                            const uint32_t *x = &s[c][4 * i];
                            unpack2(fma2(pack2u(x[0], x[1]), sc2, l.x), p[c][4 * i], p[c][4 * i + 1]);
                            unpack2(fma2(pack2u(x[2], x[3]), sc2, l.y), p[c][4 * i + 2], p[c][4 * i + 3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[c][4 * i + e] = ex2(p[c][4 * i + e]);
                        }
                        if (cut) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i < lim) p[c][i] = 0.f;
                        }
                        hand_over(tSh + c * 16, p[c], &bar.p_full[ns & 1][c]);
                    }
                    if (!(ok = wait.all(&bar.dp_full, nd & 1))) break;
                    tc_fence_after();
                    tmem_ld32(tPh, s[0]);
                    tmem_ld32(tPh + 32, s[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const ulonglong2 d = ndelta[c * 8 + i];
                            const uint32_t *x = &s[c][4 * i];
                            float *y = &p[c][4 * i];   // dS in its place
                            unpack2(mul2(pack2(y[0], y[1]), add2(pack2u(x[0], x[1]), d.x)), y[0], y[1]);
                            unpack2(mul2(pack2(y[2], y[3]), add2(pack2u(x[2], x[3]), d.y)), y[2], y[3]);
                        }
                        hand_over(tPh + c * 16, p[c], &bar.ds_full[nd & 1][c]);
                    }
                    if (++qt == w.first + w.per) qt = w.first;
                }
            } else {
                const uint32_t tPh = tm + cP2 + lane_base + half * 64;
                const int last = w.t0 + row + w.off;   // causal: last key of the row
                for (int j = 0; j < w.n; ++j, ++nd) {
                    const uint32_t tSj = tm + (j & 1) * 128 + lane_base + half * 64;
                    int &sn = j & 1 ? s1 : s0;
                    if (!(ok = wait.all(&bar.s_full[j & 1], sn & 1))) break;
                    ++sn;
                    tc_fence_after();
                    uint32_t s[2][32];
                    tmem_ld32(tSj, s[0]);
                    tmem_ld32(tSj + 32, s[1]);
                    tmem_ld_wait();
                    float p[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            unpack2(fma2(pack2u(s[c][i], s[c][i + 1]), sc2, nl2), p[c][i], p[c][i + 1]);
                            p[c][i] = ex2(p[c][i]), p[c][i + 1] = ex2(p[c][i + 1]);
                        }
                    const int k0 = j * kTcTile, keys = min(kTcTile, w.olen - k0);
                    if (keys < kTcTile || (a.causal && k0 + kTcTile - 1 > w.t0 + quarter * 32 + w.off)) {
                        const int lim = (a.causal ? min(keys, last + 1 - k0) : keys) - half * 64;
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i >= lim) p[i / 32][i % 32] = 0.f;
                    }
                    if (!(ok = wait.all(&bar.dp_full, nd & 1))) break;
                    tc_fence_after();
                    tmem_ld32(tPh, s[0]);
                    tmem_ld32(tPh + 32, s[1]);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.dp_read);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)   // dS in its place
                            unpack2(mul2(pack2(p[c][i], p[c][i + 1]), add2(pack2u(s[c][i], s[c][i + 1]), nd2)), p[c][i], p[c][i + 1]);
                        hand_over(tSj + c * 16, p[c], &bar.ds_full[nd & 1][c]);
                    }
                }
            }
            if (!ok || !(ok = fetch()) || !(ok = wait.all(&bar.fin, nf & 1))) break;
            ++nf;
            na += w.n;
            tc_fence_after();
            uint8_t *tile = sa + (na - 1) % L::kAs * L::kTile;   // of the last tile: no longer read, not yet loaded again
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.acc_free);
            };
            if (kShares && dkv) {
                tc_store_fp32<KS>(half, tile, tm + cV + lane_base, 1.f, quarter * 32, w.rows, part0, part_ts, a.D, [] {});
                tc_store_fp32<KS>(half, tile, tm + cK + lane_base, a.scale, quarter * 32, w.rows, part1, part_ts, a.D, release);
            } else if (dkv) {
                tc_store_half<KS>(half, tile, tm + cV + lane_base, 1.f, quarter * 32, w.rows, out0, ts0, a.D, [] {});
                __syncwarp();
                tc_store_half<KS>(half, tile, tm + cK + lane_base, a.scale, quarter * 32, w.rows, out1, ts1, a.D, release);
            } else {
                tc_store_half<KS>(half, tile, tm + cQ + lane_base, a.scale, quarter * 32, w.rows, out0, ts0, a.D, release);
            }
            fence_proxy_async_smem();   // the slot goes back to the loads
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.staged[(nf - 1) & 1]);
        }
        tc_fence_before();
    }
    griddep_wait();   // also where nothing was read of the launch before: the grid must not end ahead of it
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

}  // namespace lce
