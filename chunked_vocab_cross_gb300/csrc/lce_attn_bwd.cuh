// Attention backward on the tensor cores (bf16): two kinds of blocks, so that
// every gradient is summed in TMEM by one CTA in a fixed order, without atomics
// and without a gradient buffer of partial sums. The probabilities are
// recomputed in both (7 products of tiles instead of 5).
//
// dq_block: 128 query rows, walking the keys.
//   S = Q K^T, dP = dO V^T (128 x 128 fp32 in TMEM, rows = queries)
//   dS = 2^(S - lse) (dP - delta), bf16 over S in TMEM;  dQ += dS K
// dkv_block: 128 keys of one key head, walking the queries of its query heads.
//   S^T = K Q^T, dP^T = V dO^T (rows = keys)
//   P^T over S^T: dV += P^T dO;  dS^T over dP^T: dK += dS^T Q
// P and dS go back to TMEM as the A operands, so they never touch shared
// memory.
//
// 320 threads: warps 0-7 the elementwise part (two threads a row, 64 columns
// each), warp 8 TMA loads, warp 9 MMA issue. One CTA an SM: dkv fills the 512
// columns of TMEM (S, dP, dV, dK), and the tiles fill the shared memory.
#pragma once

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kBwdThreads = 320;

template <int KS>
struct DqSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kKs = 3, kVs = 2;                         // ring slots of K and V
    static constexpr int kBars = (2 + kKs + kVs) * kTile;          // Q, dO, rings
    static constexpr int kBytes = kBars + 168;
};

// Block `block` of `blocks`; so too in dkv_block.
template <int KS>
__device__ __forceinline__ void dq_block(const AttnArgs &a, const AttnMaps &maps, uint8_t *smem, int block, int blocks) {
    using L = DqSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *sq = smem, *sg = smem + L::kTile, *sk = smem + 2 * L::kTile, *sv = sk + L::kKs * L::kTile;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint64_t *k_full = bars, *k_empty = bars + 3, *v_full = bars + 6, *v_empty = bars + 8, *q_full = bars + 10,
             *s_full = bars + 11 /* two */, *dp_full = bars + 13, *ds_full = bars + 14, *fin = bars + 15;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 16);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 16; ++i) mbar_init(&bars[i], i == 14 ? 8 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    const int h = block % a.Hq, hk = h / a.group;
    const int slot = blocks / a.Hq - 1 - block / a.Hq;   // under a causal mask the last tiles have the most keys
    const TileInfo t = tile_info<kTcTile>(a.sq, a.sk, slot);
    const int rows = min(kTcTile, t.len - t.t0);
    if (t.t0 < 0 || rows <= 0) return;
    const int off = t.olen - t.len;
    const int kend = a.causal ? min(t.olen, t.t0 + rows + off) : t.olen;
    const int64_t tok = t.s0 + t.t0;
    __nv_bfloat16 *dq = static_cast<__nv_bfloat16 *>(a.dq) + tok * a.dq_ts + h * a.dq_hs;
    if (kend <= 0) {
        const int per = a.D / 8;
        for (int i = threadIdx.x; i < rows * per; i += kBwdThreads)
            *reinterpret_cast<uint4 *>(dq + (i / per) * a.dq_ts + (i % per) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    const int n = (kend + kTcTile - 1) / kTcTile;

    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t tS[2] = {tmem, tmem + 128}, tP = tmem + 256, tQ = tmem + 384;
    const TcWaits wait{abort_flag, a.status};

    if (warp == 8) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, 2 * L::kTile);
            tc_load_tile<NB>(sq, &maps.q, q_full, h, static_cast<int>(tok));
            tc_load_tile<NB>(sg, &maps.dO, q_full, h, static_cast<int>(tok));
            int j = 0, kl = 0, vl = 0;   // loads issued of each ring
            for (; j < n; ++j) {
                const int ki = j % L::kKs, vi = j % L::kVs, at = t.o0 + j * kTcTile;
                if (!wait(&k_empty[ki], ((j / L::kKs) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(&k_full[ki], L::kTile);
                tc_load_tile<NB>(sk + ki * L::kTile, &maps.k, &k_full[ki], hk, at);
                ++kl;
                if (!wait(&v_empty[vi], ((j / L::kVs) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(&v_full[vi], L::kTile);
                tc_load_tile<NB>(sv + vi * L::kTile, &maps.v, &v_full[vi], hk, at);
                ++vl;
            }
            if (j < n) {
                tc_drain(q_full, 0);
                for (int i = max(0, kl - L::kKs); i < kl; ++i) tc_drain(&k_full[i % L::kKs], (i / L::kKs) & 1);
                for (int i = max(0, vl - L::kVs); i < vl; ++i) tc_drain(&v_full[i % L::kVs], (i / L::kVs) & 1);
            }
        }
    } else if (warp == 9) {
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false), idQ = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint32_t idSn = idS | (a.scale < 0.f ? kIdescNegA : 0);
        const uint64_t dQ = tc_desc_k(sq), dG = tc_desc_k(sg);
        // S_j from K_j; its tokens past the sequence's end are zeroed for the sum that follows
        auto scores = [&](int j) {
            const int ki = j % L::kKs;
            if (!wait.all(&k_full[ki], (j / L::kKs) & 1)) return false;
            const int keys = min(kTcTile, t.olen - j * kTcTile);
            if (keys < kTcTile) tc_zero_rows<NB>(sk + ki * L::kTile, keys);
            if (elect_one()) {
                tc_fence_after();
                tc_mma_scores<KS>(tS[j & 1], dQ, tc_desc_k(sk + ki * L::kTile), idSn);
                umma_commit(&s_full[j & 1]);
            }
            __syncwarp();
            return true;
        };
        auto dprobs = [&](int j) {
            const int vi = j % L::kVs;
            if (!wait.all(&v_full[vi], (j / L::kVs) & 1)) return false;
            const int keys = min(kTcTile, t.olen - j * kTcTile);
            if (keys < kTcTile) tc_zero_rows<NB>(sv + vi * L::kTile, keys);
            if (elect_one()) {
                tc_fence_after();
                tc_mma_scores<KS>(tP, dG, tc_desc_k(sv + vi * L::kTile), idS);
                umma_commit(&v_empty[vi]);
                umma_commit(dp_full);
            }
            __syncwarp();
            return true;
        };
        bool ok = wait.all(q_full, 0) && scores(0) && dprobs(0);
        for (int j = 0; ok && j < n; ++j) {
            if (j + 1 < n && !(ok = scores(j + 1))) break;
            if (!(ok = wait.all(ds_full, j & 1))) break;
            tc_fence_after();
            if (j + 1 < n && !(ok = dprobs(j + 1))) break;
            if (elect_one()) {
                const uint64_t dK = tc_desc_mn(sk + (j % L::kKs) * L::kTile);
                tc_mma_tokens<true>(tQ, tS[j & 1], dK, idQ, j > 0);
                umma_commit(&k_empty[j % L::kKs]);
                if (j + 1 == n) umma_commit(fin);
            }
            __syncwarp();
        }
        if (!ok && elect_one()) {
            umma_commit(fin);
            tc_drain(fin, 0);
        }
    } else {
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int half = warp >> 2;   // columns [64*half, +64)
        const int row = (warp & 3) * 32 + lane;
        const int last = t.t0 + row + off;
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);
        const int64_t at = h * a.stat_stride + static_cast<int64_t>(slot) * kTcTile + row;
        const float lse2 = a.lse2[at], delta = a.delta[at];
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const uint32_t tSj = tS[j & 1] + lane_base + half * 64;
            if (!(ok = wait.all(&s_full[j & 1], (j >> 1) & 1))) break;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(tSj, s[0]);
            tmem_ld32(tSj + 32, s[1]);
            tmem_ld_wait();
            float p[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) p[i] = ex2(fmaf(__uint_as_float(s[i / 32][i % 32]), sc, -lse2));
            const int k0 = j * kTcTile, keys = min(kTcTile, t.olen - k0);
            if (keys < kTcTile || (a.causal && k0 + kTcTile - 1 > t.t0 + (warp & 3) * 32 + off)) {
                const int lim = (a.causal ? min(keys, last + 1 - k0) : keys) - half * 64;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= lim) p[i] = 0.f;
            }
            if (!(ok = wait.all(dp_full, j & 1))) break;
            tc_fence_after();
            tmem_ld32(tP + lane_base + half * 64, s[0]);
            tmem_ld32(tP + lane_base + half * 64 + 32, s[1]);
            tmem_ld_wait();
            uint32_t ds[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
                ds[i] = pack_bf16(p[2 * i] * (__uint_as_float(s[i / 16][2 * (i % 16)]) - delta),
                                  p[2 * i + 1] * (__uint_as_float(s[i / 16][2 * (i % 16) + 1]) - delta));
            tmem_st32(tSj, ds);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        if (ok && wait.all(fin, 0)) {
            tc_fence_after();
            tc_store_half<KS>(half, sq, tQ + lane_base, a.scale, (warp & 3) * 32, rows, dq, a.dq_ts, a.D, [] {});
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KS>
struct DkvSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kQs = 3, kGs = 2;                             // ring slots of Q and dO
    static constexpr int kStat = 2 * kTcTile * 4;                      // lse2 and delta of a Q tile; two slots
    static constexpr int kStats = (2 + kQs + kGs) * kTile;             // K, V, rings
    static constexpr int kBars = kStats + 2 * kStat;
    static constexpr int kBytes = kBars + 168;   // no room for alignment slack: the kernel checks the base it gets
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

template <int KS>
__device__ __forceinline__ void dkv_block(const AttnArgs &a, const AttnMaps &maps, uint8_t *smem, int block) {
    using L = DkvSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *sk = smem, *sv = smem + L::kTile, *sq = smem + 2 * L::kTile, *sg = sq + L::kQs * L::kTile;
    float *stats = reinterpret_cast<float *>(smem + L::kStats);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint64_t *q_full = bars, *q_empty = bars + 3, *g_full = bars + 6, *g_empty = bars + 8, *kv_full = bars + 10,
             *s_full = bars + 11, *dp_full = bars + 12, *p_full = bars + 13, *ds_full = bars + 14, *fin = bars + 15,
             *st_full = bars + 16 /* two */;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 18);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 18; ++i) mbar_init(&bars[i], i == 13 || i == 14 ? 8 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    const int hk = block % a.Hk, slot = block / a.Hk;   // under a causal mask the first tiles have the most queries
    const TileInfo t = tile_info<kTcTile>(a.sk, a.sq, slot);      // own side: keys
    const int keys = min(kTcTile, t.len - t.t0);
    if (t.t0 < 0 || keys <= 0) return;
    const int off = t.len - t.olen;   // causal: query i sees keys [0, i + off]
    const int64_t tok = t.s0 + t.t0;
    __nv_bfloat16 *dk = static_cast<__nv_bfloat16 *>(a.dk) + tok * a.dk_ts + hk * a.dk_hs;
    __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv) + tok * a.dv_ts + hk * a.dv_hs;
    const int first = a.causal ? max(0, t.t0 - off) / kTcTile : 0;   // first query tile that sees the tile's first key
    const int per_head = (t.olen + kTcTile - 1) / kTcTile - first;
    if (per_head <= 0) {
        const int per = a.D / 8;
        for (int i = threadIdx.x; i < keys * per; i += kBwdThreads) {
            *reinterpret_cast<uint4 *>(dk + (i / per) * a.dk_ts + (i % per) * 8) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(dv + (i / per) * a.dv_ts + (i % per) * 8) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int n = per_head * a.group;

    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;
    const TcWaits wait{abort_flag, a.status};

    if (warp == 8) {
        if (lane == 0) {
            mbar_arrive_expect_tx(kv_full, 2 * L::kTile);
            tc_load_tile<NB>(sk, &maps.k, kv_full, hk, static_cast<int>(tok));
            tc_load_tile<NB>(sv, &maps.v, kv_full, hk, static_cast<int>(tok));
            const int64_t qslot0 = slot_base<kTcTile>(a.sq, t.b);
            int h = hk * a.group, qt = first, j = 0, ql = 0, gl = 0, sl = 0;
            for (; j < n; ++j) {
                const int qi = j % L::kQs, gi = j % L::kGs, at = t.o0 + qt * kTcTile;
                if (!wait(&q_empty[qi], ((j / L::kQs) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(&q_full[qi], L::kTile);
                tc_load_tile<NB>(sq + qi * L::kTile, &maps.q, &q_full[qi], h, at);
                ++ql;
                if (!wait(&g_empty[gi], ((j / L::kGs) & 1) ^ 1)) break;
                mbar_arrive_expect_tx(&g_full[gi], L::kTile);
                tc_load_tile<NB>(sg + gi * L::kTile, &maps.dO, &g_full[gi], h, at);
                ++gl;
                // the statistics' slot is free once dK_(j-2), which follows their last use, has been summed
                if (j >= 2 && !wait(&q_empty[(j - 2) % L::kQs], ((j - 2) / L::kQs) & 1)) break;
                const int64_t st = h * a.stat_stride + (qslot0 + qt) * kTcTile;
                float *dst = stats + (j & 1) * 2 * kTcTile;
                mbar_arrive_expect_tx(&st_full[j & 1], L::kStat);
                bulk_load(dst, a.lse2 + st, kTcTile * 4, &st_full[j & 1]);
                bulk_load(dst + kTcTile, a.delta + st, kTcTile * 4, &st_full[j & 1]);
                ++sl;
                if (++qt == first + per_head) qt = first, ++h;
            }
            if (j < n) {
                tc_drain(kv_full, 0);
                for (int i = max(0, ql - L::kQs); i < ql; ++i) tc_drain(&q_full[i % L::kQs], (i / L::kQs) & 1);
                for (int i = max(0, gl - L::kGs); i < gl; ++i) tc_drain(&g_full[i % L::kGs], (i / L::kGs) & 1);
                for (int i = max(0, sl - 2); i < sl; ++i) tc_drain(&st_full[i & 1], (i >> 1) & 1);
            }
        }
    } else if (warp == 9) {
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false), idG = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint32_t idSn = idS | (a.scale < 0.f ? kIdescNegA : 0);
        const uint64_t dK = tc_desc_k(sk), dV = tc_desc_k(sv);
        auto queries = [&](int j) { return min(kTcTile, t.olen - (first + j % per_head) * kTcTile); };
        auto scores = [&](int j) {
            const int qi = j % L::kQs;
            if (!wait.all(&q_full[qi], (j / L::kQs) & 1)) return false;
            const int q = queries(j);
            if (q < kTcTile) tc_zero_rows<NB>(sq + qi * L::kTile, q);
            if (elect_one()) {
                tc_fence_after();
                tc_mma_scores<KS>(tS, dK, tc_desc_k(sq + qi * L::kTile), idSn);
                umma_commit(s_full);
            }
            __syncwarp();
            return true;
        };
        auto dprobs = [&](int j) {
            const int gi = j % L::kGs;
            if (!wait.all(&g_full[gi], (j / L::kGs) & 1)) return false;
            const int q = queries(j);
            if (q < kTcTile) tc_zero_rows<NB>(sg + gi * L::kTile, q);
            if (elect_one()) {
                tc_fence_after();
                tc_mma_scores<KS>(tP, dV, tc_desc_k(sg + gi * L::kTile), idS);
                umma_commit(dp_full);
            }
            __syncwarp();
            return true;
        };
        // acc (+)= A[keys x queries] . tile, A in two halves of 64 queries, 64 columns apart
        auto gather = [&](uint32_t acc, uint32_t A, const uint8_t *tile, int j, uint64_t *release) {
            if (elect_one()) {
                tc_fence_after();
                tc_mma_tokens<true>(acc, A, tc_desc_mn(tile), idG, j > 0);
                umma_commit(release);
            }
            __syncwarp();
        };
        bool ok = wait.all(kv_full, 0) && scores(0) && dprobs(0);
        for (int j = 0; ok && j < n; ++j) {
            if (!(ok = wait.all(p_full, j & 1))) break;
            gather(tV, tS, sg + (j % L::kGs) * L::kTile, j, &g_empty[j % L::kGs]);
            if (j + 1 < n && !(ok = scores(j + 1))) break;
            if (!(ok = wait.all(ds_full, j & 1))) break;
            gather(tK, tP, sq + (j % L::kQs) * L::kTile, j, &q_empty[j % L::kQs]);
            if (j + 1 < n && !(ok = dprobs(j + 1))) break;
        }
        if (elect_one()) {
            umma_commit(fin);
            if (!ok) tc_drain(fin, 0);
        }
    } else {
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int half = warp >> 2;
        const int key = t.t0 + (warp & 3) * 32 + lane;
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);
        const uint32_t tSh = tS + lane_base + half * 64, tPh = tP + lane_base + half * 64;
        bool ok = true;
        int qt = first;
        for (int j = 0; j < n; ++j) {
            const float4 *lse2 = reinterpret_cast<const float4 *>(stats + (j & 1) * 2 * kTcTile + half * 64);
            const float4 *delta = lse2 + kTcTile / 4;
            if (!(ok = wait.all(&st_full[j & 1], (j >> 1) & 1))) break;
            if (!(ok = wait.all(s_full, j & 1))) break;
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(tSh, s[0]);
            tmem_ld32(tSh + 32, s[1]);
            tmem_ld_wait();
            float p[64];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 l = lse2[i];
                const uint32_t *x = &s[i / 8][4 * (i % 8)];
                p[4 * i] = ex2(fmaf(__uint_as_float(x[0]), sc, -l.x));
                p[4 * i + 1] = ex2(fmaf(__uint_as_float(x[1]), sc, -l.y));
                p[4 * i + 2] = ex2(fmaf(__uint_as_float(x[2]), sc, -l.z));
                p[4 * i + 3] = ex2(fmaf(__uint_as_float(x[3]), sc, -l.w));
            }
            // causal: query i sees the key from i = key - off on; the warp's last key is its tightest
            if (a.causal && qt * kTcTile < t.t0 + (warp & 3) * 32 + 31 - off) {
                const int lim = key - off - qt * kTcTile - half * 64;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i < lim) p[i] = 0.f;
            }
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
            tmem_st32(tSh, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            if (!(ok = wait.all(dp_full, j & 1))) break;
            tc_fence_after();
            tmem_ld32(tPh, s[0]);
            tmem_ld32(tPh + 32, s[1]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 d = delta[i];
                const uint32_t *x = &s[i / 8][4 * (i % 8)];
                w[2 * i] = pack_bf16(p[4 * i] * (__uint_as_float(x[0]) - d.x), p[4 * i + 1] * (__uint_as_float(x[1]) - d.y));
                w[2 * i + 1] = pack_bf16(p[4 * i + 2] * (__uint_as_float(x[2]) - d.z),
                                         p[4 * i + 3] * (__uint_as_float(x[3]) - d.w));
            }
            tmem_st32(tPh, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
            if (++qt == first + per_head) qt = first;
        }
        if (ok && wait.all(fin, 0)) {
            tc_fence_after();
            tc_store_half<KS>(half, sv, tV + lane_base, 1.f, (warp & 3) * 32, keys, dv, a.dv_ts, a.D, [] {});
            tc_store_half<KS>(half, sk, tK + lane_base, a.scale, (warp & 3) * 32, keys, dk, a.dk_ts, a.D, [] {});
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both in one launch, the longer dK/dV blocks first: they share nothing but
// their inputs, so the dQ blocks fill the SMs that the others leave idle.
template <int KS>
__global__ void __launch_bounds__(kBwdThreads, 1) k_attn_bwd(const __grid_constant__ AttnArgs a,
                                                             const __grid_constant__ AttnMaps maps, int dkv_blocks) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {   // swizzled tiles need it; a launch has no other way to say so
        if (threadIdx.x == 0) atomicOr(a.status, kDevTimeout);
        return;
    }
    const int block = blockIdx.x;
    if (threadIdx.x == 32) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        tma_prefetch_map(&maps.dO);
    }
    if (block < dkv_blocks) dkv_block<KS>(a, maps, smem, block);
    else dq_block<KS>(a, maps, smem, block - dkv_blocks, gridDim.x - dkv_blocks);
}

}  // namespace lce
