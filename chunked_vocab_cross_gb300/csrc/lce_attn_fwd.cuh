// Attention forward on the tensor cores (bf16).
//
// One CTA takes 128 query rows of one head and walks the keys in tiles of
// 128, with a running maximum and sum per row (two threads a row, 64 keys
// each, that exchange their maxima); two CTAs share an SM, so that one's
// softmax runs beside the other's MMAs. 320 threads: warps 0-7 softmax, warp 8
// TMA loads, warp 9 MMA issue.
//   S = Q K^T        128 x 128 fp32 in TMEM
//   P = 2^(S - m)    bf16, written over S in TMEM, the A operand of
//   O += P V         fp32 in TMEM
// The maximum a row's exponents refer to moves only when it grows by more than
// 2^8 (kLazy): until then P stays below 256 and O needs no rescaling, which
// costs a round trip of O through registers. The last reference divides out.
#pragma once

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kFwdThreads = 320;
constexpr float kLazy = 8.f;

template <int KS>
struct FwdSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kMax = 3 * kTile;               // Q, two ring slots
    static constexpr int kBars = kMax + 4 * kTcTile * 4; // row maxima: two buffers of two halves
    static constexpr int kBytes = kBars + 128 + 1024;    // alignment slack
};

template <int KS>
__global__ void __launch_bounds__(kFwdThreads, 2) k_attn_fwd(const __grid_constant__ AttnArgs a,
                                                             const __grid_constant__ AttnMaps maps) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    using L = FwdSmem<KS>;
    constexpr int NB = L::NB;
    uint8_t *sq = smem, *ring = smem + L::kTile;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBars);
    uint64_t *full = bars, *empty = bars + 2, *q_full = bars + 4, *s_full = bars + 5, *p_full = bars + 6,
             *o_done = bars + 7, *fin = bars + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 9);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 8);
        mbar_init(o_done, 1);
        mbar_init(fin, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    const int h = blockIdx.x % a.Hq, hk = h / a.group;
    // longest rows first: under a causal mask the last tiles have the most keys
    const int slot = gridDim.x / a.Hq - 1 - blockIdx.x / a.Hq;
    const TileInfo t = tile_info<kTcTile>(a.sq, a.sk, slot);
    if (blockIdx.x == 0 && warp == 8) {
        check_offsets(a.sq, a.status);
        check_offsets(a.sk, a.status);
    }
    const int rows = min(kTcTile, t.len - t.t0);
    if (t.t0 < 0 || rows <= 0) return;
    const int off = t.olen - t.len;   // causal: row i sees keys [0, i + off]
    const int kend = a.causal ? min(t.olen, t.t0 + rows + off) : t.olen;
    const int64_t tok = t.s0 + t.t0;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + tok * a.o_ts + h * a.o_hs;
    float *lse = a.lse + static_cast<int64_t>(h) * a.sq.T + tok;
    if (kend <= 0) {   // no row of the tile sees a key
        const int per = a.D / 8;
        for (int i = threadIdx.x; i < rows * per; i += kFwdThreads)
            *reinterpret_cast<uint4 *>(o + (i / per) * a.o_ts + (i % per) * 8) = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < rows; i += kFwdThreads) lse[i] = -INFINITY;
        return;
    }
    const int n = (kend + kTcTile - 1) / kTcTile;

    if (warp == 9) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t tS = tmem, tO = tmem + 128;
    const TcWaits wait{abort_flag, a.status};

    if (warp == 8) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, L::kTile);
            tc_load_tile<NB>(sq, &maps.q, q_full, h, static_cast<int>(tok));
            int it = 0;   // ring: K0 V0 K1 V1 ...
            bool ok = true;
            for (; it < 2 * n; ++it) {
                if (!(ok = wait(&empty[it & 1], ((it >> 1) & 1) ^ 1))) break;
                mbar_arrive_expect_tx(&full[it & 1], L::kTile);
                tc_load_tile<NB>(ring + (it & 1) * L::kTile, it & 1 ? &maps.v : &maps.k, &full[it & 1], hk,
                                 t.o0 + (it >> 1) * kTcTile);
            }
            if (!ok) {
                tc_drain(q_full, 0);
                for (int i = max(0, it - 2); i < it; ++i) tc_drain(&full[i & 1], (i >> 1) & 1);
            }
        }
    } else if (warp == 9) {
        const uint32_t idS = idesc_f32acc(1, 128, 128, false, false) | (a.scale < 0.f ? kIdescNegA : 0);
        const uint32_t idO = idesc_f32acc(1, 128, KS * 16, false, true);
        const uint64_t dq = tc_desc_k(sq), dk = tc_desc_k(ring), dv = tc_desc_mn(ring + L::kTile);
        bool ok = wait.all(q_full, 0);
        for (int j = 0; ok && j < n; ++j) {
            if (!(ok = wait.all(&full[0], j & 1))) break;
            if (elect_one()) {
                tc_fence_after();
                tc_mma_scores<KS>(tS, dq, dk, idS);
                umma_commit(&empty[0]);
                umma_commit(s_full);
            }
            __syncwarp();
            if (!(ok = wait.all(&full[1], j & 1))) break;
            const int keys = min(kTcTile, t.olen - j * kTcTile);
            if (keys < kTcTile) tc_zero_rows<NB>(ring + L::kTile, keys);
            if (!(ok = wait.all(p_full, j & 1))) break;
            if (elect_one()) {
                tc_fence_after();
                tc_mma_tokens<true>(tO, tS, dv, idO, j > 0);
                umma_commit(&empty[1]);
                umma_commit(o_done);
            }
            __syncwarp();
        }
        if (!ok && elect_one()) {   // let the MMAs issued so far finish
            umma_commit(fin);
            tc_drain(fin, 0);
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;   // keys [64*half, +64) of a tile
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const int row = quarter * 32 + lane;
        const int last = t.t0 + row + off;   // causal: last key of the row
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);   // never 0: a masked -inf stays -inf
        const uint32_t tSh = tS + lane_base + half * 64;
        float *maxima = reinterpret_cast<float *>(smem + L::kMax);
        // what the row's other thread has to say (`slot`: one of two buffers in turn)
        auto exchange = [&](int slot, float v) {
            float *at = maxima + slot * 2 * kTcTile;
            at[half * kTcTile + row] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(quarter + 1) : "memory");
            return at[(half ^ 1) * kTcTile + row];
        };
        // a warp that gives up before an exchange must not leave its partner waiting in it; in all later
        // waits the partner gives up too, since this warp's share of P never comes
        auto leave = [&] { asm volatile("bar.arrive %0, 64;" ::"r"(quarter + 1) : "memory"); };
        float m = -INFINITY;                       // reference maximum (of S, unscaled)
        f32x2 l2 = both(0.f);                      // sum, of this thread's keys
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!(ok = wait.all(s_full, j & 1))) {
                leave();
                break;
            }
            tc_fence_after();
            const int k0 = j * kTcTile;
            const int keys = min(kTcTile, t.olen - k0);
            // the warp's first row is its tightest
            const bool cut = keys < kTcTile || (a.causal && k0 + kTcTile - 1 > t.t0 + quarter * 32 + off);
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
            top = fmaxf(top, exchange(j & 1, top));
            const bool grow = (top - m) * sc > kLazy || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grow)) {
                const float next = grow ? top : m;
                if (j > 0) {
                    const float fix = grow ? ex2((m - next) * sc) : 1.f;   // m = -inf: 2^-inf = 0 on an O of zeros
                    l2 = mul2(l2, both(fix));
                    if (!(ok = wait.all(o_done, (j - 1) & 1))) break;
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
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float x, y;
                unpack2(fma2(pack2u(s[i / 16][2 * (i % 16)], s[i / 16][2 * (i % 16) + 1]), sc2, base), x, y);
                x = ex2(x), y = ex2(y);
                l2 = add2(l2, pack2(x, y));
                p[i] = pack_bf16(x, y);
            }
            tmem_st32(tSh, p);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        if (ok && !(ok = wait.all(o_done, (n - 1) & 1))) leave();
        if (ok) {
            tc_fence_after();
            const float part = hsum2(l2), l = part + exchange(n & 1, part);
            const float inv = l != 0.f ? 1.f / l : 0.f;   // l of an empty row is 0; NaN stays
            tc_store_half<KS>(half, sq, tO + lane_base, inv, quarter * 32, rows, o, a.o_ts, a.D);
            if (half == 0 && row < rows) lse[row] = l == 0.f ? -INFINITY : (m * sc + log2f(l)) * (1.f / kAttnLog2e);
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

}  // namespace lce
