// Attention forward on the tensor cores (bf16).
//
// One CTA takes 128 query rows of one head and walks the keys in tiles of
// 128, with a running maximum and sum per row (one thread a row); two CTAs
// share an SM, so that one's softmax runs beside the other's MMAs. 192
// threads: warps 0-3 softmax, warp 4 TMA loads, warp 5 MMA issue.
//   S = Q K^T        128 x 128 fp32 in TMEM
//   P = 2^(S - m)    bf16, written over S in TMEM, the A operand of
//   O += P V         fp32 in TMEM
// The maximum a row's exponents refer to moves only when it grows by more than
// 2^8 (kLazy): until then P stays below 256 and O needs no rescaling, which
// costs a round trip of O through registers. The last reference divides out.
#pragma once

#include "lce_attn_tc.cuh"

namespace lce {

constexpr int kFwdThreads = 192;
constexpr float kLazy = 8.f;

template <int KS>
struct FwdSmem : Chan<KS> {
    using Chan<KS>::kTile;
    static constexpr int kBars = 3 * kTile;              // Q, two ring slots
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

    const int h = blockIdx.x % a.Hq, hk = h / a.group;
    // longest rows first: under a causal mask the last tiles have the most keys
    const int slot = gridDim.x / a.Hq - 1 - blockIdx.x / a.Hq;
    const TileInfo t = tile_info<kTcTile>(a.sq, a.sk, slot);
    if (blockIdx.x == 0 && warp == 4) {
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

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, 4);
        mbar_init(o_done, 1);
        mbar_init(fin, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t tS = tmem, tO = tmem + 128;
    const TcWaits wait{abort_flag, a.status};

    if (warp == 4) {
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
    } else if (warp == 5) {
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
                tc_mma_tokens<false>(tO, tS, dv, idO, j > 0);
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
        const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
        const int row = warp * 32 + lane;
        const int last = t.t0 + row + off;   // causal: last key of the row
        const float sc = fmaxf(fabsf(a.scale_log2), 1.2e-38f);   // never 0: a masked -inf stays -inf
        float m = -INFINITY, l = 0.f;   // reference maximum (of S, unscaled) and sum
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!(ok = wait.all(s_full, j & 1))) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + lane_base + c * 32, s[c]);
            tmem_ld_wait();
            const int k0 = j * kTcTile;
            const int keys = min(kTcTile, t.olen - k0);
            // the warp's first row is its tightest
            if (keys < kTcTile || (a.causal && k0 + kTcTile - 1 > t.t0 + warp * 32 + off)) {
                const int lim = a.causal ? min(keys, last + 1 - k0) : keys;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + i >= lim) s[c][i] = 0xff800000u;   // -inf
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(s[c][i]));
            const bool grow = (mx - m) * sc > kLazy || (m == -INFINITY && mx > m);
            if (__any_sync(0xffffffffu, grow)) {
                const float next = grow ? mx : m;
                if (j > 0) {
                    const float fix = grow ? ex2((m - next) * sc) : 1.f;   // m = -inf: 2^-inf = 0 on an O of zeros
                    l *= fix;
                    if (!(ok = wait.all(o_done, (j - 1) & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < NB * 2; ++c) {
                        if (c * 32 >= KS * 16) break;
                        uint32_t v[32];
                        tmem_ld32(tO + lane_base + c * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fix);
                        tmem_st32(tO + lane_base + c * 32, v);
                    }
                }
                m = next;
            }
            const float base = m == -INFINITY ? 0.f : m * sc;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = ex2(fmaf(__uint_as_float(s[2 * c + i / 16][2 * (i % 16)]), sc, -base));
                    const float y = ex2(fmaf(__uint_as_float(s[2 * c + i / 16][2 * (i % 16) + 1]), sc, -base));
                    sum[i & 3] += x + y;
                    p[i] = pack_bf16(x, y);
                }
                tmem_st32(tS + lane_base + c * 32, p);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (ok) ok = wait.all(o_done, (n - 1) & 1);
        if (ok) {
            tc_fence_after();
            const float inv = l != 0.f ? 1.f / l : 0.f;   // l of an empty row is 0; NaN stays
            tc_store_rows<NB>(sq, tO + lane_base, inv, warp * 32, rows, o, a.o_ts, a.D);
            if (row < rows) lse[row] = l == 0.f ? -INFINITY : (m * sc + log2f(l)) * (1.f / kAttnLog2e);
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

}  // namespace lce
