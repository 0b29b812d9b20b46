// Attention of fp32 tensors, in fp32 arithmetic: tiles of 64 queries by 64 keys in shared
// memory, 256 threads in a 16 x 16 grid, each with four query rows (or key
// rows) and every 16th column of each product. Bound by shared-memory loads
// (eight for sixteen multiply-adds).
#pragma once

#include "lce_attn.cuh"

namespace lce {

constexpr int kSimtTile = 64;
constexpr int kSimtThreads = 256;
constexpr int kSimtP = kSimtTile + 1;   // row pitch of a 64 x 64 tile: odd, so that columns are free of bank conflicts

constexpr int simt_smem(int DP, int operands, int tiles) {
    return (operands * kSimtTile * (DP + 1) + tiles * kSimtTile * kSimtP + 2 * kSimtTile) * 4;
}

// rows [0, 64) x [0, DP) of fp32 from `rows` token rows of D elements; zero outside
template <int DP>
__device__ __forceinline__ void simt_load(float *dst, const float *src, int64_t stride, int rows, int D) {
    for (int i = threadIdx.x; i < kSimtTile * DP; i += kSimtThreads) {
        const int r = i / DP, c = i % DP;
        dst[r * (DP + 1) + c] = (r < rows && c < D) ? src[r * stride + c] : 0.f;
    }
}

// acc[i][j] = A[ty*4+i] . B[tx+16j] over DP
template <int DP>
__device__ __forceinline__ void simt_dot(const float *A, const float *B, int ty, int tx, float (&acc)[4][4]) {
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int c = 0; c < DP; ++c) {
        float x[4], y[4];
        for (int i = 0; i < 4; ++i) x[i] = A[(ty * 4 + i) * (DP + 1) + c];
        for (int j = 0; j < 4; ++j) y[j] = B[(tx + 16 * j) * (DP + 1) + c];
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
}

// acc[i][c] += sum_j P[ty*4+i][j] * B[j][tx+16c]   (kT: P is read as P[j][ty*4+i])
template <int DP, bool kT>
__device__ __forceinline__ void simt_mix(const float *P, const float *B, int ty, int tx, float (&acc)[4][DP / 16]) {
    for (int j = 0; j < kSimtTile; ++j) {
        float x[4];
        for (int i = 0; i < 4; ++i) x[i] = kT ? P[j * kSimtP + ty * 4 + i] : P[(ty * 4 + i) * kSimtP + j];
        for (int c = 0; c < DP / 16; ++c) {
            const float y = B[j * (DP + 1) + tx + 16 * c];
            for (int i = 0; i < 4; ++i) acc[i][c] = fmaf(x[i], y, acc[i][c]);
        }
    }
}

template <int DP>
__device__ __forceinline__ void simt_store(float *dst, int64_t stride, int rows, int D, int ty, int tx, float mul,
                                           const float (&acc)[4][DP / 16]) {
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= rows) continue;
        for (int c = 0; c < DP / 16; ++c)
            if (tx + 16 * c < D) dst[r * stride + tx + 16 * c] = acc[i][c] * mul;
    }
}

template <int DP>
__global__ void __launch_bounds__(kSimtThreads) k_attn_fwd_simt(const AttnArgs a) {
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + kSimtTile * (DP + 1), *V = K + kSimtTile * (DP + 1), *P = V + kSimtTile * (DP + 1);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int h = blockIdx.x % a.Hq, hk = h / a.group;
    if (blockIdx.x == 0 && tid < 32) {
        check_offsets(a.sq, a.status);
        check_offsets(a.sk, a.status);
    }
    const TileInfo t = tile_info<kSimtTile>(a.sq, a.sk, blockIdx.x / a.Hq);
    const int rows = min(kSimtTile, t.len - t.t0);
    if (t.t0 < 0 || rows <= 0) return;
    const int off = t.olen - t.len;   // causal: row i sees keys [0, i + off]
    const int kend = a.causal ? min(t.olen, t.t0 + rows + off) : t.olen;
    simt_load<DP>(Q, static_cast<const float *>(a.q) + (t.s0 + t.t0) * a.q_ts + h * a.q_hs, a.q_ts, rows, a.D);
    float o[4][DP / 16] = {}, m[4], l[4] = {};
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY;
    for (int k0 = 0; k0 < kend; k0 += kSimtTile) {
        const int keys = min(kSimtTile, t.olen - k0);
        __syncthreads();
        simt_load<DP>(K, static_cast<const float *>(a.k) + (t.o0 + k0) * a.k_ts + hk * a.k_hs, a.k_ts, keys, a.D);
        simt_load<DP>(V, static_cast<const float *>(a.v) + (t.o0 + k0) * a.v_ts + hk * a.v_hs, a.v_ts, keys, a.D);
        __syncthreads();
        float s[4][4];
        simt_dot<DP>(Q, K, ty, tx, s);
        for (int i = 0; i < 4; ++i) {
            const int row = t.t0 + ty * 4 + i;
            const int lim = a.causal ? min(keys, row + off + 1 - k0) : keys;
            float mx = m[i];
            for (int j = 0; j < 4; ++j) {
                s[i][j] = tx + 16 * j < lim ? s[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float base = mx == -INFINITY ? 0.f : mx;
            const float fix = exp2f(m[i] - base);
            float sum = 0.f;
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sum += p;
                P[(ty * 4 + i) * kSimtP + tx + 16 * j] = p;
            }
            for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * fix + sum;
            m[i] = mx;
            for (int c = 0; c < DP / 16; ++c) o[i][c] *= fix;
        }
        __syncwarp();   // a row's 16 threads, which write and read its probabilities, are half a warp
        simt_mix<DP, false>(P, V, ty, tx, o);
    }
    for (int i = 0; i < 4; ++i) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        for (int c = 0; c < DP / 16; ++c) o[i][c] *= inv;
        const int r = ty * 4 + i;
        if (tx == 0 && r < rows)
            a.lse[static_cast<int64_t>(h) * a.sq.T + t.s0 + t.t0 + r] =
                l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * (1.f / kAttnLog2e);
    }
    simt_store<DP>(static_cast<float *>(a.o) + (t.s0 + t.t0) * a.o_ts + h * a.o_hs, a.o_ts, rows, a.D, ty, tx, 1.f, o);
}

// p and ds of one 64 x 64 tile from Q, K, dO, V in shared memory: rows are
// queries, stored [query][key].
template <int DP>
__device__ __forceinline__ void simt_probs(const AttnArgs &a, const float *Q, const float *K, const float *G,
                                           const float *V, const float *stat, int q0, int k0, int keys, int off,
                                           int ty, int tx, float *P, float *dS) {
    float s[4][4], d[4][4];
    simt_dot<DP>(Q, K, ty, tx, s);
    simt_dot<DP>(G, V, ty, tx, d);
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        const int lim = a.causal ? min(keys, q0 + r + off + 1 - k0) : keys;
        const float lse2 = stat[r], delta = stat[kSimtTile + r];
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const float p = c < lim ? exp2f(fmaf(s[i][j], a.scale_log2, -lse2)) : 0.f;
            if (P) P[r * kSimtP + c] = p;
            dS[r * kSimtP + c] = c < lim ? p * (d[i][j] - delta) : 0.f;
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(kSimtThreads) k_attn_dq_simt(const AttnArgs a) {
    extern __shared__ float sm[];
    constexpr int kOp = kSimtTile * (DP + 1);
    float *Q = sm, *G = Q + kOp, *K = G + kOp, *V = K + kOp, *dS = V + kOp, *stat = dS + kSimtTile * kSimtP;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int h = blockIdx.x % a.Hq, hk = h / a.group, slot = blockIdx.x / a.Hq;
    const TileInfo t = tile_info<kSimtTile>(a.sq, a.sk, slot);
    const int rows = min(kSimtTile, t.len - t.t0);
    if (t.t0 < 0 || rows <= 0) return;
    const int off = t.olen - t.len;
    const int kend = a.causal ? min(t.olen, t.t0 + rows + off) : t.olen;
    const int64_t tok = t.s0 + t.t0;
    simt_load<DP>(Q, static_cast<const float *>(a.q) + tok * a.q_ts + h * a.q_hs, a.q_ts, rows, a.D);
    simt_load<DP>(G, static_cast<const float *>(a.dO) + tok * a.dO_ts + h * a.dO_hs, a.dO_ts, rows, a.D);
    if (tid < kSimtTile) {
        const int64_t at = h * a.stat_stride + static_cast<int64_t>(slot) * kSimtTile + tid;
        stat[tid] = a.lse2[at];
        stat[kSimtTile + tid] = a.delta[at];
    }
    float acc[4][DP / 16] = {};
    for (int k0 = 0; k0 < kend; k0 += kSimtTile) {
        const int keys = min(kSimtTile, t.olen - k0);
        __syncthreads();
        simt_load<DP>(K, static_cast<const float *>(a.k) + (t.o0 + k0) * a.k_ts + hk * a.k_hs, a.k_ts, keys, a.D);
        simt_load<DP>(V, static_cast<const float *>(a.v) + (t.o0 + k0) * a.v_ts + hk * a.v_hs, a.v_ts, keys, a.D);
        __syncthreads();
        simt_probs<DP>(a, Q, K, G, V, stat, t.t0, k0, keys, off, ty, tx, nullptr, dS);
        __syncwarp();
        simt_mix<DP, false>(dS, K, ty, tx, acc);
    }
    simt_store<DP>(static_cast<float *>(a.dq) + tok * a.dq_ts + h * a.dq_hs, a.dq_ts, rows, a.D, ty, tx, a.scale, acc);
}

template <int DP>
__global__ void __launch_bounds__(kSimtThreads) k_attn_dkv_simt(const AttnArgs a) {
    extern __shared__ float sm[];
    constexpr int kOp = kSimtTile * (DP + 1), kTl = kSimtTile * kSimtP;
    float *Q = sm, *G = Q + kOp, *K = G + kOp, *V = K + kOp, *P = V + kOp, *dS = P + kTl, *stat = dS + kTl;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int hk = blockIdx.x % a.Hk, slot = blockIdx.x / a.Hk;
    const TileInfo t = tile_info<kSimtTile>(a.sk, a.sq, slot);   // own side: keys
    const int keys = min(kSimtTile, t.len - t.t0);
    if (t.t0 < 0 || keys <= 0) return;
    const int off = t.len - t.olen;
    const int64_t tok = t.s0 + t.t0;
    simt_load<DP>(K, static_cast<const float *>(a.k) + tok * a.k_ts + hk * a.k_hs, a.k_ts, keys, a.D);
    simt_load<DP>(V, static_cast<const float *>(a.v) + tok * a.v_ts + hk * a.v_hs, a.v_ts, keys, a.D);
    // the first query row that sees this tile's first key
    const int qfirst = a.causal ? max(0, t.t0 - off) / kSimtTile * kSimtTile : 0;
    float dk[4][DP / 16] = {}, dv[4][DP / 16] = {};
    const int qslot0 = t.olen > 0 ? slot_base<kSimtTile>(a.sq, t.b) : 0;
    for (int h = hk * a.group; h < (hk + 1) * a.group; ++h) {
        for (int q0 = qfirst; q0 < t.olen; q0 += kSimtTile) {
            const int rows = min(kSimtTile, t.olen - q0);
            const int64_t qt = t.o0 + q0;
            __syncthreads();
            simt_load<DP>(Q, static_cast<const float *>(a.q) + qt * a.q_ts + h * a.q_hs, a.q_ts, rows, a.D);
            simt_load<DP>(G, static_cast<const float *>(a.dO) + qt * a.dO_ts + h * a.dO_hs, a.dO_ts, rows, a.D);
            if (tid < kSimtTile) {
                const int64_t at = h * a.stat_stride + static_cast<int64_t>(qslot0 + q0 / kSimtTile) * kSimtTile + tid;
                stat[tid] = a.lse2[at];
                stat[kSimtTile + tid] = a.delta[at];
            }
            __syncthreads();
            simt_probs<DP>(a, Q, K, G, V, stat, q0, t.t0, keys, off, ty, tx, P, dS);
            __syncthreads();
            simt_mix<DP, true>(P, G, ty, tx, dv);
            simt_mix<DP, true>(dS, Q, ty, tx, dk);
        }
    }
    simt_store<DP>(static_cast<float *>(a.dk) + tok * a.dk_ts + hk * a.dk_hs, a.dk_ts, keys, a.D, ty, tx, a.scale, dk);
    simt_store<DP>(static_cast<float *>(a.dv) + tok * a.dv_ts + hk * a.dv_hs, a.dv_ts, keys, a.D, ty, tx, 1.f, dv);
}

}  // namespace lce
