// Attention of fp32 tensors, in fp32 arithmetic: tiles of 64 queries by 64 keys
// in shared memory, 256 threads in a 16 x 16 grid, each with four query rows
// (or key rows) and every 16th row of the other side, or DP/16 channels. Rows
// are four floats longer than their data, so that both the reads along a row
// (16 bytes at a time, 16 rows apart by lane) and those across it are free of
// bank conflicts; 16-byte reads bring eight loads for 64 multiply-adds. What
// bounds it is the multiply-adds with those loads, and at a few hundred tokens
// the walk of the longest row (512 tokens, 4 heads of 64 channels, causal:
// forward 42 us, backward 76). Training runs in bf16; this is for the small
// fp32 configurations and for checking.
#pragma once

#include "lce_attn.cuh"

namespace lce {

constexpr int kSimtTile = 64;
constexpr int kSimtThreads = 256;
constexpr int kSimtP = kSimtTile + 4;   // row pitch of a 64 x 64 tile

constexpr int simt_smem(int DP, int operands, int tiles) {
    return (operands * kSimtTile * (DP + 4) + tiles * kSimtTile * kSimtP + 2 * kSimtTile) * 4;
}

// rows [0, 64) x [0, DP) from `rows` token rows of D floats; zero outside
template <int DP>
__device__ __forceinline__ void simt_load(float *dst, const float *src, int64_t stride, int rows, int D) {
#pragma unroll 4
    for (int i = threadIdx.x; i < kSimtTile * DP / 4; i += kSimtThreads) {
        const int r = i / (DP / 4), c = i % (DP / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && c < D) v = *reinterpret_cast<const float4 *>(src + r * stride + c);
        *reinterpret_cast<float4 *>(dst + r * (DP + 4) + c) = v;
    }
}

// acc[i][j] = A[ty*4+i] . B[tx+16j] over DP
template <int DP>
__device__ __forceinline__ void simt_dot(const float *A, const float *B, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < DP; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (ty * 4 + i) * (DP + 4) + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * (DP + 4) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
    }
}

// A thread's channels: DP/16 of them, in runs of at most four; run k starts at simt_col(tx, k).
template <int DP>
struct SimtCols {
    static constexpr int kN = DP / 16, kRun = kN < 4 ? kN : 4, kRuns = kN / kRun;
    static __device__ __forceinline__ int at(int tx, int run) { return run * 16 * kRun + tx * kRun; }
};

// acc[i][c] += sum_j P[ty*4+i][j] * B[j][column c]   (kT: P is read as P[j][ty*4+i])
template <int DP, bool kT>
__device__ __forceinline__ void simt_mix(const float *P, const float *B, int ty, int tx, float (&acc)[4][DP / 16]) {
    using C = SimtCols<DP>;
#pragma unroll 2
    for (int j = 0; j < kSimtTile; j += 4) {
        float x[4][4];   // [row][j]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(kT ? P + (j + i) * kSimtP + ty * 4 : P + (ty * 4 + i) * kSimtP + j);
            if (kT) x[0][i] = v.x, x[1][i] = v.y, x[2][i] = v.z, x[3][i] = v.w;
            else x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < C::kRuns; ++r) {
                float y[C::kRun];
                const float *b = B + (j + k) * (DP + 4) + C::at(tx, r);
                if (C::kRun == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(b);
                    y[0] = v.x, y[1] = v.y, y[C::kRun / 2] = v.z, y[C::kRun - 1] = v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(b);
                    y[0] = v.x, y[1] = v.y;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < C::kRun; ++c) acc[i][r * C::kRun + c] = fmaf(x[i][k], y[c], acc[i][r * C::kRun + c]);
            }
    }
}

template <int DP>
__device__ __forceinline__ void simt_store(float *dst, int64_t stride, int rows, int D, int ty, int tx, float mul,
                                           const float (&acc)[4][DP / 16]) {
    using C = SimtCols<DP>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= rows) continue;
#pragma unroll
        for (int c = 0; c < C::kN; ++c) {
            const int col = C::at(tx, c / C::kRun) + c % C::kRun;
            if (col < D) dst[r * stride + col] = acc[i][c] * mul;
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(kSimtThreads) k_attn_fwd_simt(const AttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + kSimtTile * (DP + 4), *V = K + kSimtTile * (DP + 4), *P = V + kSimtTile * (DP + 4);
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
        const float nlse2 = stat[r], ndelta = stat[kSimtTile + r];
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            const float p = c < lim ? exp2f(fmaf(s[i][j], a.scale_log2, nlse2)) : 0.f;
            if (P) P[r * kSimtP + c] = p;
            dS[r * kSimtP + c] = c < lim ? p * (d[i][j] + ndelta) : 0.f;
        }
    }
}

template <int DP>
__device__ __forceinline__ void dq_block_simt(const AttnArgs &a, float *sm, int block, int blocks) {
    constexpr int kOp = kSimtTile * (DP + 4);
    float *Q = sm, *G = Q + kOp, *K = G + kOp, *V = K + kOp, *dS = V + kOp, *stat = dS + kSimtTile * kSimtP;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int h = block % a.Hq, hk = h / a.group, slot = blocks / a.Hq - 1 - block / a.Hq;
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
        stat[tid] = a.nlse2[at];
        stat[kSimtTile + tid] = a.ndelta[at];
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
__device__ __forceinline__ void dkv_block_simt(const AttnArgs &a, float *sm, int block) {
    constexpr int kOp = kSimtTile * (DP + 4), kTl = kSimtTile * kSimtP;
    float *Q = sm, *G = Q + kOp, *K = G + kOp, *V = K + kOp, *P = V + kOp, *dS = P + kTl, *stat = dS + kTl;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int hk = block % a.Hk, slot = block / a.Hk;
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
                stat[tid] = a.nlse2[at];
                stat[kSimtTile + tid] = a.ndelta[at];
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

// Both kinds of blocks in one launch, the longer dK/dV blocks first.
template <int DP>
__global__ void __launch_bounds__(kSimtThreads) k_attn_bwd_simt(const AttnArgs a, int dkv_blocks) {
    extern __shared__ __align__(16) float sm[];
    const int block = blockIdx.x;
    if (block < dkv_blocks) dkv_block_simt<DP>(a, sm, block);
    else dq_block_simt<DP>(a, sm, block - dkv_blocks, gridDim.x - dkv_blocks);
}

}  // namespace lce
