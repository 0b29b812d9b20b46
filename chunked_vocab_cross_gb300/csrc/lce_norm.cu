// Norms before and after a block, fused with its gate and residual scale:
// kernels and host side of lce_block_norm_forward / _backward.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "lce_host.h"
#include "row_ring.cuh"

using namespace lce;

namespace {

struct NormArgs {
    const void *x, *b, *w_post, *gate, *w_pre, *r_in, *dr, *dn;
    void *r, *n, *dx, *db, *dgate;
    float *rstd_post, *rstd_pre;
    int64_t ld_x, ld_b, ld_gate, ld_r, ld_dr, ld_dn;
    int64_t N;
    int d, gate_full;
    float scale, eps;
    int *status;
    float *part;   // backward: partial column sums [3][groups][d] (w_pre, w_post, gate)
};

// Few rows: one block a row, a thread holds CH packs of its row's elements.
// What bounds it is latency: a launch, the loads, two sums over the block
// (one row of 4096 bf16: 2.7 us, 305 rows 4.4 us).
template <typename T, int CH>
__global__ void __launch_bounds__(512) k_norm_fwd(const NormArgs a) {
    __shared__ float red[64];
    int flip = 0;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    float r[CH][kVec];
    const int d = a.d;
    float s[1] = {0.f};
    if (a.b) {
        const T *b = static_cast<const T *>(a.b) + row * a.ld_b;
        float y[CH][kVec];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col < d) load_pack(b + col).get(y[c]);
            else
#pragma unroll
                for (int i = 0; i < kVec; ++i) y[c][i] = 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[0] = fmaf(y[c][i], y[c][i], s[0]);
        }
        float rs = 1.f;
        if (a.w_post) {
            block_sum(s, red, flip);
            rs = rsqrtf(s[0] / d + a.eps);
            if (threadIdx.x == 0) a.rstd_post[row] = rs;
        }
        const T *wp = static_cast<const T *>(a.w_post);
        const T *g = static_cast<const T *>(a.gate) + (a.gate_full ? row * a.ld_gate : 0);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col < d) {
                float t[kVec];
                if (a.w_post) {
                    load_pack(wp + col).get(t);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[c][i] *= rs * t[i];
                }
                if (a.gate) {
                    load_pack(g + col).get(t);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[c][i] *= t[i];
                }
                load_pack(x + col).get(t);
#pragma unroll
                for (int i = 0; i < kVec; ++i) r[c][i] = fmaf(a.scale, y[c][i], t[i]);
                store_pack(static_cast<T *>(a.r) + row * d + col, r[c]);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col < d) load_pack(x + col).get(r[c]);
        }
    }
    if (!a.w_pre) return;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if ((c * blockDim.x + threadIdx.x) * kVec < d)
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[0] = fmaf(r[c][i], r[c][i], s[0]);
    block_sum(s, red, flip);
    const float rs = rsqrtf(s[0] / d + a.eps);
    if (threadIdx.x == 0) a.rstd_pre[row] = rs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * blockDim.x + threadIdx.x) * kVec;
        if (col < d) {
            float t[kVec];
            load_pack(static_cast<const T *>(a.w_pre) + col).get(t);
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] *= r[c][i] * rs;
            store_pack(static_cast<T *>(a.n) + row * d + col, t);
        }
    }
}

// Rows too wide for the ring kernels below: persistent blocks, one row at a
// time. What bounds it is latency, with nothing loaded ahead (8192 rows of 8192
// bf16 took it 474 us, the ring 141). The two row sums of the formulas are taken
// in one round: with u = w_pre dn, m1 = mean(u rhat) and
// z = scale gate w_post bhat, the second is
//   sum(w_post dy bhat) = sum z (dr + rstd_pre u) - rstd_pre m1 sum z rhat.
// Column sums (weights, a gate per channel) stay in shared memory, each
// column owned by one thread, until the block's rows are done.
template <typename T, int CH>
__global__ void __launch_bounds__(512) k_norm_bwd(const NormArgs a) {
    extern __shared__ float sums[];   // [3][d]
    __shared__ float red[2 * 32 * 3];
    int flip = 0;
    const int d = a.d;
    const float inv_d = 1.f / d;
    for (int i = threadIdx.x; i < 3 * d; i += blockDim.x) sums[i] = 0.f;
    __syncthreads();
    const bool col_gate = a.gate && !a.gate_full;
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const float rp = a.w_pre ? a.rstd_pre[row] : 0.f, ro = a.w_post ? a.rstd_post[row] : 1.f;
        float hat[CH][kVec], u[CH][kVec], g[CH][kVec], bh[CH][kVec];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
#pragma unroll
            for (int i = 0; i < kVec; ++i) hat[c][i] = u[c][i] = g[c][i] = bh[c][i] = 0.f;
            if (col >= d) continue;
            float t[kVec], z[kVec];
            if (a.dr) load_pack(static_cast<const T *>(a.dr) + row * a.ld_dr + col).get(g[c]);
            if (a.w_pre) {
                load_pack(static_cast<const T *>(a.r_in) + row * a.ld_r + col).get(hat[c]);
                load_pack(static_cast<const T *>(a.dn) + row * a.ld_dn + col).get(u[c]);
                load_pack(static_cast<const T *>(a.w_pre) + col).get(t);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    hat[c][i] *= rp;
                    sums[col + i] += u[c][i] * hat[c][i];
                    u[c][i] *= t[i];
                    s[0] = fmaf(u[c][i], hat[c][i], s[0]);
                }
            }
            if (a.b) {
                load_pack(static_cast<const T *>(a.b) + row * a.ld_b + col).get(bh[c]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    bh[c][i] *= ro;
                    z[i] = a.scale * bh[c][i];
                }
                if (a.w_post) {
                    load_pack(static_cast<const T *>(a.w_post) + col).get(t);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) z[i] *= t[i];
                }
                if (a.gate) {
                    load_pack(static_cast<const T *>(a.gate) + (a.gate_full ? row * a.ld_gate : 0) + col).get(t);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) z[i] *= t[i];
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    s[1] = fmaf(z[i], fmaf(rp, u[c][i], g[c][i]), s[1]);
                    s[2] = fmaf(z[i], hat[c][i], s[2]);
                }
            }
        }
        block_sum(s, red, flip);
        const float m1 = s[0] * inv_d;
        const float m2 = (s[1] - rp * m1 * s[2]) * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col >= d) continue;
            float w[kVec], t[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) g[c][i] = fmaf(rp, u[c][i] - hat[c][i] * m1, g[c][i]);
            store_pack(static_cast<T *>(a.dx) + row * d + col, g[c]);
            if (!a.b) continue;
#pragma unroll
            for (int i = 0; i < kVec; ++i) g[c][i] *= a.scale, w[i] = 1.f;
            if (a.w_post) load_pack(static_cast<const T *>(a.w_post) + col).get(w);
            if (a.gate) {
                float dg[kVec];
                load_pack(static_cast<const T *>(a.gate) + (a.gate_full ? row * a.ld_gate : 0) + col).get(t);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    dg[i] = g[c][i] * bh[c][i] * w[i];
                    g[c][i] *= t[i];
                }
                if (a.gate_full) store_pack(static_cast<T *>(a.dgate) + row * d + col, dg);
                else
#pragma unroll
                    for (int i = 0; i < kVec; ++i) sums[2 * d + col + i] += dg[i];
            }
            if (a.w_post) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    sums[d + col + i] += g[c][i] * bh[c][i];
                    g[c][i] = ro * (g[c][i] * w[i] - bh[c][i] * m2);
                }
            }
            store_pack(static_cast<T *>(a.db) + row * d + col, g[c]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 3 * d; i += blockDim.x) {
        const int k = i / d;
        if (k == 0 ? a.w_pre != nullptr : k == 1 ? a.w_post != nullptr : col_gate)
            a.part[(static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * d + i % d] = sums[i];
    }
}

// ---------------------------------------------------------------- ring kernels
//
// Persistent blocks whose rows arrive through a ring of shared-memory stages,
// filled by untiled bulk copies that one thread issues: the copies of the next
// rows are in flight while a row's sums are joined, so HBM is kept busy with
// few threads and no registers for prefetching. A stage holds `groups`
// consecutive rows, each taken by `tpr` threads with CH packs of 16 bytes;
// the groups join their sums on barriers of their own and so cover each
// other's waits. Weights (ones where there are none) stay in shared memory.
// What bounds them is HBM, once the work between two rows hides behind it. That
// work is mostly issue slots: hence the packed fp32 arithmetic, 16 to 32
// elements a thread against the fixed cost of a sum, and no branches on the
// options inside a row. The forward's inputs and r ask to leave L2 first (16384
// rows of 4096 bf16, calls in a row on inputs from HBM: 90 us, 95 without; the
// backward gains nothing from that); n does not, since the block's first product
// reads it next (8192 rows of 2048, norm, product, norm: 80.5 us, 84.8 with n
// marked too, 83.5 with nothing marked). At 16384 x 4096, with norms on both
// sides and a gate per channel: forward 90 us (6.0 TB/s; 94.5 among other calls),
// 125 with a block for each row; backward 139 us with the 4 us of k_norm_cols
// (5.8 TB/s).
enum NormMode : int { NORM_ANY, NORM_ALL, NORM_FULL_GATE, NORM_NO_DR, NORM_PRE, NORM_POST };


// NORM_ALL: b, w_post and w_pre are there and the gate, if any, is per channel;
// NORM_FULL_GATE: with a gate per element. Those options are known when the
// kernel is compiled (4096 rows of 4096 bf16:
// 21.1 us against 22.8; no difference where HBM alone bounds it).
template <typename T, int CH, int kMode>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_fwd_ring(const NormArgs a, const RingGeo g) {
    constexpr int V = kPack<T>, P = V / 2;
    extern __shared__ __align__(128) uint8_t smem[];   // ring, then w_post, gate, w_pre
    __shared__ RingBars bars;
    __shared__ __align__(16) float red[16 * kRedFloats];
    const int nwarps = blockDim.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], nwarps);
        for (int i = 0; i < 16; ++i) bars.gave_up[i] = 0;
        fence_mbar_init();
    }
    const int d = a.d;
    const bool has_b = kMode || a.b, has_post = kMode || a.w_post, has_pre = kMode || a.w_pre,
               full_gate = kMode == NORM_FULL_GATE || (kMode == NORM_ANY && a.gate && a.gate_full);
    uint8_t *w_post = smem + g.stages * g.stage_bytes, *gate = w_post + g.row_bytes, *w_pre = gate + g.row_bytes;
    load_weights<T>(w_post, a.w_post, g.row_bytes);
    load_weights<T>(gate, full_gate ? nullptr : a.gate, g.row_bytes);
    load_weights<T>(w_pre, a.w_pre, g.row_bytes);
    for (int i = threadIdx.x; i < 16 * kRedFloats; i += blockDim.x) red[i] = 0.f;
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.groups;
    int64_t r0 = static_cast<int64_t>(blockIdx.x) * g.groups;
    const RingSource<T, 3, true> src = {{static_cast<const T *>(a.x), static_cast<const T *>(a.b), full_gate ? static_cast<const T *>(a.gate) : nullptr},
                                  {a.ld_x, a.ld_b, a.ld_gate}};
    if (threadIdx.x == 0)
        for (int i = 0; i < g.stages; ++i) src.issue(smem, bars, g, g.groups, i, r0 + i * step, a.N, d);
    const int group = threadIdx.x / g.tpr, t = threadIdx.x % g.tpr;
    float *my_red = red + group * kRedFloats;
    const float inv_d = 1.f / d;
    uint8_t *out_r = static_cast<uint8_t *>(a.r) + (r0 + group) * g.row_bytes + t * 16;
    uint8_t *out_n = static_cast<uint8_t *>(a.n) + (r0 + group) * g.row_bytes + t * 16;
    int flip = 0, s = 0;
    uint32_t phase = 0;
    for (; r0 < a.N; r0 += step, out_r += step * g.row_bytes, out_n += step * g.row_bytes) {
        const int64_t row = r0 + group;
        // the vote also tells the compiler that the warp is together again
        if (!__all_sync(0xffffffffu, ring_wait(&bars.full[s], phase, a.status))) bars.gave_up[group] = 1;
        const bool live = row < a.N;
        const uint8_t *at = smem + s * g.stage_bytes + group * g.row_bytes;
        f32x2 r[CH][P];
        uint4 vb[CH], vg[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            uint4 x = make_uint4(0, 0, 0, 0);
            vb[c] = vg[c] = x;
            if (byte < g.row_bytes) {
                x = *reinterpret_cast<const uint4 *>(at + byte);
                if (has_b) vb[c] = *reinterpret_cast<const uint4 *>(at + g.array_bytes + byte);
                if (full_gate) vg[c] = *reinterpret_cast<const uint4 *>(at + 2 * g.array_bytes + byte);
            }
            Pack16<T>::get(x, r[c]);
        }
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(&bars.empty[s]);   // everything is in registers
        {
            float rs = 1.f;
            if (has_post) {
                f32x2 q = both(0.f);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    f32x2 b[P];
                    Pack16<T>::get(vb[c], b);
#pragma unroll
                    for (int i = 0; i < P; ++i) q = fma2(b[i], b[i], q);
                }
                float sum[1] = {hsum2(q)};
                group_sum(sum, my_red, flip, g.tpr, group, t);
                rs = rsqrtf(sum[0] * inv_d + a.eps);
                if (t == 0 && live) a.rstd_post[row] = rs;
            }
            if (has_b) {
                const f32x2 f = both(rs * a.scale);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int byte = (c * g.tpr + t) * 16;
                    if (byte >= g.row_bytes) continue;
                    f32x2 y[P], w[P];
                    Pack16<T>::get(vb[c], y);
                    Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_post + byte), w);
#pragma unroll
                    for (int i = 0; i < P; ++i) y[i] = mul2(y[i], w[i]);
                    Pack16<T>::get(full_gate ? vg[c] : *reinterpret_cast<const uint4 *>(gate + byte), w);
#pragma unroll
                    for (int i = 0; i < P; ++i) r[c][i] = fma2(mul2(y[i], w[i]), f, r[c][i]);
                    if (live) __stcs(reinterpret_cast<uint4 *>(out_r + c * g.tpr * 16), Pack16<T>::set(r[c]));
                }
            }
        }
        float sum[1] = {0.f};
        if (has_pre) {
            f32x2 q = both(0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < P; ++i) q = fma2(r[c][i], r[c][i], q);   // zeros past d
            sum[0] = hsum2(q);
            group_sum(sum, my_red, flip, g.tpr, group, t);
        }
        if (bars.gave_up[group]) {
            if (threadIdx.x == 0) ring_drain(bars, g, g.groups, s, phase, r0, a.N);
            break;
        }
        // the stage's next rows, once every warp has taken its share
        if (threadIdx.x == 0 && r0 + g.stages * step < a.N && ring_wait(&bars.empty[s], phase, a.status))
            src.issue(smem, bars, g, g.groups, s, r0 + g.stages * step, a.N, d);
        if (has_pre) {
            const float rs = rsqrtf(sum[0] * inv_d + a.eps);
            if (t == 0 && live) a.rstd_pre[row] = rs;
            const f32x2 f = both(rs);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int byte = (c * g.tpr + t) * 16;
                if (byte >= g.row_bytes) continue;
                f32x2 w[P];
                Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_pre + byte), w);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = mul2(mul2(r[c][i], f), w[i]);
                if (live) *reinterpret_cast<uint4 *>(out_n + c * g.tpr * 16) = Pack16<T>::set(w);
            }
        }
        if (++s == g.stages) s = 0, phase ^= 1;
    }
}

// The two row sums in one round as in k_norm_bwd, with factors that are the
// same for a whole row taken out: hat = rstd_pre r, t = dr + rstd_pre u,
// z = b w_post gate, f = scale rstd_post:
//   m1 = mean(u hat),  m2 = f (sum z t - rstd_pre m1 sum z hat) / d,
//   dx = t - rstd_pre m1 hat,  e = f dx:  dgate = e b w_post,
//   dw_post = e gate b,  db = e gate w_post - rstd_post^2 m2 b   (no w_post: the last term is 0).
// A thread takes its columns of R = 2 rows at a time where it has the registers,
// which halves what it spends on weights (16384 rows of 4096 bf16: 140 us, 192
// with one). The column sums stay in registers, one set a row group, and are
// joined across the groups in shared memory at the end.
// What is there is known when the kernel is compiled, since the registers go
// to what might be: NORM_ALL: dr, dn, b and w_pre, and a gate per channel if
// any; NORM_NO_DR: the same without dr; NORM_FULL_GATE: a gate per element;
// NORM_PRE: no b; NORM_POST: no w_pre (8192 rows of 8192 bf16: 140, 131,
// 171, 100 and 125 us; with options read in the kernel 233 for the first, 320,
// 379, 270 and 295).
template <typename T, int CH, int R, int kMode>
__global__ void __launch_bounds__(kRingThreads, 1) k_norm_bwd_ring(const NormArgs a, const RingGeo g) {
    constexpr int V = kPack<T>, P = V / 2;
    extern __shared__ __align__(128) uint8_t smem[];   // ring, then w_post, gate, w_pre
    __shared__ RingBars bars;
    __shared__ __align__(16) float red[16 * kRedFloats];
    const int nwarps = blockDim.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], nwarps);
        for (int i = 0; i < 16; ++i) bars.gave_up[i] = 0;
        fence_mbar_init();
    }
    const int d = a.d;
    const bool has_pre = kMode != NORM_POST, has_b = kMode != NORM_PRE, has_dr = kMode == NORM_ALL || (kMode != NORM_NO_DR && a.dr),
               full_gate = kMode == NORM_FULL_GATE || (kMode == NORM_POST && a.gate && a.gate_full);
    uint8_t *w_post = smem + g.stages * g.stage_bytes, *gate = w_post + g.row_bytes, *w_pre = gate + g.row_bytes;
    load_weights<T>(w_post, a.w_post, g.row_bytes);
    load_weights<T>(gate, full_gate ? nullptr : a.gate, g.row_bytes);
    load_weights<T>(w_pre, a.w_pre, g.row_bytes);
    for (int i = threadIdx.x; i < 16 * kRedFloats; i += blockDim.x) red[i] = 0.f;
    __syncthreads();
    const int per = g.groups * R;   // rows of a stage
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    int64_t r0 = static_cast<int64_t>(blockIdx.x) * per;
    const RingSource<T, 5, false> src = {{a.w_pre ? static_cast<const T *>(a.r_in) : nullptr, a.w_pre ? static_cast<const T *>(a.dn) : nullptr,
                                   static_cast<const T *>(a.b), full_gate ? static_cast<const T *>(a.gate) : nullptr, static_cast<const T *>(a.dr)},
                                  {a.ld_r, a.ld_dn, a.ld_b, a.ld_gate, a.ld_dr}};
    // places of the arrays in a stage
    const uint32_t at_n = g.array_bytes, at_b = has_pre ? 2 * g.array_bytes : 0, at_g = at_b + (has_b ? g.array_bytes : 0),
                   at_d = at_g + (full_gate ? g.array_bytes : 0);
    if (threadIdx.x == 0)
        for (int i = 0; i < g.stages; ++i) src.issue(smem, bars, g, per, i, r0 + i * step, a.N, d);
    const int group = threadIdx.x / g.tpr, t = threadIdx.x % g.tpr;
    float *my_red = red + group * kRedFloats;
    const float inv_d = 1.f / d;
    f32x2 s_pre[CH][P], s_post[CH][P], s_gate[CH][P];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < P; ++i) s_pre[c][i] = s_post[c][i] = s_gate[c][i] = both(0.f);
    uint8_t *out_x = static_cast<uint8_t *>(a.dx) + (r0 + group * R) * g.row_bytes + t * 16;
    uint8_t *out_b = static_cast<uint8_t *>(a.db) + (r0 + group * R) * g.row_bytes + t * 16;
    int flip = 0, s = 0;
    uint32_t phase = 0;
    float rp_next[R], ro_next[R];   // 1/rms of the rows to come, asked for a round ahead; zeros past the last row
    auto rstd = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool live = row + k < a.N;
            rp_next[k] = has_pre && live ? a.rstd_pre[row + k] : 0.f;
            ro_next[k] = !live ? 0.f : a.w_post ? a.rstd_post[row + k] : 1.f;
        }
    };
    rstd(r0 + group * R);
    for (; r0 < a.N; r0 += step, out_x += step * g.row_bytes, out_b += step * g.row_bytes) {
        const int64_t row = r0 + group * R;
        float rp[R], ro[R];
#pragma unroll
        for (int k = 0; k < R; ++k) rp[k] = rp_next[k], ro[k] = ro_next[k];
        rstd(row + step);
        // the vote also tells the compiler that the warp is together again
        if (!__all_sync(0xffffffffu, ring_wait(&bars.full[s], phase, a.status))) bars.gave_up[group] = 1;
        uint8_t *at = smem + s * g.stage_bytes + group * R * g.row_bytes;
        if (row + R > a.N) {   // rows past the last add nothing to the columns: zeros, as 0 * inf would
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const int byte = (c * g.tpr + t) * 16;
                    if (row + k < a.N || byte >= g.row_bytes) continue;
                    for (uint8_t *p = at + k * g.row_bytes + byte, *end = smem + (s + 1) * g.stage_bytes; p < end; p += g.array_bytes)
                        *reinterpret_cast<uint4 *>(p) = make_uint4(0, 0, 0, 0);
                }
        }
        f32x2 hat[R][CH][P], x[R][CH][P];
        uint4 vb[R][CH];
        f32x2 q[R][3];
#pragma unroll
        for (int k = 0; k < R; ++k) q[k][0] = q[k][1] = q[k][2] = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            if (byte >= g.row_bytes) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    vb[k][c] = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < P; ++i) hat[k][c][i] = x[k][c][i] = both(0.f);
                }
                continue;
            }
            f32x2 w[P], wz[P], u[P];
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_post + byte), wz);
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(gate + byte), w);
#pragma unroll
            for (int i = 0; i < P; ++i) wz[i] = mul2(wz[i], w[i]);
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_pre + byte), w);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const uint8_t *p = at + k * g.row_bytes + byte;
                uint4 v = make_uint4(0, 0, 0, 0), vn = v, vd = v;
                vb[k][c] = v;
                if (has_pre) {
                    v = *reinterpret_cast<const uint4 *>(p);
                    vn = *reinterpret_cast<const uint4 *>(p + at_n);
                }
                if (has_b) vb[k][c] = *reinterpret_cast<const uint4 *>(p + at_b);
                if (has_dr) vd = *reinterpret_cast<const uint4 *>(p + at_d);
                Pack16<T>::get(v, hat[k][c]);
                Pack16<T>::get(vn, u);
                Pack16<T>::get(vd, x[k][c]);
                const f32x2 rp2 = both(rp[k]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    hat[k][c][i] = mul2(hat[k][c][i], rp2);
                    s_pre[c][i] = fma2(u[i], hat[k][c][i], s_pre[c][i]);
                    u[i] = mul2(u[i], w[i]);
                    q[k][0] = fma2(u[i], hat[k][c][i], q[k][0]);
                    x[k][c][i] = fma2(rp2, u[i], x[k][c][i]);
                }
                Pack16<T>::get(vb[k][c], u);
                if (full_gate) {
                    f32x2 gt[P];
                    Pack16<T>::get(*reinterpret_cast<const uint4 *>(p + at_g), gt);
#pragma unroll
                    for (int i = 0; i < P; ++i) u[i] = mul2(u[i], gt[i]);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    u[i] = mul2(u[i], wz[i]);
                    q[k][1] = fma2(u[i], x[k][c][i], q[k][1]);
                    q[k][2] = fma2(u[i], hat[k][c][i], q[k][2]);
                }
            }
        }
        float sum[3 * R];
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int i = 0; i < 3; ++i) sum[3 * k + i] = hsum2(q[k][i]);
        group_sum(sum, my_red, flip, g.tpr, group, t);
        if (bars.gave_up[group]) {
            if (threadIdx.x == 0) ring_drain(bars, g, per, s, phase, r0, a.N);
            break;
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            if (byte >= g.row_bytes) continue;
            f32x2 w[P], gw[P];
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_post + byte), w);
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(gate + byte), gw);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const bool live = row + k < a.N;
                const uint32_t o = k * g.row_bytes + c * g.tpr * 16;
                const float m1 = rp[k] * sum[3 * k] * inv_d, f = a.scale * ro[k];
                const f32x2 m1n = both(-m1), f2 = both(f);
                const f32x2 m2n = both(a.w_post ? -(ro[k] * ro[k] * f * (sum[3 * k + 1] - m1 * sum[3 * k + 2]) * inv_d) : 0.f);
                f32x2 (&y)[P] = x[k][c];
#pragma unroll
                for (int i = 0; i < P; ++i) y[i] = fma2(m1n, hat[k][c][i], y[i]);
                if (live) *reinterpret_cast<uint4 *>(out_x + o) = Pack16<T>::set(y);
                if (!has_b) continue;
                f32x2 b[P], dg[P];
                Pack16<T>::get(vb[k][c], b);
#pragma unroll
                for (int i = 0; i < P; ++i) y[i] = mul2(y[i], f2), dg[i] = mul2(b[i], w[i]);
                if (full_gate) {
                    f32x2 gt[P];
                    Pack16<T>::get(*reinterpret_cast<const uint4 *>(at + k * g.row_bytes + byte + at_g), gt);
#pragma unroll
                    for (int i = 0; i < P; ++i) dg[i] = mul2(y[i], dg[i]), y[i] = mul2(y[i], gt[i]);
                    if (live) *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.dgate) + (row + k) * g.row_bytes + byte) = Pack16<T>::set(dg);
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) s_gate[c][i] = fma2(y[i], dg[i], s_gate[c][i]), y[i] = mul2(y[i], gw[i]);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    s_post[c][i] = fma2(y[i], b[i], s_post[c][i]);
                    y[i] = fma2(m2n, b[i], mul2(y[i], w[i]));
                }
                if (live) *reinterpret_cast<uint4 *>(out_b + o) = Pack16<T>::set(y);
            }
        }
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(&bars.empty[s]);
        // the stage's next rows, once every warp is through with it
        if (threadIdx.x == 0 && r0 + g.stages * step < a.N && ring_wait(&bars.empty[s], phase, a.status))
            src.issue(smem, bars, g, per, s, r0 + g.stages * step, a.N, d);
        if (++s == g.stages) s = 0, phase ^= 1;
    }
    // the groups' sums, [group][d] at a time through the (now idle) ring
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (!(k == 0 ? a.w_pre != nullptr : k == 1 ? a.w_post != nullptr : a.gate && !a.gate_full)) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * g.tpr + t) * V;
            if (col >= d) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 v;
                unpack2(k == 0 ? s_pre[c][i] : k == 1 ? s_post[c][i] : s_gate[c][i], v.x, v.y);
                *reinterpret_cast<float2 *>(sums + group * d + col + 2 * i) = v;
            }
        }
        __syncthreads();
        float *out = a.part + (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * d;
        for (int i = threadIdx.x; i < d; i += blockDim.x) {
            float v = 0.f;
            for (int q = 0; q < g.groups; ++q) v += sums[q * d + i];
            out[i] = v;
        }
        __syncthreads();
    }
}

constexpr int64_t kMaxD = 16384;

lce_status_t check_rows(const void *p, int64_t ld, int elt) {
    if (ld < 0 || ld >= (int64_t(1) << 36)) return LCE_ERR_SHAPE;
    if (host_misaligned(p) || (ld * elt) % 16) return LCE_ERR_ALIGN;
    return LCE_OK;
}

lce_status_t check_norm(const lce_norm_t *a, bool backward) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->N < 0 || a->N >= (int64_t(1) << 31) || a->d < 8 || a->d > kMaxD) return LCE_ERR_SHAPE;
    if (a->d % 8) return LCE_ERR_ALIGN;
    if (a->scale - a->scale != 0.f || !(a->eps >= 0.f) || a->eps - a->eps != 0.f) return LCE_ERR_ARG;
    if (!a->b && (a->w_post || a->gate)) return LCE_ERR_ARG;   // nothing to norm or to gate
    if (!a->b && !a->w_pre) return LCE_ERR_ARG;                // nothing to do
    if (a->N == 0 && !backward) return LCE_OK;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    // `rows`: touched only when there are rows (the column sums are written without any)
    struct { const void *p; int64_t ld; bool want, rows; } in[] = {
        {a->x, a->ld_x, !backward, true}, {a->b, a->ld_b, false, true}, {a->w_post, 0, false, false},
        {a->w_pre, 0, false, false}, {a->gate, a->ld_gate, false, false},
        {a->r, a->ld_r, backward ? a->w_pre != nullptr : a->b != nullptr, true},
        {a->n, 0, !backward && a->w_pre, true}, {a->dn, a->ld_dn, backward && a->w_pre, true},
        {a->dr, a->ld_dr, false, true}, {a->dx, 0, backward, true}, {a->db, 0, backward && a->b, true},
        {a->dgate, 0, backward && a->gate, a->gate_full != 0}, {a->dw_post, 0, backward && a->w_post, false},
        {a->dw_pre, 0, backward && a->w_pre, false}};
    if (a->N > 0 && ((a->w_post && !a->rstd_post) || (a->w_pre && !a->rstd_pre))) return LCE_ERR_NULL;
    for (const auto &t : in) {
        if (t.rows && a->N == 0) continue;
        if (t.want && !t.p) return LCE_ERR_NULL;
        const lce_status_t s = check_rows(t.p, t.ld, elt);
        if (s != LCE_OK) return s;
    }
    return LCE_OK;
}

NormArgs make_norm(const lce_norm_t *a) {
    NormArgs r{};
    r.x = a->x, r.b = a->b, r.w_post = a->w_post, r.gate = a->gate, r.w_pre = a->w_pre, r.r_in = a->r;
    r.dr = a->dr, r.dn = a->dn, r.r = a->r, r.n = a->n, r.dx = a->dx, r.db = a->db, r.dgate = a->dgate;
    r.rstd_post = a->rstd_post, r.rstd_pre = a->rstd_pre;
    auto ld = [&](int64_t v) { return v ? v : a->d; };
    r.ld_x = ld(a->ld_x), r.ld_b = ld(a->ld_b), r.ld_gate = ld(a->ld_gate), r.ld_r = ld(a->ld_r);
    r.ld_dr = ld(a->ld_dr), r.ld_dn = ld(a->ld_dn);
    r.N = a->N, r.d = static_cast<int>(a->d), r.gate_full = a->gate_full != 0;
    r.scale = a->scale, r.eps = a->eps;
    return r;
}

// Threads of a row's block: one pack each up to 512 of them, then more packs.
int row_threads(int d) {
    const int packs = d / kVec;
    return packs >= 512 ? 512 : (packs + 31) / 32 * 32;
}
int row_packs(int d) { return (d / kVec + 511) / 512; }

constexpr int kRingBytes = 208 * 1024;   // dynamic shared memory of a ring kernel's block at most
// Ring of the forward, if two stages do not take more: 128 KB are enough in flight, and less in turns is easier on
// HBM (131072 rows of 512 bf16: 92 us, 95 with all of kRingBytes; 32768 rows of 2048: 89 us, 92).
constexpr int kFwdRingBytes = 128 * 1024;
// Few rows have nothing to run ahead of: up to this much of an array the forward takes a block for each row, with
// fewer steps before its first load (rows of 4096 bf16: 305 in 4.4 us, 5.6 through the ring; 608 in 7.6 us, 6.4;
// of 1024: 1216 in 4.5 us, 5.5; 4096 in 9.3 us, 8.6).
constexpr int64_t kDirectBytes = 4 << 20;
constexpr int kColGroups = 304;          // blocks of the backward at most (bounds its workspace)

// The ring kernels' geometry for rows of d elements in `arrays` arrays, `ch`
// packs a thread and `per` rows a group and stage; false where rows are too wide
// for the threads of a block or for two stages.
bool ring_geo(RingGeo *g, int d, int elt, int arrays, int ch, int per, int bytes) {
    const int packs = d * elt / 16;
    g->tpr = ((packs + ch - 1) / ch + 31) / 32 * 32;
    if (g->tpr > kRingThreads) return false;
    g->groups = kRingThreads / g->tpr;
    g->row_bytes = d * elt;
    g->array_bytes = g->groups * per * g->row_bytes;
    g->stage_bytes = arrays * g->array_bytes;
    if (2 * g->stage_bytes + 3 * g->row_bytes > kRingBytes) return false;
    g->stages = std::max(2, std::min(kRingMaxStages, static_cast<int>(std::min<int>(bytes, kRingBytes - 3 * g->row_bytes) / g->stage_bytes)));
    return true;
}

// Packs a thread in the forward: as few as leave a row to 32 threads, at most
// 32 elements (16384 rows of 4096 bf16: 90 us with four packs, 137 with one).
int ring_packs(int d, int elt, int most) {
    int ch = 1;
    while (ch < most && d * elt / 16 > 32 * ch) ch *= 2;
    return ch;
}

// Rows are handed out a stage at a time; at least one block, so that column
// sums of no rows come out as zeros.
int ring_grid(int64_t N, int groups, int most) {
    const int64_t n = (N + groups - 1) / groups;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, most)));
}

template <auto kKernel>
lce_status_t launch_ring(const HostDev &dev, const NormArgs &r, const RingGeo &g, int grid, int smem, cudaStream_t st) {
    const lce_status_t s = host_smem<kKernel>(dev, kRingBytes);
    if (s != LCE_OK) return s;
    kKernel<<<grid, g.tpr * g.groups, smem, st>>>(r, g);
    return host_launched();
}

template <typename T>
lce_status_t forward(const lce_norm_t *a, const HostDev &dev, cudaStream_t st) {
    NormArgs r = make_norm(a);
    r.status = dev.status;
    RingGeo g;
    const int ch = ring_packs(r.d, sizeof(T), 32 / kPack<T>);
    const int arrays = (r.b ? 2 : 1) + (r.gate && r.gate_full ? 1 : 0);
    if (a->N * r.d * static_cast<int64_t>(sizeof(T)) > kDirectBytes && ring_geo(&g, r.d, sizeof(T), arrays, ch, 1, kFwdRingBytes)) {
        const int grid = ring_grid(a->N, g.groups, dev.sms), smem = g.stages * g.stage_bytes + 3 * g.row_bytes;
        const int mode = !(r.b && r.w_post && r.w_pre) ? NORM_ANY : r.gate && r.gate_full ? NORM_FULL_GATE : NORM_ALL;
        auto go = [&](auto c) {
            constexpr int CH = decltype(c)::value;
            return mode == NORM_ALL         ? launch_ring<k_norm_fwd_ring<T, CH, NORM_ALL>>(dev, r, g, grid, smem, st)
                   : mode == NORM_FULL_GATE ? launch_ring<k_norm_fwd_ring<T, CH, NORM_FULL_GATE>>(dev, r, g, grid, smem, st)
                                            : launch_ring<k_norm_fwd_ring<T, CH, NORM_ANY>>(dev, r, g, grid, smem, st);
        };
        switch (ch) {
            case 1: return go(std::integral_constant<int, 1>());
            case 2: return go(std::integral_constant<int, 2>());
            case 4: return go(std::integral_constant<int, 4>());
            default: return go(std::integral_constant<int, 32 / kPack<T>>());   // fp32: 8
        }
    }
    const unsigned grid = static_cast<unsigned>(a->N);
    const int th = row_threads(r.d);
    switch (row_packs(r.d)) {
        case 1: k_norm_fwd<T, 1><<<grid, th, 0, st>>>(r); break;
        case 2: k_norm_fwd<T, 2><<<grid, th, 0, st>>>(r); break;
        default: k_norm_fwd<T, 4><<<grid, th, 0, st>>>(r); break;
    }
    return host_launched();
}

template <typename T>
lce_status_t backward(const lce_norm_t *a, float *part, const HostDev &dev, cudaStream_t st) {
    NormArgs r = make_norm(a);
    r.part = part;
    r.status = dev.status;
    const bool full_gate = r.gate && r.gate_full;
    const int arrays = (r.w_pre ? 2 : 0) + (r.b ? 1 : 0) + (full_gate ? 1 : 0) + (r.dr ? 1 : 0);
    RingGeo g;
    int grid;
    lce_status_t s;
    // two rows a thread while a row's packs go round once (their sums and the column sums fill the registers), else one;
    // packs a thread: one, or as many as a row needs of 512 threads
    const int packs = r.d * static_cast<int>(sizeof(T)) / 16;
    const int ch = packs <= kRingThreads ? 1 : packs <= 2 * kRingThreads ? 2 : 16 / kPack<T>, per = ch == 1 ? 2 : 1;
    if (ring_geo(&g, r.d, sizeof(T), arrays, ch, per, kRingBytes)) {
        grid = ring_grid(a->N, g.groups * per, dev.sms);
        const int smem = std::max<int>(g.stages * g.stage_bytes + 3 * g.row_bytes, g.groups * r.d * 4);
        const int mode = !r.w_pre ? NORM_POST : !r.b ? NORM_PRE : full_gate ? NORM_FULL_GATE : r.dr ? NORM_ALL : NORM_NO_DR;
        auto go = [&](auto c, auto rows) {
            constexpr int CH = decltype(c)::value, R = decltype(rows)::value;
            switch (mode) {
                case NORM_ALL: return launch_ring<k_norm_bwd_ring<T, CH, R, NORM_ALL>>(dev, r, g, grid, smem, st);
                case NORM_NO_DR: return launch_ring<k_norm_bwd_ring<T, CH, R, NORM_NO_DR>>(dev, r, g, grid, smem, st);
                case NORM_FULL_GATE: return launch_ring<k_norm_bwd_ring<T, CH, R, NORM_FULL_GATE>>(dev, r, g, grid, smem, st);
                case NORM_PRE: return launch_ring<k_norm_bwd_ring<T, CH, R, NORM_PRE>>(dev, r, g, grid, smem, st);
                default: return launch_ring<k_norm_bwd_ring<T, CH, R, NORM_POST>>(dev, r, g, grid, smem, st);
            }
        };
        switch (ch) {
            case 1: s = go(std::integral_constant<int, 1>(), std::integral_constant<int, 2>()); break;
            case 2: s = go(std::integral_constant<int, 2>(), std::integral_constant<int, 1>()); break;
            default: s = go(std::integral_constant<int, 16 / kPack<T>>(), std::integral_constant<int, 1>());   // fp32: 4
        }
    } else {
        grid = ring_grid(a->N, 1, kColGroups);
        const int th = row_threads(r.d), smem = 3 * r.d * 4;
        auto go = [&](auto kernel) {
            kernel<<<grid, th, smem, st>>>(r);
            return host_launched();
        };
        // (over 8192 elements of bf16, over 4096 of fp32: the ring takes the others whatever the options)
        constexpr int kWide = sizeof(T) == 4 ? 2 : 4;
        if (row_packs(r.d) <= kWide) s = host_smem<k_norm_bwd<T, kWide>>(dev, 3 * kWide * 4096 * 4);
        else s = host_smem<k_norm_bwd<T, 4>>(dev, 3 * 4 * 4096 * 4);
        if (s == LCE_OK) s = row_packs(r.d) <= kWide ? go(k_norm_bwd<T, kWide>) : go(k_norm_bwd<T, 4>);
    }
    if (s != LCE_OK) return s;
    T *dgate = r.gate && !full_gate ? static_cast<T *>(a->dgate) : nullptr;
    T *dpre = r.w_pre ? static_cast<T *>(a->dw_pre) : nullptr, *dpost = r.w_post ? static_cast<T *>(a->dw_post) : nullptr;
    if (!dgate && !dpre && !dpost) return LCE_OK;
    return host_launch_early(k_norm_cols<T>, dim3((r.d + 31) / 32, 3), 256, 0, st, part, grid, r.d, dpre, dpost, dgate);
}

}  // namespace

extern "C" {

size_t lce_block_norm_workspace_size(const lce_norm_t *a) {
    if (!a || a->N < 0 || a->N >= (int64_t(1) << 31) || a->d < 8 || a->d > kMaxD || a->d % 8) return 0;
    return static_cast<size_t>(3 * kColGroups * a->d) * sizeof(float);
}

lce_status_t lce_block_norm_forward(const lce_norm_t *a) {
    lce_status_t s = check_norm(a, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (a->N == 0) return LCE_OK;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    return a->dtype == LCE_BF16 ? forward<__nv_bfloat16>(a, dev, st) : forward<float>(a, dev, st);
}

lce_status_t lce_block_norm_backward(const lce_norm_t *a) {
    lce_status_t s = check_norm(a, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    if ((s = scratch.get(a->workspace, a->workspace_bytes, lce_block_norm_workspace_size(a), &base)) != LCE_OK) return s;
    float *part = reinterpret_cast<float *>(base);
    return a->dtype == LCE_BF16 ? backward<__nv_bfloat16>(a, part, dev, st) : backward<float>(a, part, dev, st);
}

}  // extern "C"
