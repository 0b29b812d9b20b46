// Layer norm with the residual sum before it: kernels and host side of
// lce_layer_norm_forward / _backward.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "e4m3.cuh"
#include "lce_host.h"
#include "row_ring.cuh"

using namespace lce;

namespace {

struct LnArgs {
    const void *x, *b, *w, *c, *r_in, *dr, *dn;
    void *r, *n, *dx;
    float *mean, *rstd;
    uint8_t *codes;
    int8_t *exps;
    int64_t ld_x, ld_b, ld_r, ld_dr, ld_dn, ld_codes, ld_exps;
    int64_t N;
    int d;
    float eps;
    int *status;
    float *part;   // backward: partial column sums [2][groups][d] (weight, bias)
};

// One block a row, a thread holds CH packs of its row's elements.
template <typename T, int CH>
__global__ void __launch_bounds__(512) k_ln_fwd(const LnArgs a) {
    __shared__ float red[64];
    int flip = 0;
    const int64_t row = blockIdx.x;
    const int d = a.d;
    float r[CH][kVec], s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * blockDim.x + threadIdx.x) * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i) r[c][i] = 0.f;
        if (col < d) {
            load_pack(static_cast<const T *>(a.x) + row * a.ld_x + col).get(r[c]);
            if (a.b) {
                float t[kVec];
                load_pack(static_cast<const T *>(a.b) + row * a.ld_b + col).get(t);
#pragma unroll
                for (int i = 0; i < kVec; ++i) t[i] += r[c][i];
                Pack<T> v;
                v.set(t);
                *reinterpret_cast<Pack<T> *>(static_cast<T *>(a.r) + row * d + col) = v;
                v.get(r[c]);   // as it is stored
            }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) s[0] += r[c][i];
        if (a.codes) {
            uint32_t bits[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) bits[i] = __float_as_uint(r[c][i]);
            const int e = pack_exponent(block_top<float, kVec, kPackBlock / kVec>(bits));
            if (col < d) {
                *reinterpret_cast<uint2 *>(a.codes + row * a.ld_codes + col) = codes8(r[c], pack_scale(e));
                if (col % kPackBlock == 0) a.exps[col / kPackBlock * a.ld_exps + row] = static_cast<int8_t>(e);
            }
        }
    }
    block_sum(s, red, flip);
    const float mean = s[0] / d;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if ((c * blockDim.x + threadIdx.x) * kVec < d)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                r[c][i] -= mean;
                s[0] = fmaf(r[c][i], r[c][i], s[0]);
            }
    block_sum(s, red, flip);
    const float rs = rsqrtf(s[0] / d + a.eps);
    if (threadIdx.x == 0) a.mean[row] = mean, a.rstd[row] = rs;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * blockDim.x + threadIdx.x) * kVec;
        if (col < d) {
            float w[kVec], t[kVec];
            load_pack(static_cast<const T *>(a.w) + col).get(w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = 0.f;
            if (a.c) load_pack(static_cast<const T *>(a.c) + col).get(t);
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = fmaf(r[c][i] * rs, w[i], t[i]);
            store_pack(static_cast<T *>(a.n) + row * d + col, t);
        }
    }
}

// Persistent blocks, one row at a time; the column sums stay in shared memory,
// each column owned by one thread, until the block's rows are done. For rows that
// leave no room for two stages of a ring: nothing is loaded ahead, and every
// element reads and writes two sums (8192 x 8192 fp32 with dr 434 us, where the
// copy rate would take 158; from 8 bits the ring holds them: 137).
template <typename T, int CH>
__global__ void __launch_bounds__(512) k_ln_bwd(const LnArgs a) {
    extern __shared__ float sums[];   // [2][d]
    __shared__ float red[2 * 32 * 2];
    int flip = 0;
    const int d = a.d;
    const float inv_d = 1.f / d;
    for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) sums[i] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const float mean = a.mean[row], rs = a.rstd[row];
        float hat[CH][kVec], u[CH][kVec];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col >= d) continue;
            float t[kVec];
            if (a.codes) values8(*reinterpret_cast<const uint2 *>(a.codes + row * a.ld_codes + col),
                                 unpack_scale(a.exps[col / kPackBlock * a.ld_exps + row]), hat[c]);
            else load_pack(static_cast<const T *>(a.r_in) + row * a.ld_r + col).get(hat[c]);
            load_pack(static_cast<const T *>(a.dn) + row * a.ld_dn + col).get(u[c]);
            load_pack(static_cast<const T *>(a.w) + col).get(t);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                hat[c][i] = (hat[c][i] - mean) * rs;
                sums[col + i] += u[c][i] * hat[c][i];
                sums[d + col + i] += u[c][i];
                u[c][i] *= t[i];
                s[0] += u[c][i];
                s[1] = fmaf(u[c][i], hat[c][i], s[1]);
            }
        }
        block_sum(s, red, flip);
        const float m0 = s[0] * inv_d, m1 = s[1] * inv_d;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * blockDim.x + threadIdx.x) * kVec;
            if (col >= d) continue;
            float t[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = 0.f;
            if (a.dr) load_pack(static_cast<const T *>(a.dr) + row * a.ld_dr + col).get(t);
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = fmaf(rs, u[c][i] - m0 - hat[c][i] * m1, t[i]);
            store_pack(static_cast<T *>(a.dx) + row * d + col, t);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d; i += blockDim.x)
        a.part[(static_cast<int64_t>(i / d) * gridDim.x + blockIdx.x) * d + i % d] = sums[i];
}

// ---------------------------------------------------------------- ring kernels
//
// Persistent blocks whose rows arrive through a ring of bulk copies, as in the
// block norms; what a thread holds of a row are packs of 16 bytes, `tpr` threads
// a row, and row groups join their sums on barriers of their own.

constexpr int kLnArrays = 3;
struct LnGeo {
    int tpr, groups, stages, arrays;
    uint32_t row_bytes;                              // of the tensors' type
    uint32_t bytes[kLnArrays], at[kLnArrays];        // of a row of each array; the array's place in a stage
    uint32_t stage_bytes;
};
struct LnSource {
    const uint8_t *src[kLnArrays];
    int64_t ld[kLnArrays];   // bytes
    // Starts the copies of the `per` rows from r0 on into stage s, if there are
    // any. Rows past the last arrive as copies of the last.
    template <bool kOnce>
    __device__ __forceinline__ void issue(uint8_t *ring, RingBars &bars, const LnGeo &g, int per, int s, int64_t r0, int64_t N) const {
        if (r0 >= N) return;
        mbar_arrive_expect_tx(&bars.full[s], g.stage_bytes);
        uint8_t *stage = ring + s * g.stage_bytes;
        auto load = [&](uint8_t *to, const uint8_t *from, uint32_t bytes) {
            if (kOnce) bulk_load_once(to, from, bytes, &bars.full[s]);
            else bulk_load(to, from, bytes, &bars.full[s]);
        };
#pragma unroll
        for (int k = 0; k < kLnArrays; ++k) {
            if (k >= g.arrays) continue;
            if (ld[k] == g.bytes[k] && r0 + per <= N) load(stage + g.at[k], src[k] + r0 * ld[k], per * g.bytes[k]);
            else
                for (int r = 0; r < per; ++r) load(stage + g.at[k] + r * g.bytes[k], src[k] + min(r0 + r, N - 1) * ld[k], g.bytes[k]);
        }
    }
};
// After a wait that gave up in stage s: lets the copies in flight land.
__device__ __forceinline__ void ln_drain(RingBars &bars, const LnGeo &g, int per, int s, uint32_t phase, int64_t r0, int64_t N) {
    for (int i = 0; i < g.stages && r0 < N; ++i, r0 += static_cast<int64_t>(gridDim.x) * per) {
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&bars.full[s]), phase) && clock64() - t0 < kNormWaitCycles / 10) {}
        if (++s == g.stages) s = 0, phase ^= 1;
    }
}

// A row's weights in shared memory (zeros where there are none)
__device__ __forceinline__ void load_row(uint8_t *dst, const void *w, int row_bytes) {
    for (int i = threadIdx.x * 16; i < row_bytes; i += blockDim.x * 16)
        *reinterpret_cast<uint4 *>(dst + i) = w ? *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(w) + i) : make_uint4(0, 0, 0, 0);
}

// Forward. kAdd: there is a block's output to add; kKeep: r is packed as well (a
// block of 128 channels lies in 16 lanes' packs of bf16, in a warp's of fp32).
template <typename T, int CH, bool kAdd, bool kKeep>
__global__ void __launch_bounds__(kRingThreads, 1) k_ln_fwd_ring(const LnArgs a, const LnGeo g) {
    constexpr int V = kPack<T>, P = V / 2;
    extern __shared__ __align__(128) uint8_t smem[];   // ring, then weight, bias
    __shared__ RingBars bars;
    __shared__ __align__(16) float red[16 * kRedFloats];
    const int nwarps = blockDim.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], nwarps);
        for (int i = 0; i < 16; ++i) bars.gave_up[i] = 0;
        fence_mbar_init();
    }
    uint8_t *w_row = smem + g.stages * g.stage_bytes, *c_row = w_row + g.row_bytes;
    load_row(w_row, a.w, g.row_bytes);
    load_row(c_row, a.c, g.row_bytes);
    for (int i = threadIdx.x; i < 16 * kRedFloats; i += blockDim.x) red[i] = 0.f;
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.groups;
    int64_t r0 = static_cast<int64_t>(blockIdx.x) * g.groups;
    const LnSource src = {{static_cast<const uint8_t *>(a.x), static_cast<const uint8_t *>(a.b), nullptr},
                          {a.ld_x * static_cast<int>(sizeof(T)), a.ld_b * static_cast<int>(sizeof(T)), 0}};
    if (threadIdx.x == 0)
        for (int i = 0; i < g.stages; ++i) src.issue<true>(smem, bars, g, g.groups, i, r0 + i * step, a.N);
    const int group = threadIdx.x / g.tpr, t = threadIdx.x % g.tpr;
    float *my_red = red + group * kRedFloats;
    const float inv_d = 1.f / a.d;
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
        f32x2 q = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            const bool in = byte < g.row_bytes;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(at + byte);
            Pack16<T>::get(x, r[c]);
            if (kAdd) {
                f32x2 b[P];
                uint4 v = make_uint4(0, 0, 0, 0);
                if (in) v = *reinterpret_cast<const uint4 *>(at + g.at[1] + byte);
                Pack16<T>::get(v, b);
#pragma unroll
                for (int i = 0; i < P; ++i) b[i] = add2(r[c][i], b[i]);
                x = Pack16<T>::set(b);
                if (live && in) __stcs(reinterpret_cast<uint4 *>(out_r + c * g.tpr * 16), x);
                Pack16<T>::get(x, r[c]);   // as it is stored
            }
#pragma unroll
            for (int i = 0; i < P; ++i) q = add2(q, r[c][i]);
            if (kKeep) {
                const uint32_t words[4] = {x.x, x.y, x.z, x.w};
                const uint32_t top = block_top<T, 4, kPackBlock / V>(words);
                const int e = pack_exponent(top), col = (c * g.tpr + t) * V;
                const uint2 codes = pack_codes<T>(r[c], pack_scale(e));
                if (live && in) {
                    uint8_t *to = a.codes + row * a.ld_codes + col;
                    if (sizeof(T) == 2) *reinterpret_cast<uint2 *>(to) = codes;
                    else *reinterpret_cast<uint32_t *>(to) = codes.x;
                    if (col % kPackBlock == 0) a.exps[col / kPackBlock * a.ld_exps + row] = static_cast<int8_t>(e);
                }
            }
        }
        float sum[1] = {hsum2(q)};
        group_sum(sum, my_red, flip, g.tpr, group, t);
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(&bars.empty[s]);   // everything is in registers: it has gone into the sum
        const float mean = sum[0] / a.d;   // not * inv_d: a row of one value has that as its mean, and no spread
        const f32x2 minus = both(-mean);
        q = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if ((c * g.tpr + t) * 16 >= g.row_bytes) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) r[c][i] = add2(r[c][i], minus), q = fma2(r[c][i], r[c][i], q);
        }
        sum[0] = hsum2(q);
        group_sum(sum, my_red, flip, g.tpr, group, t);
        if (bars.gave_up[group]) {
            if (threadIdx.x == 0) ln_drain(bars, g, g.groups, s, phase, r0, a.N);
            break;
        }
        // the stage's next rows, once every warp has taken its share
        if (threadIdx.x == 0 && r0 + g.stages * step < a.N && ring_wait(&bars.empty[s], phase, a.status))
            src.issue<true>(smem, bars, g, g.groups, s, r0 + g.stages * step, a.N);
        const float rs = rsqrtf(sum[0] * inv_d + a.eps);
        if (t == 0 && live) a.mean[row] = mean, a.rstd[row] = rs;
        const f32x2 f = both(rs);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            if (byte >= g.row_bytes) continue;
            f32x2 w[P], y[P];
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_row + byte), w);
            Pack16<T>::get(*reinterpret_cast<const uint4 *>(c_row + byte), y);
#pragma unroll
            for (int i = 0; i < P; ++i) y[i] = fma2(mul2(r[c][i], f), w[i], y[i]);
            if (live) *reinterpret_cast<uint4 *>(out_n + c * g.tpr * 16) = Pack16<T>::set(y);
        }
        if (++s == g.stages) s = 0, phase ^= 1;
    }
}

// Backward (16384 x 4096 bf16 with dr 92 us, 86% of the copy rate; from 8 bits 96,
// though that reads 67 MB less: both are at the pace of a row's instructions and
// its sums, 16 warps an SM issuing in 53% of the cycles, and from codes a row
// takes 6% more of them; fp32, half the elements a byte, 159 and 155).
// A thread's columns of R rows at a time: the two row sums in one
// round; the column sums stay in registers, one set a row group, and are joined
// across the groups in shared memory at the end. kCodes: the stream comes in 8
// bits; kDr: there is a gradient of r.
template <typename T, int CH, int R, bool kCodes, bool kDr>
__global__ void __launch_bounds__(kRingThreads, 1) k_ln_bwd_ring(const LnArgs a, const LnGeo g) {
    constexpr int V = kPack<T>, P = V / 2;
    extern __shared__ __align__(128) uint8_t smem[];   // ring, then weight
    __shared__ RingBars bars;
    __shared__ __align__(16) float red[16 * kRedFloats];
    const int nwarps = blockDim.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], nwarps);
        for (int i = 0; i < 16; ++i) bars.gave_up[i] = 0;
        fence_mbar_init();
    }
    uint8_t *w_row = smem + g.stages * g.stage_bytes;
    load_row(w_row, a.w, g.row_bytes);
    for (int i = threadIdx.x; i < 16 * kRedFloats; i += blockDim.x) red[i] = 0.f;
    __syncthreads();
    const int per = g.groups * R;   // rows of a stage
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    int64_t r0 = static_cast<int64_t>(blockIdx.x) * per;
    const LnSource src = {{kCodes ? a.codes : static_cast<const uint8_t *>(a.r_in), static_cast<const uint8_t *>(a.dn), static_cast<const uint8_t *>(a.dr)},
                          {kCodes ? a.ld_codes : a.ld_r * static_cast<int>(sizeof(T)), a.ld_dn * static_cast<int>(sizeof(T)), a.ld_dr * static_cast<int>(sizeof(T))}};
    if (threadIdx.x == 0)
        for (int i = 0; i < g.stages; ++i) src.issue<false>(smem, bars, g, per, i, r0 + i * step, a.N);
    const int group = threadIdx.x / g.tpr, t = threadIdx.x % g.tpr;
    float *my_red = red + group * kRedFloats;
    const float inv_d = 1.f / a.d;
    f32x2 s_w[CH][P], s_c[CH][P];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < P; ++i) s_w[c][i] = s_c[c][i] = both(0.f);
    uint8_t *out = static_cast<uint8_t *>(a.dx) + (r0 + group * R) * g.row_bytes + t * 16;
    int flip = 0, s = 0;
    uint32_t phase = 0;
    // statistics (and exponents) of the rows to come, asked for a round ahead; zeros past the last row
    float mean_next[R], rs_next[R];
    int e_next[R][CH];
    auto ask = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool live = row + k < a.N;
            mean_next[k] = live ? a.mean[row + k] : 0.f;
            rs_next[k] = live ? a.rstd[row + k] : 0.f;
            if (kCodes)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int col = (c * g.tpr + t) * V;
                    e_next[k][c] = live && col < a.d ? a.exps[col / kPackBlock * a.ld_exps + row + k] : 0;
                }
        }
    };
    ask(r0 + group * R);
    for (; r0 < a.N; r0 += step, out += step * g.row_bytes) {
        const int64_t row = r0 + group * R;
        float mean[R], rs[R], scale[R][CH];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] = mean_next[k], rs[k] = rs_next[k];
            if (kCodes)
#pragma unroll
                for (int c = 0; c < CH; ++c) scale[k][c] = unpack_scale(e_next[k][c]);
        }
        ask(row + step);
        if (!__all_sync(0xffffffffu, ring_wait(&bars.full[s], phase, a.status))) bars.gave_up[group] = 1;
        const uint8_t *stage = smem + s * g.stage_bytes;
        f32x2 hat[R][CH][P], u[R][CH][P], q[R][2];
#pragma unroll
        for (int k = 0; k < R; ++k) q[k][0] = q[k][1] = both(0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            f32x2 w[P];
            const bool in = byte < g.row_bytes;
            if (in) Pack16<T>::get(*reinterpret_cast<const uint4 *>(w_row + byte), w);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (!in || row + k >= a.N) {   // rows past the last add nothing to the columns
#pragma unroll
                    for (int i = 0; i < P; ++i) hat[k][c][i] = u[k][c][i] = both(0.f);
                    continue;
                }
                if (kCodes) {
                    const uint8_t *from = stage + (group * R + k) * g.bytes[0] + (c * g.tpr + t) * V;
                    const uint2 codes = sizeof(T) == 2 ? *reinterpret_cast<const uint2 *>(from) : make_uint2(*reinterpret_cast<const uint32_t *>(from), 0);
                    pack_values<T>(codes, scale[k][c], hat[k][c]);
                }
                else Pack16<T>::get(*reinterpret_cast<const uint4 *>(stage + (group * R + k) * g.bytes[0] + byte), hat[k][c]);
                Pack16<T>::get(*reinterpret_cast<const uint4 *>(stage + g.at[1] + (group * R + k) * g.row_bytes + byte), u[k][c]);
                const f32x2 minus = both(-mean[k]), f = both(rs[k]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    hat[k][c][i] = mul2(add2(hat[k][c][i], minus), f);
                    s_w[c][i] = fma2(u[k][c][i], hat[k][c][i], s_w[c][i]);
                    s_c[c][i] = add2(u[k][c][i], s_c[c][i]);
                    u[k][c][i] = mul2(u[k][c][i], w[i]);
                    q[k][0] = add2(q[k][0], u[k][c][i]);
                    q[k][1] = fma2(u[k][c][i], hat[k][c][i], q[k][1]);
                }
            }
        }
        float sum[2 * R];
#pragma unroll
        for (int k = 0; k < R; ++k) sum[2 * k] = hsum2(q[k][0]), sum[2 * k + 1] = hsum2(q[k][1]);
        group_sum(sum, my_red, flip, g.tpr, group, t);
        if (bars.gave_up[group]) {
            if (threadIdx.x == 0) ln_drain(bars, g, per, s, phase, r0, a.N);
            break;
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int byte = (c * g.tpr + t) * 16;
            if (byte >= g.row_bytes) continue;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (row + k >= a.N) continue;
                const f32x2 m0 = both(-sum[2 * k] * inv_d), m1 = both(-sum[2 * k + 1] * inv_d), f = both(rs[k]);
                f32x2 y[P];
                if (kDr) Pack16<T>::get(*reinterpret_cast<const uint4 *>(stage + g.at[2] + (group * R + k) * g.row_bytes + byte), y);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const f32x2 v = fma2(hat[k][c][i], m1, add2(u[k][c][i], m0));
                    y[i] = kDr ? fma2(v, f, y[i]) : mul2(v, f);
                }
                *reinterpret_cast<uint4 *>(out + k * g.row_bytes + c * g.tpr * 16) = Pack16<T>::set(y);
            }
        }
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(&bars.empty[s]);
        // the stage's next rows, once every warp is through with it
        if (threadIdx.x == 0 && r0 + g.stages * step < a.N && ring_wait(&bars.empty[s], phase, a.status))
            src.issue<false>(smem, bars, g, per, s, r0 + g.stages * step, a.N);
        if (++s == g.stages) s = 0, phase ^= 1;
    }
    // the groups' sums, [group][d] at a time through the (now idle) ring
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * g.tpr + t) * V;
            if (col >= a.d) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 v;
                unpack2(k == 0 ? s_w[c][i] : s_c[c][i], v.x, v.y);
                *reinterpret_cast<float2 *>(sums + group * a.d + col + 2 * i) = v;
            }
        }
        __syncthreads();
        float *to = a.part + (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * a.d;
        for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
            float v = 0.f;
            for (int q = 0; q < g.groups; ++q) v += sums[q * a.d + i];
            to[i] = v;
        }
        __syncthreads();
    }
}

constexpr int64_t kMaxD = 16384;
constexpr int kColGroups = 304;   // blocks of the backward at most (bounds its workspace)

lce_status_t check_rows(const void *p, int64_t ld, int elt) {
    if (ld < 0 || ld >= (int64_t(1) << 36)) return LCE_ERR_SHAPE;
    if (host_misaligned(p) || (ld * elt) % 16) return LCE_ERR_ALIGN;
    return LCE_OK;
}

lce_status_t check_ln(const lce_layer_norm_t *a, bool backward) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->N < 0 || a->N >= (int64_t(1) << 31) || a->d < 8 || a->d > kMaxD) return LCE_ERR_SHAPE;
    if (a->d % 8) return LCE_ERR_ALIGN;
    if (!backward && (!(a->eps >= 0.f) || a->eps - a->eps != 0.f)) return LCE_ERR_ARG;
    if (a->N == 0 && !backward) return LCE_OK;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    // `rows`: touched only when there are rows (the column sums are written without any)
    const struct { const void *p; int64_t ld; bool used, want, rows; } all[] = {
        {a->x, a->ld_x, !backward, true, true}, {a->b, a->ld_b, !backward, false, true},
        {a->weight, 0, true, true, false}, {a->bias, 0, !backward, false, false},
        {a->r, backward ? a->ld_r : 0, backward ? !a->codes : a->b != nullptr, true, true}, {a->n, 0, !backward, true, true},
        {a->dn, a->ld_dn, backward, true, true}, {a->dr, a->ld_dr, backward, false, true}, {a->dx, 0, backward, true, true},
        {a->dweight, 0, backward, true, false}, {a->dbias, 0, backward, false, false}};
    if (a->N > 0 && (!a->mean || !a->rstd)) return LCE_ERR_NULL;
    for (const auto &t : all) {
        if (!t.used || (t.rows && a->N == 0)) continue;
        if (t.want && !t.p) return LCE_ERR_NULL;
        const lce_status_t s = check_rows(t.p, t.ld, elt);
        if (s != LCE_OK) return s;
    }
    return a->codes && a->N > 0 ? host_check_packed(a->codes, a->ld_codes, a->exps, a->ld_exps, a->N, a->d) : LCE_OK;
}

LnArgs make_args(const lce_layer_norm_t *a, const HostDev &dev) {
    LnArgs r{};
    auto ld = [&](int64_t v) { return v ? v : a->d; };
    r.x = a->x, r.b = a->b, r.w = a->weight, r.c = a->bias, r.r_in = a->r, r.dr = a->dr, r.dn = a->dn;
    r.r = a->r, r.n = a->n, r.dx = a->dx, r.mean = a->mean, r.rstd = a->rstd, r.codes = a->codes, r.exps = a->exps;
    r.ld_x = ld(a->ld_x), r.ld_b = ld(a->ld_b), r.ld_r = ld(a->ld_r), r.ld_dr = ld(a->ld_dr), r.ld_dn = ld(a->ld_dn);
    r.ld_codes = a->ld_codes, r.ld_exps = a->ld_exps;
    r.N = a->N, r.d = static_cast<int>(a->d), r.eps = a->eps, r.status = dev.status;
    return r;
}

// Threads of a row's block: one pack each up to 512 of them, then more packs.
int row_threads(int d) {
    const int packs = d / kVec;
    return packs >= 512 ? 512 : (packs + 31) / 32 * 32;
}

constexpr int kRingBytes = 208 * 1024;      // dynamic shared memory of a ring kernel's block at most
constexpr int kFwdRingBytes = 128 * 1024;   // ring of the forward, if two stages do not take more
// Few rows have nothing to run ahead of: up to this much of an array the forward takes a block for each row.
constexpr int64_t kDirectBytes = 4 << 20;

// The ring kernels' geometry for rows of d elements: `ch` packs a thread, `per` rows a group and stage, `weights` rows
// beside the ring; codes: the first array is of bytes. False where rows are too wide.
bool ln_geo(LnGeo *g, int d, int elt, int arrays, bool codes, int ch, int per, int weights, int bytes) {
    const int packs = d * elt / 16;
    g->tpr = ((packs + ch - 1) / ch + 31) / 32 * 32;
    if (g->tpr > kRingThreads) return false;
    g->groups = kRingThreads / g->tpr;
    g->arrays = arrays;
    g->row_bytes = d * elt;
    g->stage_bytes = 0;
    for (int k = 0; k < kLnArrays; ++k) {
        g->bytes[k] = k == 0 && codes ? (d + 15) / 16 * 16 : g->row_bytes;
        g->at[k] = g->stage_bytes;
        if (k < arrays) g->stage_bytes += g->groups * per * g->bytes[k];
    }
    const int rows = weights * static_cast<int>(g->row_bytes), stage = static_cast<int>(g->stage_bytes);
    if (2 * stage + rows > kRingBytes) return false;
    g->stages = std::max(2, std::min(kRingMaxStages, std::min(bytes, kRingBytes - rows) / stage));
    return true;
}

// Rows are handed out a stage at a time; at least one block, so that column sums of no rows come out as zeros.
int ring_grid(int64_t N, int rows, int most) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((N + rows - 1) / rows, most))); }

template <auto kKernel>
lce_status_t launch_ring(const HostDev &dev, const LnArgs &r, const LnGeo &g, int grid, int smem, cudaStream_t st) {
    const lce_status_t s = host_smem<kKernel>(dev, kRingBytes);
    if (s != LCE_OK) return s;
    kKernel<<<grid, g.tpr * g.groups, smem, st>>>(r, g);
    return host_launched();
}

template <typename T>
lce_status_t forward(const LnArgs &r, const HostDev &dev, cudaStream_t st) {
    LnGeo g;
    // packs a thread: as few as leave a row to 32 threads, at most 32 elements
    int ch = 1;
    while (ch < 32 / kPack<T> && r.d * static_cast<int>(sizeof(T)) / 16 > 32 * ch) ch *= 2;
    if (r.N * r.d * static_cast<int64_t>(sizeof(T)) > kDirectBytes && ln_geo(&g, r.d, sizeof(T), r.b ? 2 : 1, false, ch, 1, 2, kFwdRingBytes)) {
        const int grid = ring_grid(r.N, g.groups, dev.sms), smem = g.stages * g.stage_bytes + 2 * g.row_bytes;
        auto go = [&](auto c) {
            constexpr int CH = decltype(c)::value;
            return r.b ? r.codes ? launch_ring<k_ln_fwd_ring<T, CH, true, true>>(dev, r, g, grid, smem, st)
                                 : launch_ring<k_ln_fwd_ring<T, CH, true, false>>(dev, r, g, grid, smem, st)
                       : r.codes ? launch_ring<k_ln_fwd_ring<T, CH, false, true>>(dev, r, g, grid, smem, st)
                                 : launch_ring<k_ln_fwd_ring<T, CH, false, false>>(dev, r, g, grid, smem, st);
        };
        switch (ch) {
            case 1: return go(std::integral_constant<int, 1>());
            case 2: return go(std::integral_constant<int, 2>());
            case 4: return go(std::integral_constant<int, 4>());
            default: return go(std::integral_constant<int, 32 / kPack<T>>());   // fp32: 8
        }
    }
    const unsigned grid = static_cast<unsigned>(r.N);
    const int th = row_threads(r.d), packs = (r.d / kVec + 511) / 512;
    switch (packs) {
        case 1: k_ln_fwd<T, 1><<<grid, th, 0, st>>>(r); break;
        case 2: k_ln_fwd<T, 2><<<grid, th, 0, st>>>(r); break;
        default: k_ln_fwd<T, 4><<<grid, th, 0, st>>>(r); break;
    }
    return host_launched();
}

template <typename T>
lce_status_t backward(const lce_layer_norm_t *a, const LnArgs &r, const HostDev &dev, cudaStream_t st) {
    LnGeo g;
    int grid;
    lce_status_t s;
    // two rows a thread while a row's packs go round once, else one; packs a thread: one, or as many as a row needs of 512 threads
    const int packs = r.d * static_cast<int>(sizeof(T)) / 16;
    const int ch = packs <= kRingThreads ? 1 : packs <= 2 * kRingThreads ? 2 : 16 / kPack<T>, per = ch == 1 ? 2 : 1;
    if (ln_geo(&g, r.d, sizeof(T), r.dr ? 3 : 2, r.codes != nullptr, ch, per, 1, kRingBytes)) {
        grid = ring_grid(r.N, g.groups * per, dev.sms);
        const int smem = std::max<int>(g.stages * g.stage_bytes + g.row_bytes, g.groups * r.d * 4);
        auto go = [&](auto c, auto rows) {
            constexpr int CH = decltype(c)::value, R = decltype(rows)::value;
            return r.codes ? r.dr ? launch_ring<k_ln_bwd_ring<T, CH, R, true, true>>(dev, r, g, grid, smem, st)
                                  : launch_ring<k_ln_bwd_ring<T, CH, R, true, false>>(dev, r, g, grid, smem, st)
                           : r.dr ? launch_ring<k_ln_bwd_ring<T, CH, R, false, true>>(dev, r, g, grid, smem, st)
                                  : launch_ring<k_ln_bwd_ring<T, CH, R, false, false>>(dev, r, g, grid, smem, st);
        };
        switch (ch) {
            case 1: s = go(std::integral_constant<int, 1>(), std::integral_constant<int, 2>()); break;
            case 2: s = go(std::integral_constant<int, 2>(), std::integral_constant<int, 1>()); break;
            default: s = go(std::integral_constant<int, 16 / kPack<T>>(), std::integral_constant<int, 1>());   // fp32: 4
        }
    } else {   // rows too wide for two stages
        grid = ring_grid(r.N, 1, kColGroups);
        const int th = row_threads(r.d), smem = 2 * r.d * 4;
        if ((s = host_smem<k_ln_bwd<T, 4>>(dev, 2 * kMaxD * 4)) == LCE_OK) {
            k_ln_bwd<T, 4><<<grid, th, smem, st>>>(r);
            s = host_launched();
        }
    }
    if (s != LCE_OK) return s;
    return host_launch_early(k_norm_cols<T>, dim3((r.d + 31) / 32, 2), 256, 0, st, r.part, grid, r.d, static_cast<T *>(a->dweight),
                             static_cast<T *>(a->dbias), static_cast<T *>(nullptr));
}

}  // namespace

extern "C" {

size_t lce_layer_norm_workspace_size(const lce_layer_norm_t *a) {
    if (!a || a->N < 0 || a->N >= (int64_t(1) << 31) || a->d < 8 || a->d > kMaxD || a->d % 8) return 0;
    return static_cast<size_t>(2 * kColGroups * a->d) * sizeof(float);
}

lce_status_t lce_layer_norm_forward(const lce_layer_norm_t *a) {
    lce_status_t s = check_ln(a, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (a->N == 0) return LCE_OK;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    const LnArgs r = make_args(a, dev);
    return a->dtype == LCE_BF16 ? forward<__nv_bfloat16>(r, dev, st) : forward<float>(r, dev, st);
}

lce_status_t lce_layer_norm_backward(const lce_layer_norm_t *a) {
    lce_status_t s = check_ln(a, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    if ((s = scratch.get(a->workspace, a->workspace_bytes, lce_layer_norm_workspace_size(a), &base)) != LCE_OK) return s;
    LnArgs r = make_args(a, dev);
    r.part = reinterpret_cast<float *>(base);
    return a->dtype == LCE_BF16 ? backward<__nv_bfloat16>(a, r, dev, st) : backward<float>(a, r, dev, st);
}

}  // extern "C"
