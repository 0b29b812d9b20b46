// What the kernels over rows share: packs of a row's elements, sums over the
// threads of a block or of a row group, and a ring of shared-memory stages that
// untiled bulk copies fill with the rows to come.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "f32x2.cuh"
#include "lce.h"
#include "tc_ptx.cuh"

namespace lce {

constexpr int kVec = 8;   // elements a thread takes at a time: 16 bytes of bf16, 32 of fp32

template <typename T>
struct Pack;
template <>
struct Pack<float> {
    float4 a, b;
    __device__ __forceinline__ void get(float (&x)[kVec]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[kVec]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <>
struct Pack<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void get(float (&x)[kVec]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[kVec]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&p);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T>
__device__ __forceinline__ Pack<T> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T> *>(p);
}
template <typename T>
__device__ __forceinline__ void store_pack(T *p, const float (&x)[kVec]) {
    Pack<T> v;
    v.set(x);
    *reinterpret_cast<Pack<T> *>(p) = v;
}

// Sum of K values over the block's threads, the same for all of them, in a
// fixed order. `red`: shared, 2 x 32 x K floats; `flip` alternates between
// calls, so that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float *red, int &flip) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int m = 16; m; m >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    const int warps = blockDim.x / 32;
    if (warps == 1) return;
    float *at = red + flip * 32 * K;
    flip ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) at[(threadIdx.x / 32) * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += at[w * K + k];
}

struct RingGeo {
    int tpr, groups, stages;
    uint32_t row_bytes, array_bytes, stage_bytes;   // of one row; of one array's rows; of a stage
};

constexpr int kRingThreads = 512;   // threads of a block at most
constexpr int kRingMaxStages = 8;
constexpr long long kNormWaitCycles = 2000000000LL;   // ~1 s: far above any legitimate wait

template <typename T>
constexpr int kPack = 16 / sizeof(T);   // elements of a pack

// 16 bytes as packed pairs of fp32
template <typename T>
struct Pack16;
template <>
struct Pack16<float> {
    static __device__ __forceinline__ void get(const uint4 &v, f32x2 (&x)[2]) { x[0] = pack2u(v.x, v.y), x[1] = pack2u(v.z, v.w); }
    static __device__ __forceinline__ uint4 set(const f32x2 (&x)[2]) {
        float a, b, c, d;
        unpack2(x[0], a, b), unpack2(x[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    static constexpr uint32_t kOnes = 0x3f800000u;
};
template <>
struct Pack16<__nv_bfloat16> {
    static __device__ __forceinline__ f32x2 pair(uint32_t w) { return pack2u(w << 16, w & 0xffff0000u); }
    static __device__ __forceinline__ void get(const uint4 &v, f32x2 (&x)[4]) {
        x[0] = pair(v.x), x[1] = pair(v.y), x[2] = pair(v.z), x[3] = pair(v.w);
    }
    static __device__ __forceinline__ uint32_t word(f32x2 v) {
        float a, b;
        unpack2(v, a, b);
        __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&p);
    }
    static __device__ __forceinline__ uint4 set(const f32x2 (&x)[4]) { return make_uint4(word(x[0]), word(x[1]), word(x[2]), word(x[3])); }
    static constexpr uint32_t kOnes = 0x3f803f80u;
};

struct RingBars {
    uint64_t full[kRingMaxStages], empty[kRingMaxStages];
    volatile int gave_up[16];   // by row group
};

// A bounded wait. A row group whose wait gave up goes on to its next barrier
// all the same (its warps must not leave one another waiting there) and leaves
// the loop after it, on `gave_up`.
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, int *status) {
    const uint32_t at = smem_u32(bar);
    if (mbar_try_wait(at, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(at, parity)) {
        if (clock64() - t0 > kNormWaitCycles) {
            atomicOr(status, LCE_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The arrays of a ring, copied by thread 0 of the block. kOnce: first to leave L2.
template <typename T, int MAX, bool kOnce>
struct RingSource {
    const T *src[MAX];
    int64_t ld[MAX];   // row strides, elements
    // Starts the copies of the `per` rows from r0 on into stage s, if there are
    // any. Rows past the last arrive as copies of the last.
    __device__ __forceinline__ void issue(uint8_t *ring, RingBars &bars, const RingGeo &g, int per, int s, int64_t r0, int64_t N, int d) const {
        if (r0 >= N) return;
        int count = 0;
#pragma unroll
        for (int k = 0; k < MAX; ++k) count += src[k] != nullptr;
        mbar_arrive_expect_tx(&bars.full[s], count * per * g.row_bytes);
        uint8_t *dst = ring + s * g.stage_bytes;
#pragma unroll
        for (int k = 0; k < MAX; ++k) {
            if (!src[k]) continue;
            auto load = [&](uint8_t *to, const T *from, uint32_t bytes) {
                if (kOnce) bulk_load_once(to, from, bytes, &bars.full[s]);
                else bulk_load(to, from, bytes, &bars.full[s]);
            };
            if (ld[k] == d && r0 + per <= N) load(dst, src[k] + r0 * d, per * g.row_bytes);
            else
                for (int r = 0; r < per; ++r) load(dst + r * g.row_bytes, src[k] + min(r0 + r, N - 1) * ld[k], g.row_bytes);
            dst += g.array_bytes;
        }
    }
};

// After a wait that gave up in stage s: lets the copies in flight (of the rows
// from r0 on) land before the block gives up its memory.
__device__ __forceinline__ void ring_drain(RingBars &bars, const RingGeo &g, int per, int s, uint32_t phase, int64_t r0, int64_t N) {
    for (int i = 0; i < g.stages && r0 < N; ++i, r0 += static_cast<int64_t>(gridDim.x) * per) {
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&bars.full[s]), phase) && clock64() - t0 < kNormWaitCycles / 10) {}
        if (++s == g.stages) s = 0, phase ^= 1;
    }
}

// Sums of K <= 8 values over the `tpr` threads of a row group, the same for all
// of them, in a fixed order. Within a warp the values are dealt out while they
// are added: after exchanges over 16, 8 and 4 lanes a lane is left with one
// value's sum over a quarter of the warp (K = 1: five plain exchanges). Across
// the warps each adds up all partial sums by lanes again. `red`: the group's
// 2 x 8 x 16 floats, zero beyond its warps.
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float *red, int &flip, int tpr, int group, int t) {
    constexpr int M = K == 1 ? 1 : 8;
    const int lane = t & 31;
    float x[M];
#pragma unroll
    for (int k = 0; k < M; ++k) x[k] = k < K ? v[k] : 0.f;
    if (K == 1) {
#pragma unroll
        for (int m = 16; m; m >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], m);
    } else {
#pragma unroll
        for (int h = M / 2, m = 16; h; h >>= 1, m >>= 1) {
            const bool up = lane & m;
#pragma unroll
            for (int k = 0; k < M / 2; ++k)
                if (k < h) {
                    const float keep = up ? x[k + h] : x[k], send = up ? x[k] : x[k + h];
                    x[k] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
        }
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
        x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
    }
    // lane 4j (K > 1) now has the sum of value number j with its bits 4, 3, 2 in that order: j = lane >> 2
    if (tpr > 32) {
        float *at = red + flip * M * 16;
        flip ^= 1;
        if (K == 1 ? lane == 0 : (lane & 3) == 0) at[(K == 1 ? 0 : (lane >> 2)) * 16 + t / 32] = x[0];
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
        if (K == 1) {
            x[0] = at[lane & 15];
#pragma unroll
            for (int m = 8; m; m >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], m);
        } else {
            // four lanes a value, four warps' sums a lane
            const float4 y = *reinterpret_cast<const float4 *>(at + (lane >> 2) * 16 + (lane & 3) * 4);
            x[0] = (y.x + y.y) + (y.z + y.w);
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], 2);
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = K == 1 ? x[0] : __shfl_sync(0xffffffffu, x[0], 4 * k);
}

// Weights of a row into shared memory (ones where there are none)
template <typename T>
__device__ __forceinline__ void load_weights(uint8_t *dst, const void *w, int row_bytes) {
    constexpr uint32_t o = Pack16<T>::kOnes;
    for (int i = threadIdx.x * 16; i < row_bytes; i += blockDim.x * 16)
        *reinterpret_cast<uint4 *>(dst + i) = w ? *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(w) + i) : make_uint4(o, o, o, o);
}

constexpr int kRedFloats = 2 * 8 * 16;   // of a row group

// Adds the blocks' column sums: eight quads of columns a block, 32 threads a
// quad that each add every 32nd partial row, joined in a fixed order. Bounded by
// latency: 4 us for 152 blocks' sums over 3 x 4096 columns (in L2).
template <typename T>
__global__ void __launch_bounds__(256) k_norm_cols(const float *part, int groups, int d, T *dw_pre, T *dw_post,
                                                   T *dgate) {
    __shared__ float4 red[32][8];
    griddep_wait();
    T *out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (!out) return;
    const int x = threadIdx.x & 7, y = threadIdx.x / 8, col = (blockIdx.x * 8 + x) * 4;
    const float *p = part + static_cast<int64_t>(blockIdx.y) * groups * d + col;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < d) {
#pragma unroll 8
        for (int g = y; g < groups; g += 32) {
            const float4 v = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(g) * d);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    red[y][x] = s;
    __syncthreads();
    if (y < 4 && col < d) {   // thread y of the quad takes its column y
        const float *c = &red[0][x].x + y;
        float v = 0.f;
        for (int k = 0; k < 32; ++k) v += c[k * 32];
        out[col + y] = static_cast<T>(v);
    }
}

}  // namespace lce
