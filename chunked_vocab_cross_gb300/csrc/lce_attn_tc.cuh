// What the tensor-core attention kernels share: tiles of 128 tokens in
// 128-byte-swizzled shared memory, bounded waits, MMA issue.
//
// A tile is NB column blocks (64 channels, 128 bytes a token) of 128 rows,
// 16 KB each. Read along the channels (scores: A and B K-major) a K step of 16
// channels is 32 bytes; read along the tokens (sums over tokens: B MN-major,
// N = channels) a K step of 16 tokens is 2 KB and the next 64 channels are one
// block, 16 KB, on. Channels past D arrive as zeros from the tensor map, so
// any D runs as if rounded up to 16.
#pragma once

#include "f32x2.cuh"
#include "lce_attn.cuh"
#include "tc_ptx.cuh"

namespace lce {

constexpr int kTcTile = 128;
constexpr int kTcBlock = kTcTile * 128;                 // bytes of one column block
constexpr long long kTcWaitCycles = 2000000000LL;       // ~1 s: far above any legitimate wait
constexpr long long kTcDrainCycles = 200000000LL;

// Polls a barrier phase without a suspend-time hint: the softmax and MMA warps
// hand each other every tile, and a waiter that sleeps longer than the hardware's
// own short limit adds to that chain.
__device__ __forceinline__ bool tc_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits of one CTA: a wait that gives up raises the device status word and
// the CTA's abort flag, on which all its other waits give up too.
struct TcWaits {
    volatile int *abort_flag;
    int *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        const uint32_t a = smem_u32(bar);
        if (tc_try_wait(a, parity)) return true;
        const long long t0 = clock64();
        for (;;) {
            if (tc_try_wait(a, parity)) return true;
            if (*abort_flag) return false;
            if (clock64() - t0 > kTcWaitCycles) {
                *abort_flag = 1;
                atomicOr(status, kDevTimeout);
                return false;
            }
        }
    }
    // the same answer for all lanes of the warp
    __device__ __forceinline__ bool all(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

// Used only while shutting down: lets what is in flight land before the CTA
// gives up its memory.
__device__ __forceinline__ void tc_drain(uint64_t *bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    const long long t0 = clock64();
    while (!tc_try_wait(a, parity))
        if (clock64() - t0 > kTcDrainCycles) return;
}

// One tile: 128 tokens of one head from token `tok` on. Tokens past the
// tensor's end arrive as zeros; those of the next sequence as they are.
template <int NB>
__device__ __forceinline__ void tc_load_tile(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int head, int tok) {
#pragma unroll
    for (int b = 0; b < NB; ++b) tma_load_3d(dst + b * kTcBlock, m, bar, b * 64, head, tok);
}

// Zeroes the rows from `rows` on of a loaded tile that is summed over its
// tokens: 0 * NaN of a token beyond the sequence would reach every result.
// Called by one whole warp between the load's arrival and the MMAs.
template <int NB>
__device__ __forceinline__ void tc_zero_rows(uint8_t *tile, int rows) {
    const int lane = threadIdx.x & 31;
    const int n = (kTcTile - rows) * 8;
#pragma unroll
    for (int b = 0; b < NB; ++b)
        for (int i = lane; i < n; i += 32)
            *reinterpret_cast<uint4 *>(tile + b * kTcBlock + rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// Descriptors of a tile read along its channels / along its tokens.
__device__ __forceinline__ uint64_t tc_desc_k(const uint8_t *tile) { return sdesc_sw128(smem_u32(tile), 0, 1024); }
__device__ __forceinline__ uint64_t tc_desc_mn(const uint8_t *tile) {
    return sdesc_sw128(smem_u32(tile), kTcBlock, 1024);
}
// Offset of K step kk in descriptor units (16 bytes): along the channels, four steps a block.
__device__ __forceinline__ uint64_t tc_step_k(int kk) { return (kk >> 2) * (kTcBlock >> 4) + (kk & 3) * 2; }
__device__ __forceinline__ uint64_t tc_step_mn(int kk) { return kk * 128; }

// The kernels are compiled for KS steps of 16 channels (D rounded up), in NB
// blocks of 64.
template <int KS>
struct Chan {
    static constexpr int NB = (KS + 3) / 4;
    static constexpr int kTile = NB * kTcBlock;
};

// D = A . B^T over the channels (both operands tiles). Unrolled: one thread
// issues, and the address arithmetic of a rolled loop takes it longer than the
// MMA takes the tensor core.
template <int KS>
__device__ __forceinline__ void tc_mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) umma_f16(d, a + tc_step_k(kk), b + tc_step_k(kk), idesc, kk > 0);
}
// D (+)= P . B over tokens: P in tensor memory (two tokens a column), the
// shares of the two threads of a row (64 tokens) 64 columns apart; B a tile.
// The first (kChunk = 0) or the second 32 tokens of each share.
template <int kChunk>
__device__ __forceinline__ void tc_mma_tokens_chunk(uint32_t d, uint32_t p, uint64_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int kk = (i >> 1) * 4 + kChunk * 2 + (i & 1);
        umma_f16_ts(d, p + (kk >> 2) * 64 + (kk & 3) * 8, b + tc_step_mn(kk), idesc, accumulate || i > 0);
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

// The 32-channel chunks of an accumulator that a half of its threads takes.
template <int KS>
struct Chunks {
    static constexpr int kAll = (KS + 1) / 2, kFirst = (kAll + 1) / 2;   // of both halves, of the first
};

// 16-byte piece c of row r in a swizzled tile (byte offset).
__device__ __forceinline__ int tc_piece(int r, int c) {
    return (c >> 3) * kTcBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Writes chunks [C0, C0 + N) of a warp's 32 rows of an accumulator to global
// memory as bf16: lane r holds row r0 + r of the tile. The rows go through the
// warp's share of a free tile, so that a store covers whole lines of a few
// rows (stored by each lane on its own, 32 rows at a time, they took 4700
// cycles a tile instead of 700). `release` is called once the accumulator has
// been read.
template <int C0, int N, typename F>
__device__ __forceinline__ void tc_store_rows(uint8_t *tile, uint32_t taddr, float mul, int r0, int rows,
                                              __nv_bfloat16 *dst, int64_t stride, int D, F release) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = C0; c < C0 + N; ++c) {
        uint32_t v[32];
        tmem_ld32(taddr + c * 32, v);
        tmem_ld_wait();
        if (c + 1 == C0 + N) release();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(v[8 * i]) * mul, __uint_as_float(v[8 * i + 1]) * mul);
            w.y = pack_bf16(__uint_as_float(v[8 * i + 2]) * mul, __uint_as_float(v[8 * i + 3]) * mul);
            w.z = pack_bf16(__uint_as_float(v[8 * i + 4]) * mul, __uint_as_float(v[8 * i + 5]) * mul);
            w.w = pack_bf16(__uint_as_float(v[8 * i + 6]) * mul, __uint_as_float(v[8 * i + 7]) * mul);
            *reinterpret_cast<uint4 *>(tile + tc_piece(r0 + lane, c * 4 + i)) = w;
        }
    }
    __syncwarp();
    constexpr int kPer = N * 4;   // pieces of a row
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = k * 32 + lane, r = r0 + i / kPer, c = C0 * 4 + i % kPer;
        if (r < rows && c * 8 < D)
            *reinterpret_cast<uint4 *>(dst + r * stride + c * 8) = *reinterpret_cast<const uint4 *>(tile + tc_piece(r, c));
    }
}

// The same for the chunks of one half of the threads.
template <int KS, typename F>
__device__ __forceinline__ void tc_store_half(int half, uint8_t *tile, uint32_t taddr, float mul, int r0, int rows,
                                              __nv_bfloat16 *dst, int64_t stride, int D, F release) {
    using C = Chunks<KS>;
    if (half == 0) tc_store_rows<0, C::kFirst>(tile, taddr, mul, r0, rows, dst, stride, D, release);
    else tc_store_rows<C::kFirst, C::kAll - C::kFirst>(tile, taddr, mul, r0, rows, dst, stride, D, release);
}

// The same in fp32, 16 channels at a time: each half of the threads has its half
// of the tile's 128-byte rows.
template <int KS, typename F>
__device__ __forceinline__ void tc_store_fp32(int half, uint8_t *tile, uint32_t taddr, float mul, int r0, int rows, float *dst,
                                              int64_t stride, int D, F release) {
    using C = Chunks<KS>;
    const int lane = threadIdx.x & 31;
    const int last = half ? C::kAll : C::kFirst;
#pragma unroll 1
    for (int c = half ? C::kFirst : 0; c < last; ++c) {
        uint32_t v[32];
        tmem_ld32(taddr + c * 32, v);
        tmem_ld_wait();
        if (c + 1 == last) release();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * mul);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(tile + (r0 + lane) * 128 + half * 64 + ((i ^ (lane & 3)) << 4)) =
                    make_uint4(v[h * 16 + 4 * i], v[h * 16 + 4 * i + 1], v[h * 16 + 4 * i + 2], v[h * 16 + 4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + k * 8 + lane / 4, i = lane & 3, col = c * 32 + h * 16 + i * 4;
                if (r < rows && col < D)
                    *reinterpret_cast<uint4 *>(dst + r * stride + col) =
                        *reinterpret_cast<const uint4 *>(tile + r * 128 + half * 64 + ((i ^ (r & 3)) << 4));
            }
            __syncwarp();
        }
    }
}

struct AttnMaps {
    CUtensorMap q, k, v, dO;
};

}  // namespace lce
