// The gradient of a weight from packed activations, dw = dy^T x, on the tensor
// cores: x is widened from its codes on the way.
//
// CTA pairs (clusters of two) take 256 x 256 tiles of dw, K being the tokens, 64
// at a time. Both operands lie token-major in memory, which is MN-major for this
// product. dy comes by TMA straight into the layout the MMA reads; the codes of
// the CTA's 128 channels, and their one exponent a token (128 channels are a
// block of the format), come by TMA into a ring of their own, from which eight
// warps write the bf16 operand into a third ring. A code's bits, moved to where a
// bf16 has them, are its value times 2^-120, and a product with a power of two
// brings it to scale without a rounding (two products where the scale is above
// 2^7): three integer operations and a product for two codes. The rings are
// apart, since each has a latency of its own to hide. The other warps: 0 asks for
// dy and 2 for codes, 1 issues the MMAs (of both CTAs, in the even one), 4 to 7
// bring a finished accumulator to memory while the next one fills.
//
// What bounds it is the tensor core under the power cap: 7373 tokens, 16384 x
// 4096 bf16, 556 to 650 us with the box and the values (1520 to 1780 TFLOP/s;
// cuBLAS on plain bf16 1730 sustained, 1930 in a burst). An fp32 dw is bound by
// the sums of its runs in memory, 16 bytes of 32 rows at a time: 1502 us, and
// 220 where bf16 takes 96 (4096 tokens, 4096 x 4096). Measured on the way:
// one ring for dy and codes and eight warps that widen every step together 1780
// us; in groups that take steps in turn 1024; arrivals of cluster scope on the
// even CTA's barrier (1800 cycles each) 824, of CTA scope 594; codes and widened
// stages in multiples of the groups, two warps a group instead of four 564.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "e4m3.cuh"
#include "lce.h"
#include "tc_ptx.cuh"

namespace lce {

constexpr int kWgTile = 256, kWgHalf = 128, kWgK = 64;   // of a pair, of a CTA; tokens a step
constexpr int kWgDy = 6, kWgCodes = 8, kWgWide = 4;      // stages of dy, of codes, of widened codes
constexpr int kWgGroups = 4, kWgEach = 2;                // groups of warps that widen a step each in turn, and their warps
constexpr int kWgFirst = 8, kWgThreads = (kWgFirst + kWgGroups * kWgEach) * 32;   // the first of these warps
constexpr int kWgABytes = kWgHalf * kWgK * 2, kWgCodeBytes = kWgHalf * kWgK, kWgBlockBytes = kWgK * 128;
constexpr int kWgSmem = kWgDy * kWgABytes + kWgCodes * kWgCodeBytes + kWgWide * kWgABytes + 1024;
// A wait on a barrier tells phases apart by their parity alone: a step's stage of codes is always its group's own, and a
// group is never two rounds of the widened stages ahead of the MMAs.
static_assert(kWgCodes % kWgGroups == 0 && kWgWide >= kWgGroups, "");
constexpr long long kWgWaitCycles = 2000000000LL;   // ~1 s: far above any legitimate wait

struct WgMaps {
    CUtensorMap dy[3], codes;   // dy: itself, or the parts of an fp32 one
};
struct WgArgs {
    const int8_t *exps;
    int64_t ld_exps;
    void *out;        // dw, or the fp32 sums of the splits, one after the other
    int T, n, k;
    int parts;        // of dy
    int whole;        // n is a multiple of 64: dy has a three-dimensional map
    int mt, nt;       // tiles along n and k
    int steps, per;   // of 64 tokens; of a split
    int run;          // steps that an accumulator takes; the runs of a unit are added up in fp32 in memory (a bf16 out has one)
    int splits;
    int *status;
};

struct WgBars {
    uint64_t full_a[kWgDy], empty_a[kWgDy], full_c[kWgCodes], empty_c[kWgCodes], full_b[kWgWide], empty_b[kWgWide], full_t[2], empty_t[2], done;
    uint32_t tmem;
    volatile int abort;
    __align__(16) int8_t exps[kWgCodes][kWgK];
};

__device__ __forceinline__ bool wg_wait(uint64_t *bar, uint32_t parity, WgBars &sm, int *status) {
    const uint32_t at = smem_u32(bar);
    if (mbar_try_wait(at, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(at, parity)) {
        if (sm.abort) return false;
        if (clock64() - t0 > kWgWaitCycles) {
            sm.abort = 1;
            atomicOr(status, LCE_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void wg_drain(uint64_t *bar, uint32_t parity) {   // while leaving after a wait that gave up
    const long long t0 = clock64();
    while (!mbar_try_wait(smem_u32(bar), parity) && clock64() - t0 < kWgWaitCycles / 10) {}
}

// A unit of work: a tile and its range of steps. Tiles go by groups of eight
// along n, so that those in flight together share what they read of both sides.
struct WgUnit {
    int m, n, split, k0, k1;
};
__device__ __forceinline__ WgUnit wg_unit(const WgArgs &a, int u) {
    WgUnit r;
    r.split = u % a.splits;
    const int tile = u / a.splits, group = tile / (8 * a.nt), in = tile - group * 8 * a.nt, rows = min(8, a.mt - group * 8);
    r.n = in / rows, r.m = group * 8 + in - r.n * rows;
    r.k0 = r.split * a.per, r.k1 = min(a.steps, r.k0 + a.per);
    return r;
}

// Arrives on a barrier of either CTA. What the pair's MMAs read for it lies in the
// arriving CTA's own shared memory, and a fence has handed it to the async proxy,
// which reads it there: no release beyond the CTA is wanted.
__device__ __forceinline__ void wg_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two bytes of a word, extended by their signs to 16 bits
template <uint32_t kSelect>
__device__ __forceinline__ uint32_t wg_extend(uint32_t codes) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(codes), "n"(kSelect));
    return r;
}
// Four codes to two bf16 pairs, times a power of two (a pair as well) or two:
// a code is extended to 16 bits by its sign, moved up by 4 bits and cleared
// between sign and exponent. A NaN's code comes out as 480: lce_pack8 leaves
// them only in blocks whose exponent makes NaNs of all codes (looking for them
// here takes 600 us where the product takes 568).
template <bool kTwo>
__device__ __forceinline__ uint2 wg_widen(uint32_t codes, uint32_t s1, uint32_t s2) {
    const uint32_t lo = wg_extend<0x9180>(codes), hi = wg_extend<0xb3a2>(codes);
    uint32_t a = mul_bf16x2(lo * 16 & 0x87f087f0u, s1), b = mul_bf16x2(hi * 16 & 0x87f087f0u, s1);
    if (kTwo) a = mul_bf16x2(a, s2), b = mul_bf16x2(b, s2);
    return make_uint2(a, b);
}

template <typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgThreads, 1) k_wgrad(const __grid_constant__ WgMaps maps, const WgArgs a) {
    constexpr uint32_t kIdesc = idesc_f32acc(1, kWgTile, kWgTile, true, true);
    extern __shared__ uint8_t smem_raw[];
    __shared__ WgBars sm;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *wide = smem + kWgDy * kWgABytes, *codes = wide + kWgWide * kWgABytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, units = a.mt * a.nt * a.splits;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWgDy; ++i) mbar_init(&sm.full_a[i], 1), mbar_init(&sm.empty_a[i], 1);
        for (int i = 0; i < kWgCodes; ++i) mbar_init(&sm.full_c[i], 1), mbar_init(&sm.empty_c[i], kWgEach);
        for (int i = 0; i < kWgWide; ++i) mbar_init(&sm.full_b[i], 2 * kWgEach), mbar_init(&sm.empty_b[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.full_t[i], 1), mbar_init(&sm.empty_t[i], 8);   // four warps in each CTA
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full_even = map_to_cta(smem_u32(sm.full_a), 0);
            int it = 0;
            for (int u = pair; ok && u < units; u += pairs) {
                const WgUnit w = wg_unit(a, u);
                const int n0 = w.m * kWgTile + rank * kWgHalf;
                for (int k = w.k0; ok && k < w.k1; k += a.run)
                  for (int part = a.parts - 1; ok && part >= 0; --part)   // the small parts first
                    for (int step = k; step < min(k + a.run, w.k1); ++step, ++it) {
                        const int st = it % kWgDy, t0 = step * kWgK;
                        if (!(ok = wg_wait(&sm.empty_a[st], it / kWgDy & 1 ^ 1, sm, a.status))) break;
                        if (rank == 0) mbar_arrive_expect_tx(&sm.full_a[st], 2 * kWgABytes);
                        uint8_t *dst = smem + st * kWgABytes;
                        if (a.whole) tma_load_3d_pair(dst, &maps.dy[part], full_even + st * 8, 0, t0, n0 / 64);
                        else {
                            tma_load_2d_pair(dst, &maps.dy[part], full_even + st * 8, n0, t0);
                            tma_load_2d_pair(dst + kWgBlockBytes, &maps.dy[part], full_even + st * 8, n0 + 64, t0);
                        }
                    }
            }
            // copies in flight have to land before the pair leaves (in the normal course all have)
            for (int i = max(0, it - kWgDy); !ok && rank == 0 && i < it; ++i) wg_drain(&sm.full_a[i % kWgDy], i / kWgDy & 1);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            const int blocks = (a.k + kPackBlock - 1) / kPackBlock;
            int it = 0;
            for (int u = pair; ok && u < units; u += pairs) {
                const WgUnit w = wg_unit(a, u);
                const int k0 = w.n * kWgTile + rank * kWgHalf, block = k0 / kPackBlock;
                for (int k = w.k0; ok && k < w.k1; k += a.run)
                  for (int part = 0; ok && part < a.parts; ++part)
                    for (int step = k; step < min(k + a.run, w.k1); ++step, ++it) {
                        const int st = it % kWgCodes, t0 = step * kWgK;
                        if (!(ok = wg_wait(&sm.empty_c[st], it / kWgCodes & 1 ^ 1, sm, a.status))) break;
                        const uint32_t bytes = block < blocks ? min(kWgK, (a.T - t0 + 15) & ~15) : 0;   // rows of exps are of whole 16 bytes
                        mbar_arrive_expect_tx(&sm.full_c[st], kWgCodeBytes + bytes);
                        tma_load_2d(codes + st * kWgCodeBytes, &maps.codes, &sm.full_c[st], k0, t0);
                        if (bytes) bulk_load(sm.exps[st], a.exps + block * a.ld_exps + t0, bytes, &sm.full_c[st]);
                    }
            }
            for (int i = max(0, it - kWgCodes); !ok && i < it; ++i) wg_drain(&sm.full_c[i % kWgCodes], i / kWgCodes & 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool issue = elect_one();
            int it = 0, tile = 0;
            for (int u = pair; ok && u < units; u += pairs) {
                const WgUnit w = wg_unit(a, u);
                for (int k = w.k0; ok && k < w.k1; k += a.run, ++tile) {
                    const int acc = tile & 1, steps = (min(k + a.run, w.k1) - k) * a.parts;
                    ok = __all_sync(0xffffffffu, wg_wait(&sm.empty_t[acc], tile >> 1 & 1 ^ 1, sm, a.status));
                    if (!ok) break;
                    tc_fence_after();
                    for (int i = 0; i < steps; ++i, ++it) {
                        const int st = it % kWgDy, sb = it % kWgWide;
                        ok = wg_wait(&sm.full_a[st], it / kWgDy & 1, sm, a.status) && wg_wait(&sm.full_b[sb], it / kWgWide & 1, sm, a.status);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        if (issue) {
                            const uint32_t pa = smem_u32(smem + st * kWgABytes), pb = smem_u32(wide + sb * kWgABytes);
#pragma unroll
                            for (int kk = 0; kk < kWgK / 16; ++kk)
                                umma_f16_pair(tmem + acc * kWgTile, sdesc_sw128(pa + kk * 2048, kWgBlockBytes, 1024),
                                              sdesc_sw128(pb + kk * 2048, kWgBlockBytes, 1024), kIdesc, (i | kk) != 0);
                            umma_commit_pair_mc(&sm.empty_a[st], 3);
                            umma_commit_pair_mc(&sm.empty_b[sb], 3);
                        }
                        __syncwarp();
                    }
                    if (ok && issue) umma_commit_pair_mc(&sm.full_t[acc], 3);
                }
            }
            if (issue) {
                umma_commit_pair_mc(&sm.done, 1);
                wg_drain(&sm.done, 0);
            }
        }
    } else if (warp >= 4 && warp < kWgFirst) {
        const uint32_t empty_even = map_to_cta(smem_u32(sm.empty_t), 0);
        const int quarter = warp & 3;
        int tile = 0;
        for (int u = pair; ok && u < units; u += pairs) {
            const WgUnit w = wg_unit(a, u);
            const int row = w.m * kWgTile + rank * kWgHalf + quarter * 32 + lane, col0 = w.n * kWgTile;
            O *out = static_cast<O *>(a.out) + (static_cast<int64_t>(w.split) * a.n + row) * a.k + col0;
            for (int k = w.k0; k < w.k1; k += a.run, ++tile) {
                const int acc = tile & 1;
                ok = __all_sync(0xffffffffu, wg_wait(&sm.full_t[acc], tile >> 1 & 1, sm, a.status));
                if (!ok) break;
                tc_fence_after();
                for (int c = 0; c < kWgTile && col0 + c < a.k; c += 32) {
                    uint32_t v[32];
                    float4 sum[sizeof(O) == 2 ? 1 : 8];   // of the runs before, in flight together
                    if constexpr (sizeof(O) == 4) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            sum[i / 4] = k > w.k0 && row < a.n && col0 + c + i < a.k ? *reinterpret_cast<const float4 *>(out + c + i) : float4{};
                    }
                    tmem_ld32(tmem + acc * kWgTile + c + (static_cast<uint32_t>(quarter * 32) << 16), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (row >= a.n || col0 + c + i >= a.k) continue;   // (k is a multiple of 8)
                        if constexpr (sizeof(O) == 2) {
                            uint4 x;
                            uint32_t *p = &x.x;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[i + 2 * j]), __uint_as_float(v[i + 2 * j + 1]));
                                p[j] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            *reinterpret_cast<uint4 *>(out + c + i) = x;
                        } else {
#pragma unroll
                            for (int j = i; j < i + 8; j += 4)
                                *reinterpret_cast<float4 *>(out + c + j) =
                                    make_float4(sum[j / 4].x + __uint_as_float(v[j]), sum[j / 4].y + __uint_as_float(v[j + 1]),
                                                sum[j / 4].z + __uint_as_float(v[j + 2]), sum[j / 4].w + __uint_as_float(v[j + 3]));
                        }
                    }
                    __syncwarp();   // the next load is the whole warp's
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(empty_even + acc * 8);
            }
        }
    } else if (warp >= kWgFirst) {
        // The groups take steps in turn: each has the time of four for one, which hides the waits, the fence and the way to
        // the even CTA. 16 codes a lane and turn, 8 lanes a token, 16 tokens a warp.
        constexpr int kTurns = kWgK / kWgEach / 4;
        const uint32_t full_even = map_to_cta(smem_u32(sm.full_b), 0);
        const int group = (warp - kWgFirst) / kWgEach, row = (warp - kWgFirst) % kWgEach * (kWgK / kWgEach) + lane / 8, chunk = lane & 7;
        // The token's line, its 16-byte pieces in the order of the 128-byte swizzle. The lanes of one half of the channels
        // take their second piece first, so that eight lanes together use all banks.
        const int piece = (chunk & 3) * 2, swap = chunk >> 2;
        const int to1[2] = {swap * kWgBlockBytes + row * 128 + (((piece + swap) ^ (row & 7)) << 4),
                            swap * kWgBlockBytes + row * 128 + (((piece + swap) ^ (row & 7) ^ 4) << 4)};   // of even and odd turns
        int it = 0;
        for (int u = pair; ok && u < units; u += pairs) {
            const WgUnit w = wg_unit(a, u);
            for (int k = w.k0; ok && k < w.k1; k += a.run)
              for (int part = 0; ok && part < a.parts; ++part)
                for (int step = k; step < min(k + a.run, w.k1); ++step, ++it) {
                    if (it % kWgGroups != group) continue;
                    const int st = it % kWgCodes, sb = it % kWgWide;
                    ok = __all_sync(0xffffffffu, wg_wait(&sm.full_c[st], it / kWgCodes & 1, sm, a.status));
                    if (!ok) break;
                    const uint8_t *from = codes + st * kWgCodeBytes + row * 128 + chunk * 16;
                    uint2 first[kTurns], second[kTurns];
                    int e[kTurns];
                    bool rare = (step + 1) * kWgK > a.T;   // behind the last token the exponents are whatever lies there
#pragma unroll
                    for (int j = 0; j < kTurns; ++j) {
                        first[j] = *reinterpret_cast<const uint2 *>(from + j * 512 + swap * 8);
                        second[j] = *reinterpret_cast<const uint2 *>(from + j * 512 + 8 - swap * 8);
                        e[j] = sm.exps[st][row + j * 4];
                        rare |= e[j] > 7 || e[j] == kPackNaN;
                    }
                    rare = __any_sync(0xffffffffu, rare);
                    ok = __all_sync(0xffffffffu, wg_wait(&sm.empty_b[sb], it / kWgWide & 1 ^ 1, sm, a.status));
                    if (!ok) break;
                    uint8_t *to = wide + sb * kWgABytes;
                    auto widen = [&](auto two) {
                        constexpr bool kTwo = decltype(two)::value;
#pragma unroll
                        for (int j = 0; j < kTurns; ++j) {
                            // 2^(120 + e), twice, or two such that make it
                            const int s = 120 + e[j], half = kTwo ? s >> 1 : s;
                            uint32_t s1 = static_cast<uint32_t>(half) * 0x00800080u + 0x3f803f80u, s2 = static_cast<uint32_t>(s - half) * 0x00800080u + 0x3f803f80u;
                            if (kTwo && e[j] == kPackNaN) s1 = 0x7fff7fffu;
                            if (kTwo && step * kWgK + row + j * 4 >= a.T) s1 = s2 = 0;
                            uint8_t *line = to + j * 512 + to1[j & 1];
                            const uint2 x0 = wg_widen<kTwo>(first[j].x, s1, s2), x1 = wg_widen<kTwo>(first[j].y, s1, s2);
                            *reinterpret_cast<uint4 *>(line) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                            const uint2 x2 = wg_widen<kTwo>(second[j].x, s1, s2), x3 = wg_widen<kTwo>(second[j].y, s1, s2);
                            *reinterpret_cast<uint4 *>(to + j * 512 + (to1[j & 1] ^ 16)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
                        }
                    };
                    if (rare) widen(std::true_type());
                    else widen(std::false_type());
                    fence_proxy_async_smem();
                    __syncwarp();
                    // The codes' place is given up only now that their widened forms are out. Given up after the loads alone,
                    // an arrival could overtake loads that still waited in the queue behind the other warps' stores to memory.
                    if (lane == 0) mbar_arrive(&sm.empty_c[st]), wg_arrive(full_even + sb * 8);
                }
        }
    }
    // Both CTAs stay until every arrive, commit and copy aimed at either has landed.
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// The splits' sums, in order
template <typename O>
__global__ void __launch_bounds__(256) k_wgrad_join(const float *part, int splits, int64_t count, O *out) {
    griddep_wait();
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (at >= count) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < splits; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(part + i * count + at);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    if constexpr (sizeof(O) == 2) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(s.x, s.y), y = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2 *>(out + at) = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    } else {
        *reinterpret_cast<float4 *>(out + at) = s;
    }
}

// An fp32 dy in three bf16 parts whose sum it is, [part][T][wide], wide being n
// rounded up to 64 and the columns between zero.
__global__ void __launch_bounds__(256) k_wgrad_parts(const float *dy, int64_t ld, int T, int n, int wide, __nv_bfloat16 *out) {
    const int per = wide / 4;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = id / per, size = static_cast<int64_t>(T) * wide;
    const int col = static_cast<int>(id - row * per) * 4;
    if (row >= T) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < n) v = *reinterpret_cast<const float4 *>(dy + row * ld + col);
    float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        __nv_bfloat16 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // finite values beyond bf16's largest are rounded towards zero: to it
            h[i] = fabsf(x[i]) < INFINITY && fabsf(x[i]) > 3.3895313892515355e38f ? __float2bfloat16_rz(x[i]) : __float2bfloat16_rn(x[i]);
            const float f = __bfloat162float(h[i]);
            x[i] = fabsf(f) < INFINITY ? x[i] - f : 0.f;   // what is not finite is in the first part alone
        }
        *reinterpret_cast<uint2 *>(out + p * size + row * wide + col) = *reinterpret_cast<const uint2 *>(h);
    }
}

}  // namespace lce
