// Global gradient norm over many tensors, and clipping by it.
#include <cuda_bf16.h>

#include <algorithm>

#include "lce_host.h"
#include "tc_ptx.cuh"

using namespace lce;

namespace {

// What bounds both passes is HBM: 1.6 GB of bf16 in 20 tensors take 730 us, 4.8 GB at 6.6 TB/s (the squares alone
// 245 us). The second launch begins under the first (60 MB 26.8 -> 26.4 us, the norm alone of 8 MB 6.2 -> 5.6). The
// squares run best in many small blocks (191 us for 1.2 GB; 217 in blocks of 512 threads), the scaling in fewer, since
// each adds up all blocks' sums first (362 us; 371).
constexpr int kSqThreads = 256, kSqBlocksPerSm = 8;
constexpr int kClipThreads = 512;
constexpr int kChunkBytes = 65536;   // bytes of a tensor that a block takes at a time: 16 loads a thread (the scaling: eight)
// Tensors a launch takes: the table travels as a kernel argument (9 KB; a short
// one for short lists made no difference to the host).
constexpr int kTable = 240;
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = 256 * kSqBlocksPerSm;
// Up to 1 MB (each tensor counted in whole 4 KB) one cluster of eight blocks
// does both passes in one launch: a warp has one chunk of 4 KB and keeps it in
// registers, and the blocks' sums are joined through distributed shared memory.
// What bounds it is latency (0.1 MB in 20 tensors: 4.3 us, 5.7 with the two
// launches; 0.84 MB in 28: 6.5 us, 7.9; and one launch less for the host).
constexpr int kCluster = 8, kClusterThreads = 1024;
constexpr int kClusterChunks = kCluster * kClusterThreads / 32;
constexpr int kSmallChunkBytes = 4096;

struct ClipEntry {
    const void *g;
    void *out;
    int64_t n;
    int fp32;
};
struct ClipTable {
    int count, chunks;
    int first[kTable];   // number of a tensor's first chunk within the launch; apart from the rest, since it is searched
    ClipEntry t[kTable];
};

__device__ __forceinline__ int entry_of(const ClipTable &tab, int chunk) {
    int lo = 0, hi = tab.count;   // the last entry with first <= chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (tab.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A chunk of a tensor: elements [begin, end), of which [vb, ve) can be taken 16
// bytes at a time. Chunks are cut at multiples of their size from the 16-byte
// boundary at or before the tensor's start, so only its ends are ragged.
struct Span {
    int64_t begin, end, vb, ve;
};
template <typename T, int kBytes>
__device__ __forceinline__ Span span_of(const ClipEntry &e, int chunk) {
    constexpr int kPer = kBytes / sizeof(T), kV = 16 / sizeof(T);
    const int64_t lead = (reinterpret_cast<uintptr_t>(e.g) % 16) / sizeof(T);   // elements past a 16-byte boundary
    Span s;
    s.begin = static_cast<int64_t>(chunk) * kPer - lead;
    s.end = min(s.begin + kPer, e.n);
    s.vb = max(s.begin, int64_t(0));
    if (s.begin < 0 && lead) s.vb = kV - lead;
    s.begin = max(s.begin, int64_t(0));
    s.vb = min(s.vb, s.end);
    s.ve = s.vb + (s.end - s.vb) / kV * kV;
    return s;
}

__device__ __forceinline__ float f32(float x) { return x; }
__device__ __forceinline__ float f32(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float squares(const float4 &v, float s) {
    return fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, s))));
}
__device__ __forceinline__ float squares16(const uint4 &v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
        s = fmaf(a, a, fmaf(b, b, s));
    }
    return s;
}

// each thread takes its share of a span
template <typename T>
__device__ __forceinline__ float span_squares(const ClipEntry &e, const Span &sp) {
    const T *g = static_cast<const T *>(e.g);
    constexpr int kV = 16 / sizeof(T), nt = kSqThreads;
    const int t = threadIdx.x;
    float s = 0.f;
    for (int64_t i = sp.begin + t; i < sp.vb; i += nt) s = fmaf(f32(g[i]), f32(g[i]), s);
    for (int64_t i = sp.vb + t * kV; i < sp.ve; i += nt * kV) {
        if (sizeof(T) == 4) s = squares(*reinterpret_cast<const float4 *>(g + i), s);
        else s = squares16(*reinterpret_cast<const uint4 *>(g + i), s);
    }
    for (int64_t i = sp.ve + t; i < sp.end; i += nt) s = fmaf(f32(g[i]), f32(g[i]), s);
    return s;
}

// The same share in fp64, for squares whose sum overflows fp32 (values from about 1e18 on). A function of its own, so
// that the common case keeps its registers.
__device__ __forceinline__ double square64(float x) { return static_cast<double>(x) * x; }
template <typename T>
__device__ __noinline__ double span_squares64(const T *g, int64_t begin, int64_t vb, int64_t ve, int64_t end) {
    constexpr int kV = 16 / sizeof(T), nt = kSqThreads;
    const int t = threadIdx.x;
    double s = 0.0;
    for (int64_t i = begin + t; i < vb; i += nt) s += square64(f32(g[i]));
    for (int64_t i = vb + t * kV; i < ve; i += nt * kV)
        for (int k = 0; k < kV; ++k) s += square64(f32(g[i + k]));
    for (int64_t i = ve + t; i < end; i += nt) s += square64(f32(g[i]));
    return s;
}
template <typename T>
__device__ __forceinline__ double span_sum(const ClipEntry &e, const Span &sp) {
    const float s = span_squares<T>(e, sp);
    return isinf(s) ? span_squares64(static_cast<const T *>(e.g), sp.begin, sp.vb, sp.ve, sp.end) : s;
}

// Sum over the block, the same for all threads, in a fixed order. A warp's fp64
// addition takes 16 cycles of an SM, so one warp joins the warps' sums for all
// (done by every thread, they were half of a short call).
template <int kThreads>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[kThreads / 32], total;
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kThreads / 32 ? red[threadIdx.x] : 0.0;
        for (int m = kThreads / 64; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (threadIdx.x == 0) total = v;
    }
    __syncthreads();
    return total;
}

// part[block] = sum of the squares of the block's chunks: fp32 along a thread's
// elements of one chunk (at most 66 of fp32, 130 of bf16) while they fit it,
// fp64 across chunks and threads.
__global__ void __launch_bounds__(kSqThreads) k_clip_squares(const __grid_constant__ ClipTable tab, double *part) {
    double s = 0.0;
    for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
        const int i = entry_of(tab, c), k = c - tab.first[i];
        const ClipEntry &e = tab.t[i];
        s += e.fp32 ? span_sum<float>(e, span_of<float, kChunkBytes>(e, k))
                    : span_sum<__nv_bfloat16>(e, span_of<__nv_bfloat16, kChunkBytes>(e, k));
    }
    s = block_sum<kSqThreads>(s);
    griddep_launch_dependents();
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm from the blocks' sums, by one warp for the block.
__device__ __forceinline__ float norm_of(const double *part, int n) {
    __shared__ float norm;
    griddep_wait();   // launched early
    if (threadIdx.x < 32) {
        double s[4] = {0.0, 0.0, 0.0, 0.0};
        for (int i = threadIdx.x; i < n; i += 128)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * 32 < n) s[k] += part[i + k * 32];
        double v = (s[0] + s[1]) + (s[2] + s[3]);
        for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (threadIdx.x == 0) norm = static_cast<float>(sqrt(v));
    }
    __syncthreads();
    return norm;
}

__global__ void __launch_bounds__(kClipThreads) k_clip_norm(const double *part, int n, float *norm) {
    const float v = norm_of(part, n);
    if (threadIdx.x == 0) *norm = v;
}

// 16 bytes of T, times c
template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4 &v, float c) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (sizeof(T) == 4) w[k] = __float_as_uint(__uint_as_float(w[k]) * c);
        else {
            __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(w[k] << 16) * c, __uint_as_float(w[k] & 0xffff0000u) * c);
            w[k] = *reinterpret_cast<uint32_t *>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void span_scale(const ClipEntry &e, const Span &sp, float c) {
    const T *g = static_cast<const T *>(e.g);
    T *o = static_cast<T *>(e.out);
    constexpr int kV = 16 / sizeof(T), nt = kClipThreads;
    const int t = threadIdx.x;
    // an output that lies otherwise than its gradient takes single elements
    const bool vec = (reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) % 16 == 0;
    const int64_t vb = vec ? sp.vb : sp.begin, ve = vec ? sp.ve : sp.begin;
    for (int64_t i = sp.begin + t; i < vb; i += nt) o[i] = static_cast<T>(f32(g[i]) * c);
    for (int64_t i = vb + t * kV; i < ve; i += nt * kV)
        __stcs(reinterpret_cast<uint4 *>(o + i), scaled<T>(*reinterpret_cast<const uint4 *>(g + i), c));
    for (int64_t i = ve + t; i < sp.end; i += nt) o[i] = static_cast<T>(f32(g[i]) * c);
}

// Every block adds up the partial sums itself (a few KB, in L2), forms the
// factor and scales its chunks, the last ones first: they are what the squares
// left in L2, and the stores ask to be evicted before them. Chunks stay with
// block numbers equal modulo the grid, whose SMs then have them nearer (120 MB:
// 61 us; 62 counted straight down, 70 first chunks first; 60 MB, all of it in
// L2: 28, 34 and 29; 1.6 GB: 730 any way).
__global__ void __launch_bounds__(kClipThreads) k_clip_scale(const __grid_constant__ ClipTable tab, const double *part,
                                                             int n, float max_norm, float eps, int in_place,
                                                             float *norm, float *factor) {
    const float v = norm_of(part, n);
    float c = max_norm / (v + eps);
    if (c > 1.f) c = 1.f;   // a NaN stays
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *norm = v;
        if (factor) *factor = c;
    }
    if (in_place && c == 1.f) return;
    const int g = gridDim.x, b = blockIdx.x;
    if (b >= tab.chunks) return;
    for (int j = b + (tab.chunks - 1 - b) / g * g; j >= 0; j -= g) {
        const int i = entry_of(tab, j), k = j - tab.first[i];
        const ClipEntry &e = tab.t[i];
        if (e.fp32) span_scale<float>(e, span_of<float, kChunkBytes>(e, k), c);
        else span_scale<__nv_bfloat16>(e, span_of<__nv_bfloat16, kChunkBytes>(e, k), c);
    }
}

// A warp's chunk of a tensor in registers: its 16-byte pieces, eight a lane,
// and the up to seven elements on either side of them, one a lane.
template <typename T>
struct Held {
    static constexpr int kV = 16 / sizeof(T), kPieces = kSmallChunkBytes / 16 / 32;
    Span sp;
    uint4 v[kPieces];
    int64_t at;    // of the single element (-1: none)
    float single;

    __device__ __forceinline__ float load(const ClipEntry &e, int chunk, int lane) {
        const T *g = static_cast<const T *>(e.g);
        sp = span_of<T, kSmallChunkBytes>(e, chunk);
        at = lane < 16 ? sp.begin + lane : sp.ve + lane - 16;
        if (at >= (lane < 16 ? sp.vb : sp.end)) at = -1;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int64_t i = sp.vb + (k * 32 + lane) * kV;
            v[k] = i < sp.ve ? *reinterpret_cast<const uint4 *>(g + i) : make_uint4(0, 0, 0, 0);
        }
        single = at >= 0 ? f32(g[at]) : 0.f;
        float s = single * single;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            if (sizeof(T) == 4) s = squares(*reinterpret_cast<const float4 *>(&v[k]), s);
            else s = squares16(v[k], s);
        }
        return s;
    }
    // the lane's sum of squares in fp64
    __device__ __forceinline__ double squares64() const {
        double s = square64(single);
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const T *x = reinterpret_cast<const T *>(&v[k]);
#pragma unroll
            for (int q = 0; q < kV; ++q) s += square64(f32(x[q]));
        }
        return s;
    }
    __device__ __forceinline__ void store(const ClipEntry &e, float c, int lane) const {
        T *o = static_cast<T *>(e.out);
        const bool vec = (reinterpret_cast<uintptr_t>(e.g) ^ reinterpret_cast<uintptr_t>(o)) % 16 == 0;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int64_t i = sp.vb + (k * 32 + lane) * kV;
            if (i >= sp.ve) continue;
            const uint4 w = scaled<T>(v[k], c);
            if (vec) *reinterpret_cast<uint4 *>(o + i) = w;
            else {
                const T *x = reinterpret_cast<const T *>(&w);
#pragma unroll
                for (int q = 0; q < kV; ++q) o[i + q] = x[q];
            }
        }
        if (at >= 0) o[at] = static_cast<T>(single * c);
    }
};

// Both passes by one cluster: fp32 within a warp's chunk (a lane's 33 or 65
// elements, then the lanes) while the squares fit it, fp64 across the chunks,
// joined in block order by one warp of each block (a warp's fp64
// addition takes 16 cycles of an SM, its square root hundreds: done by every
// warp they were most of the call, 9.9 us for 0.1 MB).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
    k_clip_cluster(const __grid_constant__ ClipTable tab, int clip, float max_norm, float eps, int in_place, float *norm,
                   float *factor) {
    __shared__ double red[kClusterThreads / 32], mine;
    __shared__ float f;
    const int rank = static_cast<int>(cluster_ctarank()), warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int c0 = rank + warp * kCluster;   // neighbouring chunks to different SMs
    const bool any = c0 < tab.chunks;
    const int i = any ? entry_of(tab, c0) : 0, k = any ? c0 - tab.first[i] : 0;
    const ClipEntry &e = tab.t[i];
    Held<float> hf;
    Held<__nv_bfloat16> hb;
    float s = 0.f;
    if (any) s = e.fp32 ? hf.load(e, k, lane) : hb.load(e, k, lane);
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    double chunk = s;
    if (isinf(s)) {   // for every lane of the warp: they all have the same sum
        chunk = e.fp32 ? hf.squares64() : hb.squares64();
        for (int m = 16; m; m >>= 1) chunk += __shfl_xor_sync(0xffffffffu, chunk, m);
    }
    if (lane == 0) red[warp] = chunk;
    __syncthreads();
    if (warp == 0) {
        double v = red[lane];
        for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (lane == 0) mine = v;
    }
    cluster_sync_all();
    if (warp == 0) {
        double v = 0.0;
        if (lane < kCluster)
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(map_to_cta(smem_u32(&mine), lane)) : "memory");
        for (int m = kCluster / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (lane == 0) {
            const float n = static_cast<float>(sqrt(v));
            float c = max_norm / (n + eps);
            if (c > 1.f) c = 1.f;   // a NaN stays
            f = c;
            if (rank == 0) {
                *norm = n;
                if (factor) *factor = c;
            }
        }
    }
    cluster_sync_all();   // the factor is there, and nobody's sum goes away while another reads it
    const float c = f;
    if (!any || !clip || (in_place && c == 1.f)) return;
    if (e.fp32) hf.store(e, c, lane);
    else hb.store(e, c, lane);
}

lce_status_t check_clip(int64_t count, const void *const *grads, void *const *outs, const int64_t *sizes,
                        const int32_t *dtypes, const float *norm) {
    if (count < 0 || count >= (int64_t(1) << 24)) return LCE_ERR_SHAPE;
    if (!norm || (count > 0 && (!grads || !sizes || !dtypes))) return LCE_ERR_NULL;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != LCE_BF16 && dtypes[i] != LCE_FP32) return LCE_ERR_DTYPE;
        if (sizes[i] < 0 || sizes[i] >= (int64_t(1) << 40)) return LCE_ERR_SHAPE;
        if (sizes[i] == 0) continue;
        if (!grads[i] || (outs && !outs[i])) return LCE_ERR_NULL;
        const uintptr_t elt = dtypes[i] == LCE_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(grads[i]) % elt || (outs && reinterpret_cast<uintptr_t>(outs[i]) % elt))
            return LCE_ERR_ALIGN;
    }
    return LCE_OK;
}

// The tensors from `*at` on that fit one launch.
template <int kBytes>
void fill_table(ClipTable &tab, int64_t *at, int64_t count, const void *const *grads, void *const *outs,
                const int64_t *sizes, const int32_t *dtypes) {
    tab.count = tab.chunks = 0;
    for (; *at < count && tab.count < kTable; ++*at) {
        const int64_t i = *at;
        if (sizes[i] == 0) continue;
        const int elt = dtypes[i] == LCE_BF16 ? 2 : 4;
        const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(grads[i]) % 16);
        const int64_t chunks = (sizes[i] * elt + lead + kBytes - 1) / kBytes;
        if (tab.count && tab.chunks + chunks >= (int64_t(1) << 30)) break;
        tab.first[tab.count] = tab.chunks;
        tab.t[tab.count++] = ClipEntry{grads[i], outs ? outs[i] : const_cast<void *>(grads[i]), sizes[i],
                                       dtypes[i] == LCE_FP32};
        tab.chunks += static_cast<int>(chunks);
    }
}

struct ClipCall {
    int64_t count;
    const void *const *grads;
    void *const *outs;
    const int64_t *sizes;
    const int32_t *dtypes;
    bool clip;
    float max_norm, eps;
    float *norm, *factor;
};

// Small chunks of all tensors together (as fill_table cuts them).
int64_t count_chunks(const ClipCall &a) {
    int64_t n = 0;
    for (int64_t i = 0; i < a.count; ++i) {
        if (a.sizes[i] == 0) continue;
        const int64_t bytes = a.sizes[i] * (a.dtypes[i] == LCE_BF16 ? 2 : 4) + static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.grads[i]) % 16);
        n += (bytes + kSmallChunkBytes - 1) / kSmallChunkBytes;
    }
    return n;
}

lce_status_t launch_small(const ClipCall &a, cudaStream_t st) {
    ClipTable tab;
    int64_t at = 0;
    fill_table<kSmallChunkBytes>(tab, &at, a.count, a.grads, a.outs, a.sizes, a.dtypes);
    k_clip_cluster<<<kCluster, kClusterThreads, 0, st>>>(tab, a.clip, a.max_norm, a.eps, a.outs == nullptr, a.norm, a.factor);
    return host_launched();
}

lce_status_t launch_clip(const ClipCall &a, const HostDev &dev, double *part, cudaStream_t st) {
    lce_status_t s;
    ClipTable tab;
    int n = 0;
    const int most = dev.sms * kSqBlocksPerSm < kMaxBlocks ? dev.sms * kSqBlocksPerSm : kMaxBlocks;
    for (int64_t at = 0; at < a.count;) {
        fill_table<kChunkBytes>(tab, &at, a.count, a.grads, a.outs, a.sizes, a.dtypes);
        if (!tab.count) break;
        const int blocks = tab.chunks < most ? tab.chunks : most;
        k_clip_squares<<<blocks, kSqThreads, 0, st>>>(tab, part + n);
        if ((s = host_launched()) != LCE_OK) return s;
        n += blocks;
    }
    if (!a.clip) {
        return host_launch_early(k_clip_norm, dim3(1), kClipThreads, 0, st, part, n, a.norm);
    }
    bool done = false;
    for (int64_t at = 0; at < a.count || !done;) {
        fill_table<kChunkBytes>(tab, &at, a.count, a.grads, a.outs, a.sizes, a.dtypes);
        if (!tab.count && done) break;
        const int blocks = std::max(1, std::min(tab.chunks, dev.sms * kBlocksPerSm));
        s = host_launch_early(k_clip_scale, dim3(blocks), kClipThreads, 0, st, tab, part, n, a.max_norm, a.eps, a.outs == nullptr, a.norm, a.factor);
        if (s != LCE_OK) return s;
        done = true;
    }
    return LCE_OK;
}

lce_status_t run_clip(const ClipCall &a, void *workspace, size_t workspace_bytes, lce_stream_t stream) {
    lce_status_t s = check_clip(a.count, a.grads, a.outs, a.sizes, a.dtypes, a.norm);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (workspace && workspace_bytes < lce_clip_workspace_size(a.count)) return LCE_ERR_WORKSPACE;
    if (a.count <= kTable && count_chunks(a) <= kClusterChunks)
        return launch_small(a, st);
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    if ((s = scratch.get(workspace, workspace_bytes, lce_clip_workspace_size(a.count), &base)) != LCE_OK) return s;
    double *part = reinterpret_cast<double *>(base);
    return launch_clip(a, dev, part, st);
}

}  // namespace

extern "C" {

size_t lce_clip_workspace_size(int64_t count) {
    if (count < 0 || count >= (int64_t(1) << 24)) return 0;
    return static_cast<size_t>((count + kTable - 1) / kTable + 1) * kMaxBlocks * sizeof(double);
}

lce_status_t lce_grad_norm(int64_t count, const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                           float *norm, void *workspace, size_t workspace_bytes, lce_stream_t stream) {
    return run_clip({count, grads, nullptr, sizes, dtypes, false, 0.f, 0.f, norm, nullptr}, workspace, workspace_bytes, stream);
}

lce_status_t lce_clip_grads(int64_t count, const void *const *grads, void *const *outs, const int64_t *sizes,
                            const int32_t *dtypes, float max_norm, float eps, float *norm, float *factor,
                            void *workspace, size_t workspace_bytes, lce_stream_t stream) {
    if (!(max_norm >= 0.f) || !(eps >= 0.f)) return LCE_ERR_ARG;
    return run_clip({count, grads, outs, sizes, dtypes, true, max_norm, eps, norm, factor}, workspace, workspace_bytes, stream);
}

}  // extern "C"
