// Activations in 8 bits (lce_pack8, lce_unpack8) and the gradient of a weight
// from them (lce_packed_wgrad): kernels and host side.
#include <cuda_bf16.h>

#include <algorithm>

#include "e4m3.cuh"
#include "lce_host.h"
#include "lce_wgrad.cuh"
#include "row_ring.cuh"

using namespace lce;

namespace {

struct PackArgs {
    const void *x;
    void *out;
    uint8_t *codes;
    int8_t *exps;
    int64_t ld, ld_codes, ld_exps, N;
    int d, per;   // per: pieces of 256 channels in a row
};

// A piece is 256 channels of four rows in a row, taken by a warp: their loads
// are in flight together, and their exponents, which lie side by side, go out as
// one word (a byte at a time they are as many writes as a quarter of the codes:
// 16384 x 4096 bf16 to 8 bits 42 us, 34 this way).
constexpr int kRows = 4;

// Every gridDim.x * 8th piece, without a division a piece.
struct Pieces {
    int64_t row, rows;   // first row of the next piece; rows to go on by
    int at, ats, per;    // its place in the row; places to go on by
    __device__ __forceinline__ Pieces(int per_) : per(per_) {
        const int64_t first = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32, step = static_cast<int64_t>(gridDim.x) * 8;
        row = first / per, at = static_cast<int>(first - row * per);
        rows = step / per, ats = static_cast<int>(step - rows * per);
        row *= kRows, rows *= kRows;
    }
    __device__ __forceinline__ void next() {
        row += rows, at += ats;
        if (at >= per) at -= per, row += kRows;
    }
};

// A lane's part of a piece: 16 bytes of bf16 (a block is 16 lanes' values) or
// twice 16 bytes of fp32, a block apart (a block is 32 lanes' values).
template <typename T>
constexpr int kParts = sizeof(T) / 2;
template <typename T>
__device__ __forceinline__ int part_col(int at, int part) {
    return at * 256 + part * kPackBlock + static_cast<int>(threadIdx.x & 31) * kPack<T>;
}

// Bounded by HBM, as is the way back.
template <typename T>
__global__ void __launch_bounds__(256) k_pack8(const PackArgs a) {
    for (Pieces p(a.per); p.row < a.N; p.next()) {
        const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), a.N - p.row));
        uint4 v[kParts<T>][kRows];
#pragma unroll
        for (int h = 0; h < kParts<T>; ++h)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int col = part_col<T>(p.at, h);
                v[h][i] = make_uint4(0, 0, 0, 0);
                if (col < a.d && i < rows) v[h][i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + (p.row + i) * a.ld + col);
            }
#pragma unroll
        for (int h = 0; h < kParts<T>; ++h) {
            const int col = part_col<T>(p.at, h);
            const bool in = col < a.d;
            int e[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const uint32_t words[4] = {v[h][i].x, v[h][i].y, v[h][i].z, v[h][i].w};
                e[i] = pack_exponent(block_top<T, 4, kPackBlock / kPack<T>>(words));
                if (!in || i >= rows) continue;
                f32x2 x[kPack<T> / 2];
                Pack16<T>::get(v[h][i], x);
                const uint2 c = pack_codes<T>(x, pack_scale(e[i]));
                uint8_t *to = a.codes + (p.row + i) * a.ld_codes + col;
                if (sizeof(T) == 2) *reinterpret_cast<uint2 *>(to) = c;
                else *reinterpret_cast<uint32_t *>(to) = c.x;
            }
            if (in && col % kPackBlock == 0) {
                int8_t *to = a.exps + col / kPackBlock * a.ld_exps + p.row;
                if (rows == kRows) *reinterpret_cast<char4 *>(to) = make_char4(e[0], e[1], e[2], e[3]);
                else
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (i < rows) to[i] = static_cast<int8_t>(e[i]);
            }
        }
        __syncwarp();
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_unpack8(const PackArgs a) {
    for (Pieces p(a.per); p.row < a.N; p.next()) {
        const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), a.N - p.row));
        uint2 c[kParts<T>][kRows];
        char4 e[kParts<T>];
#pragma unroll
        for (int h = 0; h < kParts<T>; ++h) {
            const int col = part_col<T>(p.at, h);
            if (col >= a.d) continue;
            e[h] = *reinterpret_cast<const char4 *>(a.exps + col / kPackBlock * a.ld_exps + p.row);   // (rows of exps are of whole 16 bytes)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (i >= rows) continue;
                const uint8_t *from = a.codes + (p.row + i) * a.ld_codes + col;
                if (sizeof(T) == 2) c[h][i] = *reinterpret_cast<const uint2 *>(from);
                else c[h][i].x = *reinterpret_cast<const uint32_t *>(from);
            }
        }
#pragma unroll
        for (int h = 0; h < kParts<T>; ++h) {
            const int col = part_col<T>(p.at, h);
            if (col >= a.d) continue;
            const int exps[kRows] = {e[h].x, e[h].y, e[h].z, e[h].w};
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (i >= rows) continue;
                f32x2 x[kPack<T> / 2];
                pack_values<T>(c[h][i], unpack_scale(exps[i]), x);
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + (p.row + i) * a.ld + col) = Pack16<T>::set(x);
            }
        }
    }
}

lce_status_t check_plain(lce_dtype_t dtype, const void *x, int64_t ld, int64_t N, int64_t d, const void *codes, int64_t ld_codes,
                         const void *exps, int64_t ld_exps, bool out) {
    if (dtype != LCE_BF16 && dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (N < 0 || N >= (int64_t(1) << 31) || d < 8 || d >= (1 << 24)) return LCE_ERR_SHAPE;
    if (d % 8) return LCE_ERR_ALIGN;
    if (N == 0) return LCE_OK;
    if (!x) return LCE_ERR_NULL;
    if (ld < 0 || ld >= (int64_t(1) << 36) || (out && ld && ld < d)) return LCE_ERR_SHAPE;
    if (host_misaligned(x) || (ld * (dtype == LCE_BF16 ? 2 : 4)) % 16) return LCE_ERR_ALIGN;
    return host_check_packed(codes, ld_codes, exps, ld_exps, N, d);
}

PackArgs pack_args(const void *x, void *out, int64_t ld, int64_t N, int64_t d, const uint8_t *codes, int64_t ld_codes, const int8_t *exps,
                   int64_t ld_exps) {
    return PackArgs{x, out, const_cast<uint8_t *>(codes), const_cast<int8_t *>(exps), ld ? ld : d, ld_codes, ld_exps, N,
                    static_cast<int>(d), static_cast<int>((d + 255) / 256)};
}
int pack_grid(const PackArgs &r, const HostDev &dev) {
    return static_cast<int>(std::min<int64_t>(((r.N + kRows - 1) / kRows * r.per + 7) / 8, static_cast<int64_t>(dev.sms) * 8));
}

lce_status_t check_wgrad(const lce_wgrad_t *a) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->dw_dtype != LCE_FP32 && !(a->dw_dtype == LCE_BF16 && a->dtype == LCE_BF16)) return LCE_ERR_DTYPE;
    if (a->T < 0 || a->T >= (int64_t(1) << 30) || a->n < 8 || a->k < 8 || a->n >= (1 << 24) || a->k >= (1 << 24) ||
        a->n * a->k >= (int64_t(1) << 40))
        return LCE_ERR_SHAPE;
    return a->n % 8 || a->k % 8 ? LCE_ERR_ALIGN : LCE_OK;
}

// SMs that the rule below reckons with: those of the one part this library runs on, as a constant, since the workspace
// function answers from the sizes alone, without a device.
constexpr int kSms = 152;

// Splits of the tokens where there are few tiles. The times compared are in steps of 64 tokens of a unit (0.27 us): a unit
// costs 10 more for its start and output, and the join 8 and its bytes.
int splits(const lce_wgrad_t *a) {
    const int64_t tiles = (a->n + kWgTile - 1) / kWgTile * ((a->k + kWgTile - 1) / kWgTile), parts = a->dtype == LCE_FP32 ? 3 : 1,
                  steps = (a->T + kWgK - 1) / kWgK;
    auto time = [&](int64_t s) {
        const double waves = static_cast<double>((tiles * s + kSms / 2 - 1) / (kSms / 2)), sums = static_cast<double>(a->n) * a->k * 4;
        return waves * (static_cast<double>((steps + s - 1) / s * parts) + 10) + (s > 1 ? 8 + (2 * s + 1) * sums / 1.5e6 : 0);
    };
    int64_t best = 1;
    for (int64_t s = 2; s <= steps && tiles * s <= kSms; ++s)
        if (time(s) < 0.95 * time(best)) best = s;
    const int64_t per = (steps + best - 1) / best;   // no split without steps
    return static_cast<int>(steps > 0 ? (steps + per - 1) / per : 1);
}
// Steps that an accumulator takes. The tensor cores truncate their fp32 sums, which is a loss in one direction that grows
// with the number of additions, so longer sums are those of runs, added up in fp32 in memory. Off by, of the norm (all terms
// positive; in brackets terms of random signs), and the time:
//   fp32 dy, 8192 tokens: runs of 8 steps 3.2e-7 (1.7e-7), 12 5.5e-7, 16 8.3e-7, one run 1.3e-5 (3.6e-6), a product of
//     plain fp32 1.3e-6 (1.6e-6); 4096 tokens, 4096 x 4096: 533, 471, 398 us for runs of 8, 12 and 16, 295 in one
//   bf16 dy, fp32 dw, 7373 tokens: 8 2.5e-7 (1.6e-7), 16 6.7e-7 (2.9e-7), 32 1.7e-6 (6.0e-7), one run 1.0e-5 (3.2e-6), plain
//     7.7e-7 (3.4e-7); 4096 tokens, 4096 x 4096: 388, 224, 145 us for runs of 8, 16 and 32, 111 in one; 7373 tokens,
//     16384 x 4096: 2515, 1505, 955 and 584
// A bf16 dw is rounded by up to 2^-8 anyway: 32768 tokens (off by 9e-5; 65536 by 1.8e-4, 262144 by 7e-4) are one run.
int longest_run(const lce_wgrad_t *a) { return a->dw_dtype == LCE_BF16 ? 512 : a->dtype == LCE_FP32 ? 8 : 16; }
// A bf16 dw of several splits or runs is rounded from fp32 sums in scratch, by the join.
bool through_scratch(const lce_wgrad_t *a, int s) {
    return s > 1 || (a->dw_dtype == LCE_BF16 && a->T > static_cast<int64_t>(longest_run(a)) * kWgK);
}
size_t split_bytes(const lce_wgrad_t *a, int s) { return through_scratch(a, s) ? static_cast<size_t>(s) * a->n * a->k * sizeof(float) : 0; }
int64_t part_columns(const lce_wgrad_t *a) { return (a->n + 63) / 64 * 64; }
size_t part_bytes(const lce_wgrad_t *a) { return a->dtype == LCE_FP32 ? static_cast<size_t>(a->T) * part_columns(a) * 6 : 0; }

bool encode_dy(CUtensorMap *m, const HostDev &dev, const void *p, int64_t T, int64_t n, int64_t ld, bool whole) {
    const cuuint64_t two[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(T)}, row[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
    const cuuint64_t three[3] = {64, static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(n / 64)};
    const cuuint32_t box[3] = {64, kWgK, 2}, es[3] = {1, 1, 1};
    return dev.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, whole ? 3 : 2, const_cast<void *>(p), whole ? three : two, row, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_codes(CUtensorMap *m, const HostDev &dev, const void *p, int64_t T, int64_t k, int64_t ld) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(T)}, row[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {kWgHalf, kWgK}, es[2] = {1, 1};
    return dev.encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, row, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename O>
lce_status_t wgrad(const lce_wgrad_t *a, const HostDev &dev, uint8_t *scratch, cudaStream_t st) {
    WgMaps maps{};
    WgArgs r{};
    const int64_t ld = a->ld_dy ? a->ld_dy : a->n;
    r.exps = a->exps, r.ld_exps = a->ld_exps, r.T = static_cast<int>(a->T), r.n = static_cast<int>(a->n), r.k = static_cast<int>(a->k);
    r.mt = (r.n + kWgTile - 1) / kWgTile, r.nt = (r.k + kWgTile - 1) / kWgTile, r.steps = (r.T + kWgK - 1) / kWgK;
    r.splits = splits(a), r.per = (r.steps + r.splits - 1) / r.splits, r.run = longest_run(a), r.status = dev.status;
    if (!encode_codes(&maps.codes, dev, a->codes, a->T, a->k, a->ld_codes)) return LCE_ERR_SHAPE;
    if (a->dtype == LCE_FP32) {
        const int64_t wide = part_columns(a), size = a->T * wide;
        auto *parts = reinterpret_cast<__nv_bfloat16 *>(scratch + split_bytes(a, r.splits));
        r.parts = 3, r.whole = 1;
        for (int p = 0; p < 3; ++p)
            if (!encode_dy(&maps.dy[p], dev, parts + p * size, a->T, wide, wide, true)) return LCE_ERR_SHAPE;
        k_wgrad_parts<<<static_cast<unsigned>((size / 4 + 255) / 256), 256, 0, st>>>(static_cast<const float *>(a->dy), ld, r.T, r.n,
                                                                                   static_cast<int>(wide), parts);
        const lce_status_t s = host_launched();
        if (s != LCE_OK) return s;
    } else {
        r.parts = 1, r.whole = a->n % 64 == 0;
        if (!encode_dy(&maps.dy[0], dev, a->dy, a->T, a->n, ld, r.whole != 0)) return LCE_ERR_SHAPE;
    }
    const int units = r.mt * r.nt * r.splits, grid = 2 * std::min(units, dev.sms / 2);
    if (!through_scratch(a, r.splits)) {
        r.out = a->dw;
        const lce_status_t s = host_smem<k_wgrad<O>>(dev, kWgSmem);
        if (s != LCE_OK) return s;
        k_wgrad<O><<<grid, kWgThreads, kWgSmem, st>>>(maps, r);
        return host_launched();
    }
    r.out = scratch;
    lce_status_t s = host_smem<k_wgrad<float>>(dev, kWgSmem);
    if (s != LCE_OK) return s;
    k_wgrad<float><<<grid, kWgThreads, kWgSmem, st>>>(maps, r);
    if ((s = host_launched()) != LCE_OK) return s;
    const int64_t count = a->n * a->k;
    return host_launch_early(k_wgrad_join<O>, dim3(static_cast<unsigned>((count / 4 + 255) / 256)), 256, 0, st,
                             reinterpret_cast<const float *>(scratch), r.splits, count, static_cast<O *>(a->dw));
}

}  // namespace

extern "C" {

lce_status_t lce_pack8(lce_dtype_t dtype, const void *x, int64_t ld_x, int64_t N, int64_t d, uint8_t *codes, int64_t ld_codes,
                       int8_t *exps, int64_t ld_exps, lce_stream_t stream) {
    lce_status_t s = check_plain(dtype, x, ld_x, N, d, codes, ld_codes, exps, ld_exps, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (N == 0) return LCE_OK;
    const PackArgs r = pack_args(x, nullptr, ld_x, N, d, codes, ld_codes, exps, ld_exps);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LCE_BF16) k_pack8<__nv_bfloat16><<<pack_grid(r, dev), 256, 0, st>>>(r);
    else k_pack8<float><<<pack_grid(r, dev), 256, 0, st>>>(r);
    return host_launched();
}

lce_status_t lce_unpack8(lce_dtype_t dtype, const uint8_t *codes, int64_t ld_codes, const int8_t *exps, int64_t ld_exps, int64_t N,
                         int64_t d, void *out, int64_t ld_out, lce_stream_t stream) {
    lce_status_t s = check_plain(dtype, out, ld_out, N, d, codes, ld_codes, exps, ld_exps, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (N == 0) return LCE_OK;
    const PackArgs r = pack_args(nullptr, out, ld_out, N, d, codes, ld_codes, exps, ld_exps);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LCE_BF16) k_unpack8<__nv_bfloat16><<<pack_grid(r, dev), 256, 0, st>>>(r);
    else k_unpack8<float><<<pack_grid(r, dev), 256, 0, st>>>(r);
    return host_launched();
}

size_t lce_packed_wgrad_workspace_size(const lce_wgrad_t *a) {
    return check_wgrad(a) == LCE_OK ? split_bytes(a, splits(a)) + part_bytes(a) : 0;
}

lce_status_t lce_packed_wgrad(const lce_wgrad_t *a) {
    lce_status_t s = check_wgrad(a);
    if (s != LCE_OK) return s;
    if (!a->dw) return LCE_ERR_NULL;
    if (host_misaligned(a->dw)) return LCE_ERR_ALIGN;
    if (a->T > 0) {
        if (!a->dy) return LCE_ERR_NULL;
        if (a->ld_dy < 0 || a->ld_dy >= (int64_t(1) << 36)) return LCE_ERR_SHAPE;
        if (host_misaligned(a->dy) || (a->ld_dy * (a->dtype == LCE_BF16 ? 2 : 4)) % 16) return LCE_ERR_ALIGN;
        if ((s = host_check_packed(a->codes, a->ld_codes, a->exps, a->ld_exps, a->T, a->k)) != LCE_OK) return s;
    }
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    if (a->T == 0)
        return host_cuda(cudaMemsetAsync(a->dw, 0, static_cast<size_t>(a->n) * a->k * (a->dw_dtype == LCE_BF16 ? 2 : 4), st));
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    if ((s = scratch.get(a->workspace, a->workspace_bytes, lce_packed_wgrad_workspace_size(a), &base)) != LCE_OK) return s;
    return a->dw_dtype == LCE_BF16 ? wgrad<__nv_bfloat16>(a, dev, base, st) : wgrad<float>(a, dev, base, st);
}

}  // extern "C"
