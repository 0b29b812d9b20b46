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

// The pieces that a warp takes: every gridDim.x * 8th of all rows' pieces, without a division a piece.
struct Pieces {
    int64_t row, rows;   // of the next piece; rows to go on by
    int at, ats, per;    // its place in the row; places to go on by
    __device__ __forceinline__ Pieces(int per_) : per(per_) {
        const int64_t first = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32, step = static_cast<int64_t>(gridDim.x) * 8;
        row = first / per, at = static_cast<int>(first - row * per);
        rows = step / per, ats = static_cast<int>(step - rows * per);
    }
    __device__ __forceinline__ void next() {
        row += rows, at += ats;
        if (at >= per) at -= per, ++row;
    }
};

constexpr int kTogether = 4;   // pieces whose loads a warp has in flight

// Both are bounded by HBM: no lane waits for another but within 16, and four
// loads of 16 bytes (of fp32, eight) are in flight a thread.
template <typename T>
__global__ void __launch_bounds__(256) k_pack8(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    for (Pieces p(a.per); p.row < a.N;) {
        Pack<T> v[kTogether];
        int64_t row[kTogether];
        int col[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i, p.next()) {
            row[i] = p.row, col[i] = p.at * 256 + lane * kVec;
            if (col[i] >= a.d) row[i] = a.N;   // nothing there
            if (row[i] < a.N) v[i] = load_pack(static_cast<const T *>(a.x) + row[i] * a.ld + col[i]);
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            float x[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) x[k] = 0.f;
            if (row[i] < a.N) v[i].get(x);
            const int e = pack_exponent(block_top(x));
            if (row[i] >= a.N) continue;
            *reinterpret_cast<uint2 *>(a.codes + row[i] * a.ld_codes + col[i]) = codes8(x, pack_scale(e));
            if (col[i] % kPackBlock == 0) a.exps[col[i] / kPackBlock * a.ld_exps + row[i]] = static_cast<int8_t>(e);
        }
        __syncwarp();
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_unpack8(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    for (Pieces p(a.per); p.row < a.N;) {
        uint2 c[kTogether];
        int e[kTogether], col[kTogether];
        int64_t row[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i, p.next()) {
            row[i] = p.row, col[i] = p.at * 256 + lane * kVec;
            if (col[i] >= a.d) row[i] = a.N;
            if (row[i] >= a.N) continue;
            c[i] = *reinterpret_cast<const uint2 *>(a.codes + row[i] * a.ld_codes + col[i]);
            e[i] = a.exps[col[i] / kPackBlock * a.ld_exps + row[i]];
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            if (row[i] >= a.N) continue;
            float x[kVec];
            values8(c[i], unpack_scale(e[i]), x);
            store_pack(static_cast<T *>(a.out) + row[i] * a.ld + col[i], x);
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
    return static_cast<int>(std::min<int64_t>((r.N * r.per + 7) / 8, static_cast<int64_t>(dev.sms) * 8));
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
size_t split_bytes(const lce_wgrad_t *a, int s) { return s > 1 ? static_cast<size_t>(s) * a->n * a->k * sizeof(float) : 0; }
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
    r.splits = splits(a), r.per = (r.steps + r.splits - 1) / r.splits, r.status = dev.status;
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
    if (r.splits == 1) {
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
