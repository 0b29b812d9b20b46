// Activations in 8 bits (lce_pack8, lce_unpack8) and the gradient of a weight
// from them (lce_packed_wgrad): kernels and host side.
#include <cuda_bf16.h>

#include <algorithm>

#include "e4m3.cuh"
#include "lce_host.h"
#include "row_ring.cuh"

using namespace lce;

namespace {

struct PackArgs {
    const void *x;
    void *out;
    uint8_t *codes;
    int8_t *exps;
    int64_t ld, ld_codes, ld_exps, pieces;   // pieces: N * wpr
    int d, wpr;                              // wpr: pieces of 256 channels in a row, each taken by a warp
};

template <typename T>
__global__ void __launch_bounds__(256) k_pack8(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; p < a.pieces; p += step) {
        const int64_t row = p / a.wpr;
        const int col = static_cast<int>(p - row * a.wpr) * 256 + lane * kVec;
        float x[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = 0.f;
        if (col < a.d) load_pack(static_cast<const T *>(a.x) + row * a.ld + col).get(x);
        const int e = pack_exponent(block_top(x));
        if (col < a.d) {
            *reinterpret_cast<uint2 *>(a.codes + row * a.ld_codes + col) = codes8(x, pack_scale(e));
            if (col % kPackBlock == 0) a.exps[col / kPackBlock * a.ld_exps + row] = static_cast<int8_t>(e);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_unpack8(const PackArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; p < a.pieces; p += step) {
        const int64_t row = p / a.wpr;
        const int col = static_cast<int>(p - row * a.wpr) * 256 + lane * kVec;
        if (col >= a.d) continue;
        float x[kVec];
        values8(*reinterpret_cast<const uint2 *>(a.codes + row * a.ld_codes + col),
                unpack_scale(a.exps[col / kPackBlock * a.ld_exps + row]), x);
        store_pack(static_cast<T *>(a.out) + row * a.ld + col, x);
    }
}

struct WgradArgs {
    const void *dy;
    const uint8_t *codes;
    const int8_t *exps;
    void *dw;
    int64_t ld_dy, ld_codes, ld_exps;
    int T, n, k;
};

// 64 x 64 outputs a block, 4 x 4 a thread
template <typename T, typename O>
__global__ void __launch_bounds__(256) k_wgrad_simple(const WgradArgs a) {
    __shared__ float sy[16][64], sx[16][64];
    const int n0 = blockIdx.y * 64, k0 = blockIdx.x * 64;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    float acc[4][4] = {};
    for (int t0 = 0; t0 < a.T; t0 += 16) {
        for (int i = threadIdx.x; i < 16 * 64; i += 256) {
            const int t = t0 + i / 64, c = i % 64;
            sy[i / 64][c] = t < a.T && n0 + c < a.n ? static_cast<float>(static_cast<const T *>(a.dy)[t * a.ld_dy + n0 + c]) : 0.f;
            float v = 0.f, u;
            if (t < a.T && k0 + c < a.k) {
                from_codes(a.codes[t * a.ld_codes + k0 + c], v, u);
                v *= unpack_scale(a.exps[(k0 + c) / kPackBlock * a.ld_exps + t]);
            }
            sx[i / 64][c] = v;
        }
        __syncthreads();
        for (int t = 0; t < 16; ++t)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sy[t][ti + i], sx[t][tj + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (n0 + ti + i < a.n && k0 + tj + j < a.k)
                static_cast<O *>(a.dw)[static_cast<int64_t>(n0 + ti + i) * a.k + k0 + tj + j] = static_cast<O>(acc[i][j]);
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

int plain_grid(const PackArgs &r, const HostDev &dev) {
    return static_cast<int>(std::min<int64_t>((r.pieces + 7) / 8, static_cast<int64_t>(dev.sms) * 8));
}

lce_status_t check_wgrad(const lce_wgrad_t *a) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->dw_dtype != LCE_FP32 && !(a->dw_dtype == LCE_BF16 && a->dtype == LCE_BF16)) return LCE_ERR_DTYPE;
    if (a->T < 0 || a->T >= (int64_t(1) << 30) || a->n < 8 || a->k < 8 || a->n >= (1 << 24) || a->k >= (1 << 24)) return LCE_ERR_SHAPE;
    return a->n % 8 || a->k % 8 ? LCE_ERR_ALIGN : LCE_OK;
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
    const int wpr = static_cast<int>((d + 255) / 256);
    const PackArgs r{x, nullptr, codes, exps, ld_x ? ld_x : d, ld_codes, ld_exps, N * wpr, static_cast<int>(d), wpr};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LCE_BF16) k_pack8<__nv_bfloat16><<<plain_grid(r, dev), 256, 0, st>>>(r);
    else k_pack8<float><<<plain_grid(r, dev), 256, 0, st>>>(r);
    return host_launched();
}

lce_status_t lce_unpack8(lce_dtype_t dtype, const uint8_t *codes, int64_t ld_codes, const int8_t *exps, int64_t ld_exps, int64_t N,
                         int64_t d, void *out, int64_t ld_out, lce_stream_t stream) {
    lce_status_t s = check_plain(dtype, out, ld_out, N, d, codes, ld_codes, exps, ld_exps, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (N == 0) return LCE_OK;
    const int wpr = static_cast<int>((d + 255) / 256);
    const PackArgs r{nullptr, out, const_cast<uint8_t *>(codes), const_cast<int8_t *>(exps), ld_out ? ld_out : d, ld_codes, ld_exps,
                     N * wpr, static_cast<int>(d), wpr};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LCE_BF16) k_unpack8<__nv_bfloat16><<<plain_grid(r, dev), 256, 0, st>>>(r);
    else k_unpack8<float><<<plain_grid(r, dev), 256, 0, st>>>(r);
    return host_launched();
}

size_t lce_packed_wgrad_workspace_size(const lce_wgrad_t *a) {
    if (check_wgrad(a) != LCE_OK) return 0;
    return 0;
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
    const WgradArgs r{a->dy, a->codes, a->exps, a->dw, a->ld_dy ? a->ld_dy : a->n, a->ld_codes, a->ld_exps, static_cast<int>(a->T),
                      static_cast<int>(a->n), static_cast<int>(a->k)};
    const dim3 grid(static_cast<unsigned>((a->k + 63) / 64), static_cast<unsigned>((a->n + 63) / 64));
    if (a->dtype == LCE_FP32) k_wgrad_simple<float, float><<<grid, 256, 0, st>>>(r);
    else if (a->dw_dtype == LCE_FP32) k_wgrad_simple<__nv_bfloat16, float><<<grid, 256, 0, st>>>(r);
    else k_wgrad_simple<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, st>>>(r);
    return host_launched();
}

}  // extern "C"
