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
            const int e = pack_exponent(block_top(r[c]));
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
// each column owned by one thread, until the block's rows are done.
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

template <typename T>
lce_status_t forward(const LnArgs &r, cudaStream_t st) {
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
lce_status_t backward(const lce_layer_norm_t *a, LnArgs r, const HostDev &dev, cudaStream_t st) {
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(r.N, kColGroups)));
    const int th = row_threads(r.d), smem = 2 * r.d * 4, packs = (r.d / kVec + 511) / 512;
    auto go = [&](auto ch) {
        constexpr auto kernel = k_ln_bwd<T, decltype(ch)::value>;
        const lce_status_t s = host_smem<kernel>(dev, 2 * kMaxD * 4);
        if (s != LCE_OK) return s;
        kernel<<<grid, th, smem, st>>>(r);
        return host_launched();
    };
    const lce_status_t s = packs == 1   ? go(std::integral_constant<int, 1>())
                           : packs == 2 ? go(std::integral_constant<int, 2>())
                                        : go(std::integral_constant<int, 4>());
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
    return a->dtype == LCE_BF16 ? forward<__nv_bfloat16>(r, st) : forward<float>(r, st);
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
