// Norms before and after a block, fused with its gate and residual scale:
// kernels and host side of lce_block_norm_forward / _backward.
#include <cuda_bf16.h>

#include "lce_host.h"

using namespace lce;

namespace {

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

struct NormArgs {
    const void *x, *b, *w_post, *gate, *w_pre, *r_in, *dr, *dn;
    void *r, *n, *dx, *db, *dgate;
    float *rstd_post, *rstd_pre;
    int64_t ld_x, ld_b, ld_gate, ld_r, ld_dr, ld_dn;
    int64_t N;
    int d, gate_full;
    float scale, eps;
    float *part;   // backward: partial column sums [3][groups][d] (w_pre, w_post, gate)
};

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

// One block a row; a thread holds CH packs of its row's elements.
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

// Persistent blocks, one row at a time. The two row sums of the formulas are
// taken in one round: with u = w_pre dn, m1 = mean(u rhat) and
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

// Adds the blocks' column sums in block order: 32 columns a block, 8 threads
// a column, joined in a fixed tree.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_cols(const float *part, int groups, int d, T *dw_pre, T *dw_post,
                                                   T *dgate) {
    __shared__ float red[8][33];
    T *out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
    if (!out) return;
    const int x = threadIdx.x & 31, y = threadIdx.x / 32, col = blockIdx.x * 32 + x;
    const float *p = part + static_cast<int64_t>(blockIdx.y) * groups * d + col;
    float s = 0.f;
    if (col < d)
        for (int g = y; g < groups; g += 8) s += p[static_cast<int64_t>(g) * d];
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && col < d) {
        for (int k = 1; k < 8; ++k) s += red[k][x];
        out[col] = static_cast<T>(s);
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

template <typename T>
lce_status_t forward(const lce_norm_t *a, cudaStream_t st) {
    const NormArgs r = make_norm(a);
    const unsigned grid = static_cast<unsigned>(a->N);
    const int th = row_threads(r.d);
    switch (row_packs(r.d)) {
        case 1: k_norm_fwd<T, 1><<<grid, th, 0, st>>>(r); break;
        case 2: k_norm_fwd<T, 2><<<grid, th, 0, st>>>(r); break;
        default: k_norm_fwd<T, 4><<<grid, th, 0, st>>>(r); break;
    }
    return host_launched();
}

int64_t norm_groups(const lce_norm_t *a) { return a->N < 304 ? (a->N > 0 ? a->N : 1) : 304; }

template <typename K>
lce_status_t big_smem(K kernel, int smem) {
    if (smem + 1024 <= 48 * 1024) return LCE_OK;   // 1024: the kernel's static share
    return host_cuda(cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
}

template <typename T>
lce_status_t backward(const lce_norm_t *a, float *part, cudaStream_t st) {
    NormArgs r = make_norm(a);
    r.part = part;
    const int groups = static_cast<int>(norm_groups(a));
    const int th = row_threads(r.d), smem = 3 * r.d * 4;
    lce_status_t s;
    auto go = [&](auto kernel) {
        if ((s = big_smem(kernel, smem)) != LCE_OK) return s;
        kernel<<<groups, th, smem, st>>>(r);
        return host_launched();
    };
    switch (row_packs(r.d)) {
        case 1: s = go(k_norm_bwd<T, 1>); break;
        case 2: s = go(k_norm_bwd<T, 2>); break;
        default: s = go(k_norm_bwd<T, 4>); break;
    }
    if (s != LCE_OK) return s;
    T *dgate = a->gate && !a->gate_full ? static_cast<T *>(a->dgate) : nullptr;
    T *dpre = a->w_pre ? static_cast<T *>(a->dw_pre) : nullptr, *dpost = a->w_post ? static_cast<T *>(a->dw_post) : nullptr;
    if (!dgate && !dpre && !dpost) return LCE_OK;
    k_norm_cols<T><<<dim3((r.d + 31) / 32, 3), 256, 0, st>>>(part, groups, r.d, dpre, dpost, dgate);
    return host_launched();
}

}  // namespace

extern "C" {

size_t lce_block_norm_workspace_size(const lce_norm_t *a) {
    if (!a || a->N < 0 || a->N >= (int64_t(1) << 31) || a->d < 8 || a->d > kMaxD || a->d % 8) return 0;
    return static_cast<size_t>(3 * norm_groups(a) * a->d) * sizeof(float);
}

lce_status_t lce_block_norm_forward(const lce_norm_t *a) {
    lce_status_t s = check_norm(a, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (a->N == 0) return LCE_OK;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    return a->dtype == LCE_BF16 ? forward<__nv_bfloat16>(a, st) : forward<float>(a, st);
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
    return a->dtype == LCE_BF16 ? backward<__nv_bfloat16>(a, part, st) : backward<float>(a, part, st);
}

}  // extern "C"
