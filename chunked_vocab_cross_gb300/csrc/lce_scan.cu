// The gated recurrence over packed sequences: kernels and host side of
// lce_recurrence_forward / _backward.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "lce_host.h"
#include "tc_ptx.cuh"

using namespace lce;

namespace {

constexpr int kEvery = 128;   // tokens between kept states

struct ScanArgs {
    const int32_t *cu;
    int B, T, len, d;   // len: of every sequence, without offsets
    const void *x, *g, *dh;
    const float *state, *dfinal;
    float *kept, *final, *dstate;
    void *h, *dx, *dg;
    int64_t ld_x, ld_g, ld_h, ld_dh, ld_dx, ld_dg;
    int *status;
    // first token of sequence b (b <= B), within [0, T] whatever the offsets hold
    __device__ __forceinline__ int start(int b) const { return cu ? min(max(cu[b], 0), T) : b * len; }
};

// The gate and its complement, each to its own relative precision. The exponent
// is bounded so that neither the sum nor its reciprocal leaves fp32.
__device__ __forceinline__ void gate(float g, float &a, float &rest) {
    const float z = -g * 1.4426950408889634f;
    const float e = exp2f(z > 126.f ? 126.f : z);   // (a NaN stays one)
    a = 1.f / (1.f + e);
    rest = e * a;
}

__device__ __forceinline__ void check_offsets(const ScanArgs &a) {
    if (!a.cu || blockIdx.x || threadIdx.x >= 32) return;
    bool bad = false;
    for (int b = threadIdx.x; b <= a.B; b += 32) bad |= b == 0 ? a.cu[0] != 0 : a.cu[b] < a.cu[b - 1] || a.cu[b] > a.T;
    if (__any_sync(0xffffffffu, bad) && threadIdx.x == 0) atomicOr(a.status, LCE_DEV_SEQLENS);
}

// A thread a channel of a sequence
template <typename T>
__global__ void __launch_bounds__(128) k_scan_fwd_simple(const ScanArgs a, int slices) {
    check_offsets(a);
    const int b = blockIdx.x / slices, ch = (blockIdx.x - b * slices) * 128 + threadIdx.x;
    if (ch >= a.d) return;
    const int64_t at = static_cast<int64_t>(b) * a.d + ch;
    const bool tail = b == a.B;
    float h = tail || !a.state ? 0.f : a.state[at];
    const int end = tail ? a.T : max(a.start(b + 1), a.start(b));
    if (tail && a.kept) a.kept[ch] = 0.f;
    for (int t = a.start(b); t < end; ++t) {
        if (!tail) {
            float f, rest;
            gate(static_cast<float>(static_cast<const T *>(a.g)[t * a.ld_g + ch]), f, rest);
            h = fmaf(f, h, rest * static_cast<float>(static_cast<const T *>(a.x)[t * a.ld_x + ch]));
        }
        static_cast<T *>(a.h)[t * a.ld_h + ch] = static_cast<T>(h);
        if (a.kept && (t + 1) % kEvery == 0 && t + 1 < a.T) a.kept[static_cast<int64_t>((t + 1) / kEvery) * a.d + ch] = h;
    }
    if (!tail && a.final) a.final[at] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) k_scan_bwd_simple(const ScanArgs a, int slices) {
    check_offsets(a);
    const int b = blockIdx.x / slices, ch = (blockIdx.x - b * slices) * 128 + threadIdx.x;
    if (ch >= a.d) return;
    const int64_t at = static_cast<int64_t>(b) * a.d + ch;
    const bool tail = b == a.B;
    const int begin = a.start(b), end = tail ? a.T : max(a.start(b + 1), begin);
    if (tail) {
        for (int t = begin; t < end; ++t)
            static_cast<T *>(a.dx)[t * a.ld_dx + ch] = static_cast<T *>(a.dg)[t * a.ld_dg + ch] = static_cast<T>(0.f);
        return;
    }
    float m = a.dfinal ? a.dfinal[at] : 0.f;
    float before[kEvery];
    for (int hi = end; hi > begin;) {
        const int lo = max(begin, (hi - 1) / kEvery * kEvery);
        float h = lo == begin ? (a.state ? a.state[at] : 0.f) : a.kept[static_cast<int64_t>(lo / kEvery) * a.d + ch];
        for (int t = lo; t < hi; ++t) {
            float f, rest;
            gate(static_cast<float>(static_cast<const T *>(a.g)[t * a.ld_g + ch]), f, rest);
            before[t - lo] = h;
            h = fmaf(f, h, rest * static_cast<float>(static_cast<const T *>(a.x)[t * a.ld_x + ch]));
        }
        for (int t = hi - 1; t >= lo; --t) {
            float f, rest;
            gate(static_cast<float>(static_cast<const T *>(a.g)[t * a.ld_g + ch]), f, rest);
            const float l = static_cast<float>(static_cast<const T *>(a.dh)[t * a.ld_dh + ch]) + m;
            const float x = static_cast<float>(static_cast<const T *>(a.x)[t * a.ld_x + ch]);
            static_cast<T *>(a.dx)[t * a.ld_dx + ch] = static_cast<T>(rest * l);
            static_cast<T *>(a.dg)[t * a.ld_dg + ch] = static_cast<T>(l * (before[t - lo] - x) * f * rest);
            m = f * l;
        }
        hi = lo;
    }
    if (a.dstate) a.dstate[at] = m;
}

lce_status_t check_rows(const void *p, int64_t ld, int64_t d, int elt) {
    if (!p) return LCE_ERR_NULL;
    if (ld < 0 || ld >= (int64_t(1) << 36) || (ld && ld < d)) return LCE_ERR_SHAPE;
    return host_misaligned(p) || (ld * elt) % 16 ? LCE_ERR_ALIGN : LCE_OK;
}

lce_status_t check_scan(const lce_recurrence_t *a, bool backward) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    if (a->T < 0 || a->T >= (int64_t(1) << 30) || a->B < 1 || a->B >= (int64_t(1) << 30) || a->d < 8 || a->d >= (1 << 24)) return LCE_ERR_SHAPE;
    if (a->d % 8) return LCE_ERR_ALIGN;
    if (!a->cu && a->T % a->B) return LCE_ERR_SHAPE;
    for (const float *p : {a->state, static_cast<const float *>(a->kept), static_cast<const float *>(a->final), a->dfinal,
                           static_cast<const float *>(a->dstate)})
        if (host_misaligned(p)) return LCE_ERR_ALIGN;
    if (a->T == 0) return LCE_OK;
    if (backward && !a->kept) return LCE_ERR_NULL;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    const struct { const void *p; int64_t ld; bool used; } all[] = {{a->x, a->ld_x, true}, {a->g, a->ld_g, true}, {a->h, a->ld_h, !backward},
        {a->dh, a->ld_dh, backward}, {a->dx, a->ld_dx, backward}, {a->dg, a->ld_dg, backward}};
    for (const auto &t : all) {
        if (!t.used) continue;
        const lce_status_t s = check_rows(t.p, t.ld, a->d, elt);
        if (s != LCE_OK) return s;
    }
    return LCE_OK;
}

ScanArgs make_args(const lce_recurrence_t *a, const HostDev &dev) {
    ScanArgs r{};
    auto ld = [&](int64_t v) { return v ? v : a->d; };
    r.cu = a->cu, r.B = static_cast<int>(a->B), r.T = static_cast<int>(a->T), r.len = static_cast<int>(a->T / a->B);
    r.d = static_cast<int>(a->d);
    r.x = a->x, r.g = a->g, r.dh = a->dh, r.state = a->state, r.dfinal = a->dfinal;
    r.kept = a->kept, r.final = a->final, r.dstate = a->dstate, r.h = a->h, r.dx = a->dx, r.dg = a->dg;
    r.ld_x = ld(a->ld_x), r.ld_g = ld(a->ld_g), r.ld_h = ld(a->ld_h), r.ld_dh = ld(a->ld_dh), r.ld_dx = ld(a->ld_dx), r.ld_dg = ld(a->ld_dg);
    r.status = dev.status;
    return r;
}

}  // namespace

extern "C" {

lce_status_t lce_recurrence_forward(const lce_recurrence_t *a) {
    lce_status_t s = check_scan(a, false);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    const ScanArgs r = make_args(a, dev);
    const int slices = (r.d + 127) / 128;
    const unsigned grid = static_cast<unsigned>((a->B + 1) * slices);
    if (a->dtype == LCE_BF16) k_scan_fwd_simple<__nv_bfloat16><<<grid, 128, 0, st>>>(r, slices);
    else k_scan_fwd_simple<float><<<grid, 128, 0, st>>>(r, slices);
    return host_launched();
}

lce_status_t lce_recurrence_backward(const lce_recurrence_t *a) {
    lce_status_t s = check_scan(a, true);
    if (s != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    const ScanArgs r = make_args(a, dev);
    const int slices = (r.d + 127) / 128;
    const unsigned grid = static_cast<unsigned>((a->B + 1) * slices);
    if (a->dtype == LCE_BF16) k_scan_bwd_simple<__nv_bfloat16><<<grid, 128, 0, st>>>(r, slices);
    else k_scan_bwd_simple<float><<<grid, 128, 0, st>>>(r, slices);
    return host_launched();
}

}  // extern "C"
