// Host side of attention over packed sequences: argument checks, workspace
// and launches.
#include <algorithm>
#include <type_traits>

#include "lce_attn_bwd.cuh"
#include "lce_attn_fwd.cuh"
#include "lce_attn_simt.cuh"
#include "lce_host.h"

using namespace lce;

namespace {

// Whether the rows of D elements that lie t * ts + h * hs on (t < T, h < H) are apart from one another.
bool rows_apart(int64_t ts, int64_t hs, int64_t T, int64_t H, int64_t D) {
    if ((T > 1 && ts < D) || (H > 1 && hs < D)) return false;
    if (T <= 1 || H <= 1 || ts >= (H - 1) * hs + D || (hs - D) / ts >= T - 1) return true;   // tokens, or heads, outermost
    for (int64_t h = 1; h < H; ++h) {   // interleaved: the tokens on either side of the head's distance
        const int64_t t = h * hs / ts, past = h * hs - t * ts;
        if ((t < T && past < D) || (t + 1 < T && ts - past < D)) return false;
    }
    return true;
}

lce_status_t check_side(const void *p, int64_t ts, int64_t hs, int64_t T, int64_t H, int64_t D, int elt, bool out) {
    if (T == 0) return LCE_OK;   // an empty side is never read or written
    if (!p) return LCE_ERR_NULL;
    if (host_misaligned(p) || (ts * elt) % 16 || (hs * elt) % 16) return LCE_ERR_ALIGN;
    if (ts < 0 || hs < 0 || ts >= (int64_t(1) << 36) || hs >= (int64_t(1) << 36)) return LCE_ERR_SHAPE;
    if ((T > 1 && ts == 0) || (H > 1 && hs == 0)) return LCE_ERR_SHAPE;   // tensor maps have no zero strides
    if (out && !rows_apart(ts, hs, T, H, D)) return LCE_ERR_SHAPE;
    return LCE_OK;
}

lce_status_t check_shape(const lce_attn_t *a) {
    if (!a) return LCE_ERR_NULL;
    if (a->dtype != LCE_BF16 && a->dtype != LCE_FP32) return LCE_ERR_DTYPE;
    constexpr int64_t kMost = int64_t(1) << 30;
    if (a->Tq < 0 || a->Tk < 0 || a->Tq >= kMost || a->Tk >= kMost || a->B < 1 || a->B >= kMost || a->Hq < 1 ||
        a->Hk < 1 || a->Hq > 65535 || a->Hq % a->Hk || a->D < 1 || a->D > 128)
        return LCE_ERR_SHAPE;
    if (a->D % 8) return LCE_ERR_ALIGN;
    if ((a->cu_q == nullptr) != (a->cu_k == nullptr)) return LCE_ERR_NULL;
    if (!a->cu_q && (a->Tq % a->B || a->Tk % a->B)) return LCE_ERR_SHAPE;
    return LCE_OK;
}

lce_status_t check_common(const lce_attn_t *a) {
    lce_status_t s = check_shape(a);
    if (s != LCE_OK) return s;
    if (!(a->scale == a->scale) || a->scale - a->scale != 0.f) return LCE_ERR_ARG;   // NaN or infinite
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    if ((s = check_side(a->q, a->q_ts, a->q_hs, a->Tq, a->Hq, a->D, elt, false)) != LCE_OK) return s;
    if ((s = check_side(a->k, a->k_ts, a->k_hs, a->Tk, a->Hk, a->D, elt, false)) != LCE_OK) return s;
    if ((s = check_side(a->v, a->v_ts, a->v_hs, a->Tk, a->Hk, a->D, elt, false)) != LCE_OK) return s;
    if (a->Tq > 0 && !a->lse) return LCE_ERR_NULL;
    return LCE_OK;
}

AttnArgs make_args(const lce_attn_t *a, const HostDev &dev) {
    AttnArgs r{};
    r.q = a->q, r.k = a->k, r.v = a->v, r.o_in = a->o, r.dO = a->dO;
    r.o = a->o, r.dq = a->dq, r.dk = a->dk, r.dv = a->dv;
    r.lse = a->lse;
    r.q_ts = a->q_ts, r.q_hs = a->q_hs, r.k_ts = a->k_ts, r.k_hs = a->k_hs, r.v_ts = a->v_ts, r.v_hs = a->v_hs;
    r.o_ts = a->o_ts, r.o_hs = a->o_hs, r.dO_ts = a->dO_ts, r.dO_hs = a->dO_hs;
    r.dq_ts = a->dq_ts, r.dq_hs = a->dq_hs, r.dk_ts = a->dk_ts, r.dk_hs = a->dk_hs, r.dv_ts = a->dv_ts, r.dv_hs = a->dv_hs;
    const int B = static_cast<int>(a->B);
    r.sq = SeqMap{a->cu_q, B, static_cast<int>(a->Tq), static_cast<int>(a->Tq / B)};
    r.sk = SeqMap{a->cu_k, B, static_cast<int>(a->Tk), static_cast<int>(a->Tk / B)};
    r.Hq = static_cast<int>(a->Hq);
    r.Hk = static_cast<int>(a->Hk);
    r.group = r.Hq / r.Hk;
    r.D = static_cast<int>(a->D);
    r.causal = a->causal != 0;
    r.pair_heads = r.group % 2 == 0;
    r.scale = a->scale;
    r.scale_log2 = a->scale * kAttnLog2e;
    r.status = dev.status;
    return r;
}

// Tensor map of [tokens][heads][D] bf16 for boxes of 128 tokens of one head by
// 64 channels.
lce_status_t encode(CUtensorMap *m, const HostDev &dev, const void *p, int64_t T, int64_t H, int64_t D, int64_t ts,
                    int64_t hs) {
    if (H == 1) hs = D;   // strides of dimensions of one entry are not used, but have to be valid
    if (T == 1) ts = D;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
    cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(kTcTile)};
    cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = dev.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? LCE_OK : LCE_ERR_SHAPE;
}

// kEarly: see host_launch_early.
template <auto kKernel, bool kEarly = false, typename... A>
lce_status_t launch(const HostDev &dev, int64_t blocks, int threads, int smem, cudaStream_t st, const A &...args) {
    if (blocks >= (int64_t(1) << 31)) return LCE_ERR_SHAPE;
    if (smem > 48 * 1024) {
        const lce_status_t s = host_smem<kKernel>(dev, smem);
        if (s != LCE_OK) return s;
    }
    const dim3 grid(static_cast<unsigned>(blocks));
    if constexpr (kEarly) return host_launch_early(kKernel, grid, threads, smem, st, args...);
    kKernel<<<grid, threads, smem, st>>>(args...);
    return host_launched();
}

// SMs that the two rules below reckon with: those of the one part this library runs on, as a constant, since the
// workspace functions answer from the sizes alone, without a device.
constexpr int kSms = 152;

// Tiles of a sequence of average length, which is rounded up: a side with any tokens has a tile in each.
int64_t average_tiles(int64_t T, int64_t B) { return ((T + B - 1) / B + kTcTile - 1) / kTcTile; }

// Ranges that a row's keys are split into in the forward. Few rows and heads over long keys leave most SMs without
// work; their walks are split as far as that makes the longest shorter. The times compared are in key tiles of a walk
// (0.6 us): a piece costs 3 more for its start and output, 5 with an fp32 output, and the merge 3 and its bytes. Of
// the lengths only the averages are known here. (32 heads of 8 key heads of 128 channels: one row over 2048 keys 17 us
// against 26, over 32768 53 against 322; 2 heads, 8192 causal tokens: 44 against 86.)
int ranges(const lce_attn_t *a) {
    const int64_t group = a->Hq / a->Hk, tq = average_tiles(a->Tq, a->B), tk = average_tiles(a->Tk, a->B);
    if (a->dtype != LCE_BF16 || tk <= 8 || a->Tq * a->Hq > (1 << 24)) return 1;
    const double pieces = static_cast<double>(a->B) * (group % 2 == 0 ? tq * a->Hq / 2 : (tq + 1) / 2 * a->Hq),
                 mask = a->causal && a->Tq == a->Tk ? 0.5 : 1.0, merge = static_cast<double>(a->Tq * a->Hq * a->D) * 8 / 3e6;
    auto time = [&](int64_t n) {   // of the longest piece, or of everything shared out
        const double more = n > 1 ? 5 : 3, walk = static_cast<double>((tk + n - 1) / n);
        return std::max(walk + more, pieces * n * (walk * mask + more) / kSms) + (n > 1 ? 3 + n * merge : 0);
    };
    int64_t best = 1;
    for (int64_t n = 2; n <= 64 && n <= tk / 2; ++n)
        if (time(n) < 0.95 * time(best)) best = n;
    return static_cast<int>(best);
}

size_t range_bytes(const lce_attn_t *a, int n) {
    return n == 1 ? 0 : static_cast<size_t>(n) * a->Tq * a->Hq * (a->D + 1) * sizeof(float);
}

// Few outputs over short sequences: the rounding errors of P and dS do not average out over them (the norm of the
// error of a result reached 1.7 times that of rounding the result alone; 1.4 over many), and so little work does not
// fill the GPU. These calls take P and dS in two parts (backward of 256 tokens, 8 heads of 64 channels: 9.6 us against
// 8.7; of 512: 12.5 against 10.7; where the products count, 4096 tokens of one head: 49 against 37).
bool few_outputs(const lce_attn_t *a) {
    return a->Tq * a->Hq * a->D <= (1 << 18) && a->Tq <= a->B * 512 && a->Tk <= a->B * 512;
}

// The maps of one side, queries or keys. A side without tokens has none of its own and is never loaded from; the kernels
// prefetch all maps, so it gets the other side's.
lce_status_t encode_queries(AttnMaps *m, const HostDev &dev, const lce_attn_t *a, bool backward) {
    lce_status_t s = encode(&m->q, dev, a->q, a->Tq, a->Hq, a->D, a->q_ts, a->q_hs);
    if (s == LCE_OK && backward) s = encode(&m->dO, dev, a->dO, a->Tq, a->Hq, a->D, a->dO_ts, a->dO_hs);
    return s;
}
lce_status_t encode_keys(AttnMaps *m, const HostDev &dev, const lce_attn_t *a) {
    const lce_status_t s = encode(&m->k, dev, a->k, a->Tk, a->Hk, a->D, a->k_ts, a->k_hs);
    return s != LCE_OK ? s : encode(&m->v, dev, a->v, a->Tk, a->Hk, a->D, a->v_ts, a->v_hs);
}
lce_status_t encode_maps(AttnMaps *m, const HostDev &dev, const lce_attn_t *a, bool backward) {
    lce_status_t s = LCE_OK;
    if (a->Tq > 0) s = encode_queries(m, dev, a, backward);
    if (a->Tk > 0 && s == LCE_OK) s = encode_keys(m, dev, a);
    if (a->Tq == 0) m->q = m->dO = m->k;
    if (a->Tk == 0) m->k = m->v = m->q;
    return s;
}

template <int KS>
lce_status_t forward_tc(const lce_attn_t *a, const AttnArgs &r, const HostDev &dev, cudaStream_t st) {
    AttnMaps maps;
    lce_status_t s = encode_maps(&maps, dev, a, false);
    if (s != LCE_OK) return s;
    const int64_t work = r.pair_heads ? seq_slots(r.sq.T, r.sq.B, kTcTile) * (r.Hq / 2) : seq_slots(r.sq.T, r.sq.B, 2 * kTcTile) * r.Hq;
    if (r.split == 1)
        return few_outputs(a) ? launch<k_attn_fwd<KS, true, false>>(dev, work, kFwdThreads, FwdSmem<KS>::kBytes, st, r, maps)
                              : launch<k_attn_fwd<KS, false, false>>(dev, work, kFwdThreads, FwdSmem<KS>::kBytes, st, r, maps);
    s = launch<k_attn_fwd<KS, false, true>>(dev, work * r.split, kFwdThreads, FwdSmem<KS>::kBytes, st, r, maps);
    if (s != LCE_OK) return s;
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(r.sq.T) * r.Hq * 16 + kJoinThreads - 1) / kJoinThreads);
    return host_launch_early(k_attn_merge, dim3(blocks), kJoinThreads, 0, st, r);
}

// DP: channels rounded up to 32, 64 or 128 (512 tokens, 4 heads, causal, forward and backward: 32 channels 34 and 53 us,
// 64: 42 and 76, 128, or any as 128: 71 and 126).
template <int DP>
lce_status_t forward_simt(const AttnArgs &r, const HostDev &dev, cudaStream_t st) {
    const int64_t slots = seq_slots(r.sq.T, r.sq.B, kSimtTile);
    return launch<k_attn_fwd_simt<DP>>(dev, slots * r.Hq, kSimtThreads, simt_smem(DP, 3, 1), st, r);
}

// Row statistics: 16 bytes a lane, as many lanes a row as it needs (8, 16 or 32; 32 heads of 64 channels over 1024
// tokens: the backward takes 27.1 us with 8, 28.2 with 16).
template <typename T, int TILE>
lce_status_t row_stats(const AttnArgs &r, const HostDev &dev, cudaStream_t st) {
    const int64_t blocks = seq_slots(r.sq.T, r.sq.B, TILE) * r.Hq;
    const int lanes = r.D * static_cast<int>(sizeof(T)) / 16;
    if (lanes <= 8) return launch<k_attn_stats<T, TILE, 8>>(dev, blocks, kStatThreads, 0, st, r);
    if constexpr (sizeof(T) == 4)
        if (lanes > 16) return launch<k_attn_stats<T, TILE, 32>>(dev, blocks, kStatThreads, 0, st, r);
    return launch<k_attn_stats<T, TILE, 16>>(dev, blocks, kStatThreads, 0, st, r);
}

template <int DP>
lce_status_t backward_simt(const AttnArgs &r, const HostDev &dev, cudaStream_t st) {
    const int64_t dq = seq_slots(r.sq.T, r.sq.B, kSimtTile) * r.Hq, dkv = seq_slots(r.sk.T, r.sk.B, kSimtTile) * r.Hk;
    if (dq + dkv >= (int64_t(1) << 31)) return LCE_ERR_SHAPE;
    const lce_status_t s = row_stats<float, kSimtTile>(r, dev, st);
    return s != LCE_OK ? s : launch<k_attn_bwd_simt<DP>>(dev, dq + dkv, kSimtThreads, simt_smem(DP, 4, 2), st, r, static_cast<int>(dkv));
}

int stat_tile(const lce_attn_t *a) { return a->dtype == LCE_BF16 ? kTcTile : kSimtTile; }

// Shares that a dK/dV piece's query heads are split into. A piece walks the query tiles of all heads of its key head;
// where that is longer than an SM's part of all the work, shares of the heads are given to more SMs. The times compared
// are in tiles of a walk: a piece costs 3 more for its start and output, 5 with an fp32 output, and the join 3; a mask
// halves the average walk, not the longest. Of the lengths only the averages are known here. (Causal, 128 channels:
// 32 heads of 8 key heads over 512 tokens 26 us against 30, over 1024 40 against 50, of 4 over 2048 102 against 169, 8
// of 1 over 8192 295 against 631; split all the same, 28 heads of 4 over eight sequences of 256 took 59 against 32, and
// 32 of 8 over 2048 tokens 107 against 92.)
int shares(const lce_attn_t *a, bool causal) {
    const int64_t group = a->Hq / a->Hk, tq = average_tiles(a->Tq, a->B), tk = average_tiles(a->Tk, a->B);
    if (a->dtype != LCE_BF16 || group == 1 || a->Tk == 0 || a->Tk * a->Hk > (1 << 24)) return 1;
    const double kv = static_cast<double>(a->B) * tk * a->Hk, q = static_cast<double>(a->B) * tq * a->Hq, mask = causal ? 0.5 : 1.0;
    auto time = [&](int64_t n) {   // of the longest piece, or of everything shared out
        const double more = n > 1 ? 5 : 3, walk = static_cast<double>(tq * group / n);
        return std::max(walk + more, (kv * n * (walk * mask + more) + q * (tk * mask + 3)) / kSms) + (n > 1 ? 3 : 0);
    };
    int64_t best = 1;
    for (int64_t n = 2; n <= group; ++n)
        if (group % n == 0 && time(n) < 0.95 * time(best)) best = n;
    return static_cast<int>(best);
}

size_t stat_bytes(const lce_attn_t *a) {
    const size_t rows = static_cast<size_t>(seq_slots(a->Tq, a->B, stat_tile(a))) * stat_tile(a);
    return 2 * rows * static_cast<size_t>(a->Hq) * sizeof(float);
}

template <int KS>
lce_status_t backward_tc(const lce_attn_t *a, const AttnArgs &r, const HostDev &dev, cudaStream_t st) {
    const int64_t dq = seq_slots(r.sq.T, r.sq.B, kTcTile) * r.Hq, dkv = seq_slots(r.sk.T, r.sk.B, kTcTile) * r.Hk * r.split;
    if (dq + dkv >= (int64_t(1) << 31)) return LCE_ERR_SHAPE;
    AttnMaps maps;
    lce_status_t s = encode_maps(&maps, dev, a, true);
    if (s == LCE_OK) s = row_stats<__nv_bfloat16, kTcTile>(r, dev, st);
    if (s != LCE_OK) return s;
    auto go = [&](auto two, auto parts) {
        return launch<k_attn_bwd<KS, decltype(two)::value, decltype(parts)::value>, true>(dev, dq + dkv, kBwdThreads, BwdSmem<KS>::kBytes, st, r, maps,
                                                                                         static_cast<int>(dkv));
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    s = few_outputs(a) ? r.split > 1 ? go(yes, yes) : go(yes, no) : r.split > 1 ? go(no, yes) : go(no, no);
    if (s != LCE_OK || r.split == 1) return s;
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(r.sk.T) * r.Hk * 16 + kJoinThreads - 1) / kJoinThreads);
    return host_launch_early(k_attn_join, dim3(blocks, 2), kJoinThreads, 0, st, r);
}

// The tensor-core kernels exist for 64, 80, 96 and 128 channels; others run as the next of these (8192 tokens in
// sequences of 1024, causal, forward and backward: 32 heads of 64 channels 60 and 173 us, as 128 channels 69 and 222;
// 16 heads of 80: 39 and 104, 41 and 119; of 96: 40 and 109, 44 and 121).
template <typename F>
lce_status_t by_channels(int64_t D, F f) {
    if (D <= 64) return f(std::integral_constant<int, 4>());
    if (D <= 80) return f(std::integral_constant<int, 5>());
    if (D <= 96) return f(std::integral_constant<int, 6>());
    return f(std::integral_constant<int, 8>());
}

}  // namespace

extern "C" {

size_t lce_attention_workspace_size(const lce_attn_t *a) {
    if (check_shape(a) != LCE_OK) return 0;
    const int n = shares(a, true);   // the more of both masks
    return stat_bytes(a) + (n > 1 ? static_cast<size_t>(n) * 2 * a->Tk * a->Hk * a->D * sizeof(float) : 0);
}

size_t lce_attention_forward_workspace_size(const lce_attn_t *a) {
    return check_shape(a) == LCE_OK ? range_bytes(a, ranges(a)) : 0;
}

lce_status_t lce_attention_forward(const lce_attn_t *a) {
    lce_status_t s = check_common(a);
    if (s != LCE_OK) return s;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    if ((s = check_side(a->o, a->o_ts, a->o_hs, a->Tq, a->Hq, a->D, elt, true)) != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (a->Tq == 0) return LCE_OK;
    AttnArgs r = make_args(a, dev);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    r.split = ranges(a);
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    if ((s = scratch.get(a->workspace, a->workspace_bytes, range_bytes(a, r.split), &base)) != LCE_OK) return s;
    r.part = reinterpret_cast<float *>(base);
    if (a->dtype == LCE_BF16)
        return by_channels(a->D, [&](auto ks) { return forward_tc<decltype(ks)::value>(a, r, dev, st); });
    return a->D <= 32 ? forward_simt<32>(r, dev, st) : a->D <= 64 ? forward_simt<64>(r, dev, st) : forward_simt<128>(r, dev, st);
}

lce_status_t lce_attention_backward(const lce_attn_t *a) {
    lce_status_t s = check_common(a);
    if (s != LCE_OK) return s;
    const int elt = a->dtype == LCE_BF16 ? 2 : 4;
    if ((s = check_side(a->o, a->o_ts, a->o_hs, a->Tq, a->Hq, a->D, elt, false)) != LCE_OK) return s;
    if ((s = check_side(a->dO, a->dO_ts, a->dO_hs, a->Tq, a->Hq, a->D, elt, false)) != LCE_OK) return s;
    if ((s = check_side(a->dq, a->dq_ts, a->dq_hs, a->Tq, a->Hq, a->D, elt, true)) != LCE_OK) return s;
    if ((s = check_side(a->dk, a->dk_ts, a->dk_hs, a->Tk, a->Hk, a->D, elt, true)) != LCE_OK) return s;
    if ((s = check_side(a->dv, a->dv_ts, a->dv_hs, a->Tk, a->Hk, a->D, elt, true)) != LCE_OK) return s;
    HostDev dev;
    if ((s = host_device(&dev)) != LCE_OK) return s;
    if (a->Tq == 0 && a->Tk == 0) return LCE_OK;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(a->stream);
    HostScratch scratch(st);
    uint8_t *base = nullptr;
    const size_t need = lce_attention_workspace_size(a);
    if ((s = scratch.get(a->workspace, a->workspace_bytes, need, &base)) != LCE_OK) return s;
    AttnArgs r = make_args(a, dev);
    r.stat_stride = seq_slots(a->Tq, a->B, stat_tile(a)) * stat_tile(a);
    r.nlse2 = reinterpret_cast<float *>(base);
    r.ndelta = r.nlse2 + r.stat_stride * r.Hq;
    r.split = shares(a, a->causal != 0);
    r.part = reinterpret_cast<float *>(base + stat_bytes(a));
    if (a->dtype == LCE_BF16)
        return by_channels(a->D, [&](auto ks) { return backward_tc<decltype(ks)::value>(a, r, dev, st); });
    return a->D <= 32 ? backward_simt<32>(r, dev, st) : a->D <= 64 ? backward_simt<64>(r, dev, st) : backward_simt<128>(r, dev, st);
}

}  // extern "C"
