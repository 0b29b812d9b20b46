// Values in 8 bits: e4m3 codes with one power of two for a block of a row's
// channels.
#pragma once

#include <stdint.h>

#include "row_ring.cuh"

namespace lce {

constexpr int kPackBlock = 128;              // channels of a block
constexpr int kPackLow = -100, kPackHigh = 119, kPackNaN = -128;   // exponents; of a block that is not finite

// The exponent of a block whose largest magnitude has these bits: the least e
// with it <= 448 * 2^e. 448 = 1.75 * 2^8, so a mantissa up to 1.75 lies 8 below
// its own exponent, others 7.
__device__ __forceinline__ int pack_exponent(uint32_t top) {
    if (top >= 0x7f800000u) return kPackNaN;
    const int e = static_cast<int>(top >> 23) - 127 - ((top & 0x7fffffu) > 0x600000u ? 7 : 8);
    return min(max(e, kPackLow), kPackHigh);
}
__device__ __forceinline__ float pack_scale(int e) {   // 2^-e, NaN for a block that is not finite
    return e == kPackNaN ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}
__device__ __forceinline__ float unpack_scale(int e) {   // 2^e
    return e == kPackNaN ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// Two values to codes (the first in the low byte), nearest, ties to even, 448 at most.
__device__ __forceinline__ uint32_t to_codes(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// What two codes stand for without their scale.
__device__ __forceinline__ void from_codes(uint32_t codes, float &a, float &b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}" : "=f"(a), "=f"(b) : "r"(h));
}

// The bits of the largest magnitude of a block, of which this lane has the
// words `w` and each other lane of an aligned group of kLanes its own. Magnitudes
// compare as integers, bf16 ones two at a time.
template <typename T, int kWords, int kLanes>
__device__ __forceinline__ uint32_t block_top(const uint32_t (&w)[kWords]) {
    constexpr uint32_t kMask = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
    auto larger = [](uint32_t a, uint32_t b) { return sizeof(T) == 2 ? __vmaxu2(a, b) : max(a, b); };
    uint32_t top = w[0] & kMask;
#pragma unroll
    for (int i = 1; i < kWords; ++i) top = larger(top, w[i] & kMask);
#pragma unroll
    for (int m = kLanes / 2; m; m >>= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, m));
    return sizeof(T) == 2 ? max(top << 16, top & 0xffff0000u) : top;
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
    return make_uint2(to_codes(x[0] * scale, x[1] * scale) | to_codes(x[2] * scale, x[3] * scale) << 16,
                      to_codes(x[4] * scale, x[5] * scale) | to_codes(x[6] * scale, x[7] * scale) << 16);
}
__device__ __forceinline__ void values8(uint2 c, float scale, float (&x)[8]) {
    from_codes(c.x, x[0], x[1]), from_codes(c.x >> 16, x[2], x[3]);
    from_codes(c.y, x[4], x[5]), from_codes(c.y >> 16, x[6], x[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= scale;
}

// The codes of a pack's values, and from them
template <typename T>
__device__ __forceinline__ uint2 pack_codes(const f32x2 (&x)[kPack<T> / 2], float scale) {
    uint32_t c[kPack<T> / 2];
    const f32x2 f = both(scale);
#pragma unroll
    for (int i = 0; i < kPack<T> / 2; ++i) {
        float a, b;
        unpack2(mul2(x[i], f), a, b);
        c[i] = to_codes(a, b);
    }
    return sizeof(T) == 2 ? make_uint2(c[0] | c[1] << 16, c[kPack<T> / 2 - 2] | c[kPack<T> / 2 - 1] << 16) : make_uint2(c[0] | c[1] << 16, 0);
}
template <typename T>
__device__ __forceinline__ void pack_values(uint2 codes, float scale, f32x2 (&x)[kPack<T> / 2]) {
    const uint32_t w[2] = {codes.x, codes.y};   // (fp32: the first alone)
    const f32x2 f = both(scale);
#pragma unroll
    for (int i = 0; i < kPack<T> / 2; ++i) {
        float a, b;
        from_codes(w[i / 2] >> (i % 2 * 16), a, b);
        x[i] = mul2(pack2(a, b), f);
    }
}

}  // namespace lce
