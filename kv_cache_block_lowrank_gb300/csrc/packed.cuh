// packed.cuh -- the layout of the packed cache (include/hss.h) for the kernels that write and read
// it: where a token's codes and scales lie in a tile, and how a group of 32 elements is coded.
#pragma once

#include "ptx.cuh"

namespace hss {

template <int HD>
struct Tile {
    static constexpr int kGroups = HD / 32;
    static constexpr int kCodes = 8 * HD;  // bytes of the codes of K, then of V
    static constexpr int kScales = 16 * kGroups * 2;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales;
    static_assert(kBytes == 18 * HD, "as documented");
};

// (a 64-bit division is some hundred instructions, one after another)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Bytes from the cache's start to the tile that holds a slot of a head.
template <int HD>
__device__ __forceinline__ int64_t tile_at(int64_t slot, int head, int nkv, int bs) {
    const int64_t block = divide(slot, bs);
    const int in_block = static_cast<int>(slot - block * bs) / 16;
    return ((block * nkv + head) * (bs / 16) + in_block) * Tile<HD>::kBytes;
}

// Of token t's 8-element vector v: the word of K.
template <int HD>
__host__ __device__ constexpr int key_word(int t, int v) {
    return t * (HD / 2) + (v % 4) * 4 * Tile<HD>::kGroups + v / 4 * 4;
}
// Of token t's 16-element part: the byte of V with elements e (low nibble) and e + 8.
template <int HD>
__host__ __device__ constexpr int value_byte(int t, int part, int e) {
    return Tile<HD>::kCodes + (part / 4 * 32 + e * 4 + t % 8 / 2) * 16 + part % 4 * 4 + t % 2 * 2 +
           t / 8;
}
template <int HD>
__host__ __device__ constexpr int key_scale(int t, int group) {
    return 2 * Tile<HD>::kCodes + (t * Tile<HD>::kGroups + group) * 2;
}
template <int HD>
__host__ __device__ constexpr int value_scale(int t, int group) {
    return key_scale<HD>(t, group) + Tile<HD>::kScales;
}

// The scale (bf16 bits) of a group whose 32 elements four neighbouring lanes hold, 8 each: a
// seventh of the largest in fp32, rounded to bf16; NaN where an element is not finite.  All lanes
// of the warp take part.
__device__ __forceinline__ uint32_t group_scale(const uint4& x) {
    uint32_t most = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                             __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
    most = max(most & 0xFFFFu, most >> 16);
    if (most >= 0x7F80u) return 0x7FC0u;
    const float s = __fdiv_rn(__uint_as_float(most << 16), 7.0f);
    return pack_bf16x2(s, 0.0f) & 0xFFFFu;
}

// group_codes for scales whose reciprocal might not be a number, by division.
static __device__ __noinline__ uint32_t group_codes_tiny(const uint4 x, uint32_t scale) {
    const float s = __uint_as_float(scale << 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t codes = 0;
    for (int i = 0; i < 8; ++i) {
        const uint32_t half = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
        const int c = __float2int_rn(__fdiv_rn(__uint_as_float(half << 16), s));
        codes |= static_cast<uint32_t>(max(-7, min(7, c)) + 8) << (4 * i);
    }
    return codes;
}

// The codes + 8 of 8 elements, nibble by nibble: rint(x / scale), ties to even, without a division
// for each.  x and the scale have 8 bits each, so a quotient within 2^-16 of a half is one, and x
// times the scale's reciprocal is nearer than that: what it rounds to is right but for exact halves,
// and those the remainder shows, which is exact.
__device__ __forceinline__ uint32_t group_codes(const uint4& x, uint32_t scale) {
    if (scale == 0 || scale >= 0x7F80u) return 0x88888888u;
    const float s = __uint_as_float(scale << 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t codes = 0;
    if (scale < 0x0800u) return group_codes_tiny(x, scale);  // below 2^-111
    // Adding 1.5 2^23 leaves the rounded quotient in a float's low bits.
    constexpr float kAdd = 12582912.0f;
    constexpr uint32_t kAddBits = 0x4B400000u;
    const float inverse = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        uint32_t q = __float_as_uint(fmaf(e, inverse, kAdd));
        const float rest = fmaf(kAdd - __uint_as_float(q), s, e);
        if (fabsf(rest) * 2.0f == s && (q & 1)) q += rest > 0.0f ? 1u : ~0u;
        codes += q << (4 * i);
    }
    // (every nibble holds its code, with what was added to all of them taken away and 8 added)
    return codes - kAddBits * 0x11111111u + 0x88888888u;
}

}  // namespace hss
