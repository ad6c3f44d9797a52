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

// Bytes from the cache's start to the tile that holds a slot of a head.
template <int HD>
__device__ __forceinline__ int64_t tile_at(int64_t slot, int head, int nkv, int bs) {
    const int64_t block = slot / bs;
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

// The codes + 8 of 8 elements, nibble by nibble.
__device__ __forceinline__ uint32_t group_codes(const uint4& x, uint32_t scale) {
    if (scale == 0 || scale >= 0x7F80u) return 0x88888888u;
    const float s = __uint_as_float(scale << 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        const int c = max(-7, min(7, __float2int_rn(__fdiv_rn(e, s))));
        codes |= static_cast<uint32_t>(c + 8) << (4 * i);
    }
    return codes;
}

}  // namespace hss
