// pack.cu -- tokens into and out of the packed cache (include/hss.h has its layout).
//
// A group of 32 elements is four neighbouring lanes of a warp, 8 elements (16 bytes) each: its
// largest element takes two shuffles, and codes are the exactly rounded quotients (packed.cuh has
// how, mostly without a division), so that every packing of a row gives the same bits.  Of K a lane's 8 codes are one 32-bit word of the page.  Of
// V they are nibbles of 8 bytes; neighbouring lanes hold the two nibbles of a byte, and exchange
// halves so that each writes four whole bytes.
//
// Many tokens: 16 in a row that fill a tile are taken together by a CTA, a warp to a head's K or V,
// and go out (or come in) as whole 16-byte pieces of the page; V's bytes, which hold a token each,
// change places with the elements in shared memory.  What else there is goes token by token.
//
// What bounds it: few tokens, the launch (64 tokens 4 us to pack and 4 to read back); many, latency: a
// warp has a tile's rows in two goes of four loads and picks V's nibbles one by one.  8191 tokens of 8
// heads of 128, packed and read back, 33 us for 86 MB, 2.6 TB/s (apart, from graphs, 24.6 and 16.4);
// ncu shows 62 % of the issue rate and 40 % of the warps there can be.
#include <cuda_runtime.h>

#include "packed.cuh"

namespace hss {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kWindowTokens = 4096;
constexpr int kWindowElements = 1024;  // of a token, in the heads that are asked for

struct PackParams {
    const uint16_t* K;
    const uint16_t* V;
    uint16_t* K_out;
    uint16_t* V_out;
    uint8_t* cache;
    const int64_t* slots;
    int64_t tokens;
    int64_t k_stride, v_stride;
    int64_t cache_tokens;
    int bs;
    int nkv;
    int heads;  // of K, if it is wanted, and then of V
    bool keys;
    int32_t* dev_status;
    int32_t* lib_error;
};

// What the lanes work through: 8-element vectors, of a token's heads first of K (if wanted), then V.
template <int HD>
struct Item {
    static constexpr int kVecs = HD / 8;
    int64_t token;
    int vec;     // of the head
    int head;
    bool value;  // V
    // Vector i of all tokens', or of one token's heads from h0 on.
    __device__ __forceinline__ Item(int64_t i, const PackParams& p) {
        const int64_t row = divide(i, kVecs);
        vec = static_cast<int>(i - row * kVecs);
        token = divide(row, p.heads);
        choose(static_cast<int>(row - token * p.heads), p);
    }
    __device__ __forceinline__ Item(int64_t of, int h0, int i, const PackParams& p) {
        vec = i % kVecs;
        token = of;
        choose(h0 + i / kVecs, p);
    }
    __device__ __forceinline__ void choose(int h, const PackParams& p) {
        value = !p.keys || h >= p.nkv;
        head = h >= p.nkv ? h - p.nkv : h;
    }
};

// One lane's 8 elements.  All lanes of the warp come here (slot < 0: with nothing to do), the four of
// a group with the same slot.
template <int HD>
__device__ __forceinline__ uint4 load_vector(const PackParams& p, const Item<HD>& it,
                                             int64_t slot) {
    if (slot < 0 || slot >= p.cache_tokens) return make_uint4(0, 0, 0, 0);
    const uint16_t* row = it.value ? p.V + it.token * p.v_stride : p.K + it.token * p.k_stride;
    return __ldg(reinterpret_cast<const uint4*>(row + it.head * HD + 8 * it.vec));
}
template <int HD>
__device__ __forceinline__ void pack_vector(const PackParams& p, const Item<HD>& it, int64_t slot,
                                            const uint4& x) {
    if (slot >= p.cache_tokens) {
        if (it.vec == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        slot = -1;
    }
    const uint32_t scale = group_scale(x);
    const uint32_t codes = group_codes(x, scale);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
    if (slot < 0) return;
    uint8_t* tile = p.cache + tile_at<HD>(slot, it.head, p.nkv, p.bs);
    const int t = static_cast<int>(slot) & 15, group = it.vec / 4;
    if (!it.value) {
        *reinterpret_cast<uint32_t*>(tile + key_word<HD>(t, it.vec)) = codes;
        if (it.vec % 4 == 0)
            *reinterpret_cast<uint16_t*>(tile + key_scale<HD>(t, group)) =
                static_cast<uint16_t>(scale);
    } else {
        // elements e of the even lane and of the odd one: low and high nibble of byte e
        const int odd = it.vec & 1;
        const uint32_t lo = odd ? other : codes, hi = odd ? codes : other;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = 4 * odd + k;
            tile[value_byte<HD>(t, it.vec / 2, e)] =
                static_cast<uint8_t>(((lo >> (4 * e)) & 15u) | (((hi >> (4 * e)) & 15u) << 4));
        }
        if (it.vec % 4 == 0)
            *reinterpret_cast<uint16_t*>(tile + value_scale<HD>(t, group)) =
                static_cast<uint16_t>(scale);
    }
}

// Eight codes times a scale (bf16 bits), rounded once to bf16.
__device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t scale) {
    const float s = __uint_as_float(scale << 16);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        y[e] = static_cast<float>(static_cast<int>((codes >> (4 * e)) & 15u) - 8) * s;
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
}

// The codes of token t's 8-element vector v of V, from the tile's codes of V.
__device__ __forceinline__ uint32_t value_codes(const uint8_t* codes_of_v, int t, int v) {
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        codes |= ((static_cast<uint32_t>(
                       codes_of_v[(v / 8 * 32 + e * 4 + t % 8 / 2) * 16 + v / 2 % 4 * 4 +
                                  t % 2 * 2 + t / 8]) >> (v % 2 * 4)) & 15u) << (4 * e);
    return codes;
}

template <int HD>
__device__ __forceinline__ void unpack_vector(const PackParams& p, const Item<HD>& it,
                                              int64_t slot) {
    if (slot < 0) return;
    if (slot >= p.cache_tokens) {
        if (it.vec == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        return;
    }
    const uint8_t* tile = p.cache + tile_at<HD>(slot, it.head, p.nkv, p.bs);
    const int t = static_cast<int>(slot) & 15, group = it.vec / 4;
    uint32_t codes;
    uint16_t scale;
    if (!it.value) {
        codes = *reinterpret_cast<const uint32_t*>(tile + key_word<HD>(t, it.vec));
        scale = *reinterpret_cast<const uint16_t*>(tile + key_scale<HD>(t, group));
    } else {
        codes = value_codes(tile + Tile<HD>::kCodes, t, it.vec);
        scale = *reinterpret_cast<const uint16_t*>(tile + value_scale<HD>(t, group));
    }
    uint16_t* row = it.value ? p.V_out + it.token * p.v_stride : p.K_out + it.token * p.k_stride;
    *reinterpret_cast<uint4*>(row + it.head * HD + 8 * it.vec) = values_of(codes, scale);
}

// Token by token: a lane an 8-element vector.  (A row's vectors are a multiple of eight, so a
// group's lanes are all in or all out.)
template <int HD, bool UNPACK>
__global__ void __launch_bounds__(kThreads) single_kernel(const PackParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t total = p.tokens * p.heads * (HD / 8);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const Item<HD> it(i < total ? i : 0, p);
    const int64_t slot = i < total ? __ldg(p.slots + it.token) : -1;
    if constexpr (UNPACK)
        unpack_vector<HD>(p, it, slot);
    else
        pack_vector<HD>(p, it, slot, load_vector<HD>(p, it, slot));
}

// A tile that 16 tokens in a row fill, from token `first` on: K or V of one head, by a warp.
template <int HD>
__device__ __forceinline__ void pack_tile(const PackParams& p, int64_t first, uint8_t* tile,
                                          int head, bool value, uint32_t (*codes)[HD / 8 + 2]) {
    constexpr int NG = Tile<HD>::kGroups;
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int t = 8 * half + lane / 4;
        const uint16_t* row = value ? p.V + (first + t) * p.v_stride : p.K + (first + t) * p.k_stride;
        uint4 x[NG];
        uint32_t word[NG], scale[NG];
#pragma unroll
        for (int G = 0; G < NG; ++G)
            x[G] = __ldg(reinterpret_cast<const uint4*>(row + head * HD + 8 * (4 * G + c)));
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            scale[G] = group_scale(x[G]);
            word[G] = group_codes(x[G], scale[G]);
        }
        if (value) {
#pragma unroll
            for (int G = 0; G < NG; ++G) codes[t][4 * G + c] = word[G];
        } else {
            uint2* to = reinterpret_cast<uint2*>(tile + key_word<HD>(t, c));
#pragma unroll
            for (int G = 0; G < NG; G += 2) to[G / 2] = make_uint2(word[G], word[G + 1]);
        }
        if (c == 0) {
            uint32_t* to = reinterpret_cast<uint32_t*>(
                tile + (value ? value_scale<HD>(t, 0) : key_scale<HD>(t, 0)));
#pragma unroll
            for (int G = 0; G < NG; G += 2) to[G / 2] = scale[G] | scale[G + 1] << 16;
        }
    }
    if (!value) return;
    __syncwarp();
    const int shift = lane / 4 * 4;
#pragma unroll
    for (int q = 0; q < HD / 64; ++q) {
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            out[i] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // byte k: token 2 c + k / 2 + 8 (k % 2)
                const uint2 w = *reinterpret_cast<const uint2*>(
                    &codes[2 * c + k / 2 + 8 * (k % 2)][2 * (4 * q + i)]);
                const uint32_t byte = ((w.x >> shift) & 15u) | ((w.y >> shift) & 15u) << 4;
                out[i] |= byte << (8 * k);
            }
        }
        *reinterpret_cast<uint4*>(tile + Tile<HD>::kCodes + (q * 32 + lane) * 16) =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncwarp();
}

template <int HD>
__device__ __forceinline__ void unpack_tile(const PackParams& p, int64_t first,
                                            const uint8_t* tile, int head, bool value,
                                            uint32_t (*staged)[HD / 8 + 2]) {
    constexpr int NG = Tile<HD>::kGroups;
    const int lane = threadIdx.x & 31, c = lane & 3;
    uint8_t* codes_of_v = reinterpret_cast<uint8_t*>(staged);
    if (value) {
#pragma unroll
        for (int q = 0; q < HD / 64; ++q)
            reinterpret_cast<uint4*>(codes_of_v)[q * 32 + lane] = *reinterpret_cast<const uint4*>(
                tile + Tile<HD>::kCodes + (q * 32 + lane) * 16);
        __syncwarp();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = 8 * half + lane / 4;
        uint16_t* row =
            value ? p.V_out + (first + t) * p.v_stride : p.K_out + (first + t) * p.k_stride;
        const uint32_t* scale = reinterpret_cast<const uint32_t*>(
            tile + (value ? value_scale<HD>(t, 0) : key_scale<HD>(t, 0)));
        const uint32_t* word = reinterpret_cast<const uint32_t*>(tile + key_word<HD>(t, c));
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            const uint32_t codes = value ? value_codes(codes_of_v, t, 4 * G + c) : word[G];
            *reinterpret_cast<uint4*>(row + head * HD + 8 * (4 * G + c)) =
                values_of(codes, G & 1 ? scale[G / 2] >> 16 : scale[G / 2] & 0xFFFFu);
        }
    }
    __syncwarp();
}

// Many tokens: the CTAs (x, 0 .. kShares - 1) have the tokens 16 x .. 16 x + 15: of a run that begins
// there a share of the heads, of tokens in no run a share of the tokens.
constexpr int kShares = 4;
constexpr int kWindowThreads = 128;

template <int HD, bool UNPACK>
__global__ void __launch_bounds__(kWindowThreads) window_kernel(const PackParams p) {
    __shared__ int64_t slots[48];  // of the tokens 16 x - 15 ..
    __shared__ alignas(16) uint32_t codes[kWindowThreads / 32][16][HD / 8 + 2];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x < 46) {
        const int64_t i = t0 - 15 + threadIdx.x;
        slots[threadIdx.x] = i >= 0 && i < p.tokens ? __ldg(p.slots + i) : -1;
    }
    __syncthreads();
    // Bit k: the tokens from t0 - 15 + k on fill a tile.
    bool fills = false;
    if (lane < 31) {
        const int64_t s = slots[lane];
        fills = s >= 0 && s % 16 == 0 && s + 15 < p.cache_tokens;
#pragma unroll
        for (int k = 1; k < 16; ++k) fills = fills && slots[lane + k] == s + k;
    }
    const uint32_t runs = __ballot_sync(0xffffffffu, fills);
    // A run that begins among this CTA's tokens (there is one at most) is its own.
    const int begin = __ffs(runs >> 15) - 1;
    if (begin >= 0) {
        const int64_t slot = slots[15 + begin];
        for (int h = kShares * warp + blockIdx.y; h < p.heads; h += kShares * (kWindowThreads / 32)) {
            const bool value = !p.keys || h >= p.nkv;
            const int head = h >= p.nkv ? h - p.nkv : h;
            uint8_t* tile = p.cache + tile_at<HD>(slot, head, p.nkv, p.bs);
            if constexpr (UNPACK)
                unpack_tile<HD>(p, t0 + begin, tile, head, value, codes[warp]);
            else
                pack_tile<HD>(p, t0 + begin, tile, head, value, codes[warp]);
        }
    }
    // Tokens in no run, two at a time, whose loads are on their way together.
    constexpr int kAtOnce = 2;
#pragma unroll 1
    for (int t = 16 / kShares * blockIdx.y; t < 16 / kShares * (blockIdx.y + 1); t += kAtOnce) {
        uint32_t wanted = 0;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (slots[15 + t + u] >= 0 && ((runs >> (t + u)) & 0xFFFFu) == 0) wanted |= 1u << u;
        if (wanted == 0) continue;
        const int n = p.heads * (HD / 8);
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kWindowThreads) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            auto item = [&](int u) { return Item<HD>(t0 + t + u, 0, i < n ? i : 0, p); };
            auto slot = [&](int u) {
                return i < n && ((wanted >> u) & 1) ? slots[15 + t + u] : -1;
            };
            if constexpr (UNPACK) {
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) unpack_vector<HD>(p, item(u), slot(u));
            } else {
                uint4 x[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) x[u] = load_vector<HD>(p, item(u), slot(u));
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) pack_vector<HD>(p, item(u), slot(u), x[u]);
            }
        }
    }
}

template <int HD>
auto kernel_for(bool unpack, bool windows) {
    return windows ? (unpack ? window_kernel<HD, true> : window_kernel<HD, false>)
                   : (unpack ? single_kernel<HD, true> : single_kernel<HD, false>);
}

hss_status run(const hss_pack_args& a, PackParams p, bool unpack, int halves,
               cudaStream_t stream) {
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    p.slots = a.slots;
    p.tokens = a.num_tokens;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.cache_tokens = a.dims.max_blocks * a.dims.block_size;
    p.bs = a.dims.block_size;
    p.nkv = a.dims.num_kv_heads;
    p.dev_status = a.dev_status;
    p.lib_error = dev->error_word;
    p.heads = halves * p.nkv;
    const int hd = a.dims.head_dim;
    // Whole tiles only where there are CTAs and heads enough to hide how long one takes.  Packed so, and
    // token by token (K and V, from graphs, us): 8 heads of 128: 2048 tokens 13.0 and 10.2, 4096 15.1
    // and 15.7, 8191 24.5 and 26.7, 16384 40.9 and 49.2; 4 heads of 128: 4096 10.9 and 10.3, 16384 28.5
    // and 26.8; 2 heads: 16384 21.4 and 16.0; 1 head 17.1 and 10.3; 8 heads of 64: 8191 14.3 and 15.0;
    // 3 of 192: 16384 32.4 and 32.8.  Read back: 8 heads of 128: 4096 11.4 and 12.2, 16384 26.0 and 35.0.
    const bool windows = p.tokens >= kWindowTokens && p.heads * hd >= kWindowElements;
    dim3 grid;
    if (windows) {
        grid = dim3(static_cast<unsigned>((p.tokens + 15) / 16), kShares);
    } else {
        grid = dim3(static_cast<unsigned>(
            (p.tokens * p.heads * (hd / 8) + kThreads - 1) / kThreads));
    }
    auto kern = hd == 64    ? kernel_for<64>(unpack, windows)
                : hd == 128 ? kernel_for<128>(unpack, windows)
                : hd == 192 ? kernel_for<192>(unpack, windows)
                            : kernel_for<256>(unpack, windows);
    return launch_pdl(kern, grid, dim3(windows ? kWindowThreads : kThreads), 0, stream, p) ==
                   cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

}  // namespace

hss_status launch_pack(const hss_pack_args& a, const uint16_t* K, const uint16_t* V,
                       uint8_t* cache, cudaStream_t stream) {
    PackParams p = {};
    p.K = K;
    p.V = V;
    p.keys = K != nullptr;
    p.cache = cache;
    return run(a, p, false, (K != nullptr) + (V != nullptr), stream);
}

hss_status launch_unpack(const hss_pack_args& a, const uint8_t* cache, uint16_t* K, uint16_t* V,
                         cudaStream_t stream) {
    PackParams p = {};
    p.K_out = K;
    p.V_out = V;
    p.keys = K != nullptr;
    p.cache = const_cast<uint8_t*>(cache);
    return run(a, p, true, (K != nullptr) + (V != nullptr), stream);
}

}  // namespace hss
