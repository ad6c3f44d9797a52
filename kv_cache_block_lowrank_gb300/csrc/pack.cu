// pack.cu -- tokens into and out of the packed cache (include/hss.h has its layout).
//
// A group of 32 elements is four neighbouring lanes of a warp, 8 elements (16 bytes) each: its
// largest element takes two shuffles, and codes follow from an IEEE division, so that every
// packing of a row gives the same bits.  Of K a lane's 8 codes are one 32-bit word of the page.  Of
// V they are nibbles of 8 bytes; neighbouring lanes hold the two nibbles of a byte, and exchange
// halves so that each writes four whole bytes.
#include <cuda_runtime.h>

#include "packed.cuh"

namespace hss {
namespace {

constexpr int kThreads = 256;

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
    int32_t* dev_status;
    int32_t* lib_error;
};

// What the lanes work through: 8-element vectors, of a token's heads first of K (if wanted), then V.
template <int HD>
struct Item {
    int64_t token;
    int vec;     // of the head
    int head;
    bool value;  // V
    __device__ __forceinline__ Item(int64_t i, int heads, int nkv, bool keys) {
        constexpr int kVecs = HD / 8;
        vec = static_cast<int>(i % kVecs);
        const int64_t row = i / kVecs;
        head = static_cast<int>(row % heads);
        token = row / heads;
        value = !keys || head >= nkv;
        if (head >= nkv) head -= nkv;
    }
};

template <int HD>
__global__ void __launch_bounds__(kThreads) pack_kernel(const PackParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const bool keys = p.K != nullptr, values = p.V != nullptr;
    const int heads = (keys ? p.nkv : 0) + (values ? p.nkv : 0);
    const int64_t total = p.tokens * heads * (HD / 8);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    // (a row's vectors are a multiple of eight, so a group's lanes are all in or all out)
    const Item<HD> it(i < total ? i : 0, heads, p.nkv, keys);
    int64_t slot = i < total ? __ldg(p.slots + it.token) : -1;
    if (slot >= p.cache_tokens) {
        if (it.vec == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        slot = -1;
    }
    uint4 x = make_uint4(0, 0, 0, 0);
    if (slot >= 0) {
        const uint16_t* row = it.value ? p.V + it.token * p.v_stride : p.K + it.token * p.k_stride;
        x = __ldg(reinterpret_cast<const uint4*>(row + it.head * HD + 8 * it.vec));
    }
    const uint32_t scale = group_scale(x);
    const uint32_t codes = group_codes(x, scale);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
    if (slot < 0) return;
    uint8_t* tile = p.cache + tile_at<HD>(slot, it.head, p.nkv, p.bs);
    const int t = static_cast<int>(slot % 16), group = it.vec / 4;
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

template <int HD>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const PackParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const bool keys = p.K_out != nullptr, values = p.V_out != nullptr;
    const int heads = (keys ? p.nkv : 0) + (values ? p.nkv : 0);
    const int64_t total = p.tokens * heads * (HD / 8);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= total) return;
    const Item<HD> it(i, heads, p.nkv, keys);
    const int64_t slot = __ldg(p.slots + it.token);
    if (slot < 0) return;
    if (slot >= p.cache_tokens) {
        if (it.vec == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        return;
    }
    const uint8_t* tile = p.cache + tile_at<HD>(slot, it.head, p.nkv, p.bs);
    const int t = static_cast<int>(slot % 16), group = it.vec / 4;
    uint32_t codes = 0;
    uint16_t scale;
    if (!it.value) {
        codes = *reinterpret_cast<const uint32_t*>(tile + key_word<HD>(t, it.vec));
        scale = *reinterpret_cast<const uint16_t*>(tile + key_scale<HD>(t, group));
    } else {
        const int shift = (it.vec & 1) * 4;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            codes |= ((static_cast<uint32_t>(tile[value_byte<HD>(t, it.vec / 2, e)]) >> shift) & 15u)
                     << (4 * e);
        scale = *reinterpret_cast<const uint16_t*>(tile + value_scale<HD>(t, group));
    }
    const float s = __uint_as_float(static_cast<uint32_t>(scale) << 16);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        y[e] = static_cast<float>(static_cast<int>((codes >> (4 * e)) & 15u) - 8) * s;
    uint16_t* row = it.value ? p.V_out + it.token * p.v_stride : p.K_out + it.token * p.k_stride;
    *reinterpret_cast<uint4*>(row + it.head * HD + 8 * it.vec) =
        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                   pack_bf16x2(y[6], y[7]));
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
    const int hd = a.dims.head_dim;
    const int64_t items = a.num_tokens * halves * p.nkv * (hd / 8);
    const int64_t ctas = (items + kThreads - 1) / kThreads;
    if (ctas > 0x7FFFFFFF) return HSS_ERR_INVALID_ARGUMENT;
    auto kern = hd == 64    ? (unpack ? unpack_kernel<64> : pack_kernel<64>)
                : hd == 128 ? (unpack ? unpack_kernel<128> : pack_kernel<128>)
                : hd == 192 ? (unpack ? unpack_kernel<192> : pack_kernel<192>)
                            : (unpack ? unpack_kernel<256> : pack_kernel<256>);
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, p) ==
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
    p.cache = cache;
    return run(a, p, false, (K != nullptr) + (V != nullptr), stream);
}

hss_status launch_unpack(const hss_pack_args& a, const uint8_t* cache, uint16_t* K, uint16_t* V,
                         cudaStream_t stream) {
    PackParams p = {};
    p.K_out = K;
    p.V_out = V;
    p.cache = const_cast<uint8_t*>(cache);
    return run(a, p, true, (K != nullptr) + (V != nullptr), stream);
}

}  // namespace hss
