// norm_rope.cu -- root-mean-square norm of every query and key head, rotary positions, and the
// paged cache write, in one pass.
//
// y = x / sqrt(mean x^2 + eps) * (w + offset) over the head, then the first rot_dim elements turn
// in pairs by the position's angles (rope.cu has the angles' arithmetic).  A head belongs to a few
// neighbouring lanes of a warp: each holds whole 16-byte vectors in registers, in pairs that hold
// the two ends of the rotated pairs, the sum of squares takes log2(lanes) shuffles, and norm, turn
// and store follow without the element leaving its register.  Everything is fp32 until the one
// rounding at the end.
//
// What bounds it: few tokens, the launch (16 tokens 4.8 us); many, HBM and the instructions beside
// it: 8192 tokens of 64 + 8 turned heads of 128, each with weights, 59 to 62 us, 5.4 TB/s, 80 % of the
// copy rate; 1070 instructions a warp and token, issued at 66 % of the rate (ncu).  Four CTAs of 256
// threads an SM by the registers (64) and four items a thread in flight: with 80 registers 66 us, two
// items and 320 threads 63, one and 640 70.  Packed fp32 operations changed nothing (64).
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace hss {
namespace {

constexpr int kMostThreads = 256;
constexpr float kSmallest = 0x1p-100f;  // of a mean square whose bits are all there

enum RopeMode { kInterleaved, kHalf, kHalfOdd };

// A head's vectors are dealt to kLanes lanes, kPairs pairs of vectors to each.  192 elements are
// 12 pairs: four lanes of three, so that a head's lanes stay a power of two.
template <int HD>
struct Deal {
    static constexpr int kLanes = HD == 192 ? 4 : HD / 16;
    static constexpr int kPairs = HD / 16 / kLanes;
    static constexpr int kBatch = kPairs == 1 ? 4 : 1;  // items in flight per thread
};

struct NormParams {
    const uint16_t* Q;
    const uint16_t* K;
    const uint16_t* V;
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    uint16_t* Q_out;
    uint16_t* K_out;
    uint16_t* K_cache;
    uint16_t* V_cache;
    const uint64_t* turns;
    const int64_t* positions;
    const int64_t* slots;
    int64_t q_stride, k_stride, v_stride;
    int64_t q_weight_stride, k_weight_stride;
    int64_t cache_tokens;
    float magnitude, eps, offset;
    int rot;
    int q_heads;  // query heads to turn (0: none), then kv heads to turn, then values to copy
    int k_heads;
    int v_heads;
    int nkv;
    int split_items;  // items (a lane of a head) of one CTA of a token
    int32_t* dev_status;
    int32_t* lib_error;
};

// The vectors of pair j (of head_dim / 16) of a head.
template <int HD, int MODE>
__device__ __forceinline__ void pair_vectors(int j, int rot, int& v0, int& v1) {
    if constexpr (MODE == kHalf) {
        const int pairs = rot / 16;  // vectors (j, j + pairs) hold the two ends of 8 pairs
        v0 = j < pairs ? j : 2 * j;
        v1 = j < pairs ? j + pairs : 2 * j + 1;
    } else {
        v0 = j;
        v1 = j + HD / 16;
    }
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = low(w[i]);
        x[2 * i + 1] = high(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}
// Both of a word times 2^100, which is exact.
__device__ __forceinline__ uint32_t raise2(uint32_t u) {
    return pack_bf16x2(low(u) * 0x1p100f, high(u) * 0x1p100f);
}
__device__ __forceinline__ uint4 raise8(const uint4& u) {
    return make_uint4(raise2(u.x), raise2(u.y), raise2(u.z), raise2(u.w));
}
__device__ __forceinline__ float sum_squares(const uint4& u, float s) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(low(w[i]), low(w[i]), s);
        s = fmaf(high(w[i]), high(w[i]), s);
    }
    return s;
}

// Vector v of a head, normed: x (w inv + offset), with the offset times inv already.
__device__ __forceinline__ void scale8(float* x, float inv, const uint16_t* weight, int v,
                                       float offset) {
    if (weight == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
    } else {
        float w[8];
        unpack8(load16(weight + 8 * v), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= fmaf(w[e], inv, offset);
    }
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = a;
    a = x * c - b * s;
    b = b * c + x * s;
}

__device__ __forceinline__ void turn_interleaved(float* x, int v, int rot, const float2* cs) {
    if (8 * v + 8 <= rot) {
        const float4 c0 = *reinterpret_cast<const float4*>(cs + 4 * v);
        const float4 c1 = *reinterpret_cast<const float4*>(cs + 4 * v + 2);
        turn_pair(x[0], x[1], c0.x, c0.y);
        turn_pair(x[2], x[3], c0.z, c0.w);
        turn_pair(x[4], x[5], c1.x, c1.y);
        turn_pair(x[6], x[7], c1.z, c1.w);
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (8 * v + 2 * e < rot)
            turn_pair(x[2 * e], x[2 * e + 1], cs[4 * v + e].x, cs[4 * v + e].y);
}

__device__ __forceinline__ void turn_half(float* x, float* y, int j, const float2* cs) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float4 c = *reinterpret_cast<const float4*>(cs + 8 * j + e);
        turn_pair(x[e], y[e], c.x, c.y);
        turn_pair(x[e + 1], y[e + 1], c.z, c.w);
    }
}

// Half layout whose halves are not whole vectors: each element's partner is fetched by itself,
// and normed here.
__device__ __forceinline__ void turn_half_odd(float* x, const uint16_t* head,
                                              const uint16_t* weight, float up, float inv,
                                              float offset, int v, int rot, const float2* cs) {
    const int half = rot / 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = 8 * v + e;
        if (i >= rot) break;
        const bool first = i < half;
        const int other = first ? i + half : i - half;
        float o = __uint_as_float(static_cast<uint32_t>(__ldg(head + other)) << 16) * up * inv;
        if (weight != nullptr)
            o *= __uint_as_float(static_cast<uint32_t>(__ldg(weight + other)) << 16) + offset;
        const float2 c = cs[first ? i : other];
        x[e] = first ? x[e] * c.x - o * c.y : x[e] * c.x + o * c.y;
    }
}

// SMALL: eps is below kSmallest, so that a head's mean square may be.
template <int HD, int MODE, bool SMALL>
__global__ void __launch_bounds__(kMostThreads, 4) norm_rope_kernel(const NormParams p) {
    using D = Deal<HD>;
    constexpr int kLanes = D::kLanes, kPairs = D::kPairs, kBatch = D::kBatch;
    const int threads = static_cast<int>(blockDim.x);
    __shared__ alignas(16) float2 cs[128];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t token = blockIdx.x;
    const int total = (p.q_heads + p.k_heads + p.v_heads) * kLanes;
    const int begin = blockIdx.y * p.split_items;
    const int end = min(total, begin + p.split_items);
    const uint16_t* q = p.Q + token * p.q_stride;
    const uint16_t* k = p.K + token * p.k_stride;
    const uint16_t* v = p.V + token * p.v_stride;
    const bool turns = p.q_heads + p.k_heads > 0;
    int64_t pos = 0, slot = -1;
    if (turns) pos = __ldg(p.positions + token);
    if (p.slots != nullptr) slot = __ldg(p.slots + token);

    bool ready = false;
    for (int base = begin; base < end; base += threads * kBatch) {
        uint4 x[kBatch][kPairs][2];
        const uint16_t* head[kBatch];
        const int l = static_cast<int>(threadIdx.x) % kLanes;  // (items begin at a head's first)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int item = base + u * threads + static_cast<int>(threadIdx.x);
            const int h = item / kLanes;
            head[u] = h < p.q_heads               ? q + h * HD
                      : h < p.q_heads + p.k_heads ? k + (h - p.q_heads) * HD
                                                  : v + (h - p.q_heads - p.k_heads) * HD;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                int v0, v1;
                pair_vectors<HD, MODE>(l + i * kLanes, p.rot, v0, v1);
                const bool in = item < end;
                x[u][i][0] = in ? load16(head[u] + 8 * v0) : make_uint4(0, 0, 0, 0);
                x[u][i][1] = in ? load16(head[u] + 8 * v1) : make_uint4(0, 0, 0, 0);
            }
        }
        if (!ready) {
            for (int i = threadIdx.x; turns && i < p.rot / 2; i += threads) {
                const uint64_t a = static_cast<uint64_t>(pos) * __ldg(p.turns + i);
                // a signed fraction of a turn in 2^-32, so half turns in 2^-31
                const float x2 =
                    static_cast<float>(static_cast<int32_t>(a >> 32)) * (1.0f / 2147483648.0f);
                float s, c;
                sincospif(x2, &s, &c);
                cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
            }
            __syncthreads();
            ready = true;
            if (slot >= p.cache_tokens) {
                if (threadIdx.x == 0 && blockIdx.y == 0)
                    raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
                slot = -1;
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int item = base + u * threads + static_cast<int>(threadIdx.x);
            const int h = item / kLanes;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                sum = sum_squares(x[u][i][1], sum_squares(x[u][i][0], sum));
            // (by all lanes of the warp: a head's are neighbours, and what is past the end is 0)
#pragma unroll
            for (int m = 1; m < kLanes; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            const bool turned = h < p.q_heads + p.k_heads;
            float inv = rsqrtf(sum * (1.0f / HD) + p.eps);
            bool tiny = false;
            if constexpr (SMALL) {
                // A head may be so small that its squares lose their bits, or are 0: its elements are
                // then taken times 2^100 (below 2^-46 they all are), eps times 2^200.
                tiny = item < end && turned && sum * (1.0f / HD) + p.eps < kSmallest;
                if (__any_sync(0xffffffffu, tiny)) {
                    sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        if (tiny) {
                            x[u][i][0] = raise8(x[u][i][0]);
                            x[u][i][1] = raise8(x[u][i][1]);
                            sum = sum_squares(x[u][i][1], sum_squares(x[u][i][0], sum));
                        }
                    }
#pragma unroll
                    for (int m = 1; m < kLanes; m <<= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    if (tiny) inv = rsqrtf(sum * (1.0f / HD) + p.eps * 0x1p100f * 0x1p100f);
                }
            }
            if (item >= end) continue;
            const uint16_t* weight =
                h < p.q_heads ? (p.q_weight == nullptr ? nullptr : p.q_weight + h * p.q_weight_stride)
                              : (p.k_weight == nullptr
                                     ? nullptr
                                     : p.k_weight + (h - p.q_heads) * p.k_weight_stride);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const int j = l + i * kLanes;
                int v0, v1;
                pair_vectors<HD, MODE>(j, p.rot, v0, v1);
                if (turned) {
                    float a[8], b[8];
                    unpack8(x[u][i][0], a);
                    unpack8(x[u][i][1], b);
                    scale8(a, inv, weight, v0, p.offset * inv);
                    scale8(b, inv, weight, v1, p.offset * inv);
                    if constexpr (MODE == kHalf) {
                        if (j < p.rot / 16) {
                            turn_half(a, b, j, cs);
                        }
                    } else if constexpr (MODE == kInterleaved) {
                        turn_interleaved(a, v0, p.rot, cs);
                        turn_interleaved(b, v1, p.rot, cs);
                    } else {
                        turn_half_odd(a, head[u], weight, tiny ? 0x1p100f : 1.0f, inv, p.offset, v0, p.rot, cs);
                        turn_half_odd(b, head[u], weight, tiny ? 0x1p100f : 1.0f, inv, p.offset, v1, p.rot, cs);
                    }
                    x[u][i][0] = pack8(a);
                    x[u][i][1] = pack8(b);
                }
                auto store = [&](uint16_t* to) {
                    *reinterpret_cast<uint4*>(to + 8 * v0) = x[u][i][0];
                    *reinterpret_cast<uint4*>(to + 8 * v1) = x[u][i][1];
                };
                if (h < p.q_heads) {
                    store(p.Q_out + (token * p.q_heads + h) * HD);
                } else if (turned) {
                    const int kh = h - p.q_heads;
                    if (p.K_out != nullptr) store(p.K_out + (token * p.nkv + kh) * HD);
                    if (p.K_cache != nullptr && slot >= 0)
                        store(p.K_cache + (slot * p.nkv + kh) * HD);
                } else if (slot >= 0) {
                    store(p.V_cache + (slot * p.nkv + h - p.q_heads - p.k_heads) * HD);
                }
            }
        }
    }
}

template <int HD, bool SMALL>
auto kernel_for(int mode) {
    return mode == kInterleaved ? norm_rope_kernel<HD, kInterleaved, SMALL>
           : mode == kHalf      ? norm_rope_kernel<HD, kHalf, SMALL>
                                : norm_rope_kernel<HD, kHalfOdd, SMALL>;
}

template <int HD>
hss_status launch(const NormParams& p, int64_t tokens, int mode, int num_sms, cudaStream_t stream) {
    using D = Deal<HD>;
    // A token is one CTA's, unless there are too few tokens to reach every SM: then its heads are
    // split over several, down to one item a thread.
    NormParams q = p;
    const int items = (p.q_heads + p.k_heads + p.v_heads) * D::kLanes;
    int64_t splits = (2 * num_sms + tokens - 1) / tokens;
    const int most = (items + kMostThreads - 1) / kMostThreads;
    splits = splits < most ? splits : most;
    q.split_items = static_cast<int>((items + splits - 1) / splits);
    q.split_items = (q.split_items + D::kLanes - 1) / D::kLanes * D::kLanes;  // whole heads
    const dim3 grid(static_cast<unsigned>(tokens),
                    static_cast<unsigned>((items + q.split_items - 1) / q.split_items));
    const int each = splits > 1 ? 1 : D::kBatch;
    int threads = ((q.split_items + each - 1) / each + 31) / 32 * 32;
    threads = threads < 64 ? 64 : (threads > kMostThreads ? kMostThreads : threads);
    // (in a kernel of its own: the check makes 8192 tokens of 64 + 8 heads 63.5 us, not 62.3)
    const auto kern = q.eps < kSmallest ? kernel_for<HD, true>(mode) : kernel_for<HD, false>(mode);
    return launch_pdl(kern, grid, dim3(threads), 0, stream, q) == cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

}  // namespace

hss_status launch_norm_rope(const NormRopeArgs& r, cudaStream_t stream) {
    const hss_rope_args& a = r.a->rope;
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    NormParams p;
    p.Q = r.Q;
    p.K = r.K;
    p.V = r.V;
    p.q_weight = r.q_weight;
    p.k_weight = r.k_weight;
    p.Q_out = r.Q_out;
    p.K_out = r.K_out;
    p.K_cache = r.K_cache;
    p.V_cache = r.V_cache;
    p.turns = a.turns;
    p.positions = a.positions;
    p.slots = r.K_cache != nullptr || r.V_cache != nullptr ? a.slots : nullptr;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_weight_stride = r.a->q_weight_stride;
    p.k_weight_stride = r.a->k_weight_stride;
    p.cache_tokens = a.dims.max_blocks * a.dims.block_size;
    p.magnitude = a.magnitude;
    p.eps = r.a->eps;
    p.offset = r.a->weight_offset;
    p.rot = a.rot_dim;
    p.q_heads = r.Q_out != nullptr ? a.dims.num_q_heads : 0;
    p.k_heads = r.K_out != nullptr || r.K_cache != nullptr ? a.dims.num_kv_heads : 0;
    p.v_heads = r.V_cache != nullptr ? a.dims.num_kv_heads : 0;
    p.nkv = a.dims.num_kv_heads;
    p.split_items = 0;
    p.dev_status = a.dev_status;
    p.lib_error = dev->error_word;
    const int mode = a.layout == HSS_ROPE_INTERLEAVED ? kInterleaved
                     : a.rot_dim % 16 == 0            ? kHalf
                                                      : kHalfOdd;
    switch (a.dims.head_dim) {
        case 64: return launch<64>(p, a.num_tokens, mode, dev->num_sms, stream);
        case 128: return launch<128>(p, a.num_tokens, mode, dev->num_sms, stream);
        case 192: return launch<192>(p, a.num_tokens, mode, dev->num_sms, stream);
        default: return launch<256>(p, a.num_tokens, mode, dev->num_sms, stream);
    }
}

}  // namespace hss
