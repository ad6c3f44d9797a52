// rope.cu -- rotary positions for new queries and keys, and their paged cache write.
//
// Pair i of a head at position pos turns by a = 2 pi frac(pos * turns[i] / 2^64): the 64-bit
// product wraps, which is the reduction to one turn without rounding, and its upper 32 bits
// (as a signed number, a half-turn either way) go to sincospi.  The angle is the same for all
// heads of a token, so one CTA takes one token and computes its rot_dim / 2 sines and cosines
// once into shared memory.
//
// Each thread moves two 16-byte vectors of a head: in the half layout the two that hold the two
// ends of eight pairs, so that a rotated element is read once; in the interleaved layout both
// ends of a pair lie in one vector.  The loads are issued before the sines are there.
#include "ptx.cuh"

namespace hss {
namespace {

constexpr int kMostThreads = 256;
constexpr int kBatch = 4;  // items (two vectors each) in flight per thread

enum RopeMode { kInterleaved, kHalf, kHalfOdd };

struct RopeParams {
    const uint16_t* Q;
    const uint16_t* K;
    const uint16_t* V;
    uint16_t* Q_out;
    uint16_t* K_out;
    uint16_t* K_cache;
    uint16_t* V_cache;
    const uint64_t* turns;
    const int64_t* positions;
    const int64_t* slots;
    int64_t q_stride, k_stride, v_stride;
    int64_t cache_tokens;  // max_blocks * block_size
    float magnitude;
    int rot;
    int q_heads;  // query heads to rotate (0: none), then kv heads to rotate, then values to copy
    int k_heads;
    int v_heads;
    int nkv;
    int split_items;  // items of one CTA of a token
    int32_t* dev_status;
    int32_t* lib_error;
};

struct alignas(16) Vec8 {
    __nv_bfloat162 h[4];
};

// The vectors of a head that lane l (of head_dim / 16) takes.
template <int HD, int MODE>
__device__ __forceinline__ void lane_vectors(int l, int rot, int& v0, int& v1) {
    if constexpr (MODE == kHalf) {
        const int pairs = rot / 16;  // vector pairs (j, j + pairs) hold the two ends of 8 pairs
        if (l < pairs) {
            v0 = l;
            v1 = l + pairs;
        } else {
            v0 = 2 * l;  // past rot_dim: 2 pairs + 2 (l - pairs), and the one after it
            v1 = 2 * l + 1;
        }
    } else {
        v0 = l;
        v1 = l + HD / 16;
    }
}

__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
    Vec8 x;
    *reinterpret_cast<uint4*>(&x) = __ldg(reinterpret_cast<const uint4*>(p));
    return x;
}

// One vector of the interleaved layout: elements 8 v .. 8 v + 7 are pairs 4 v .. 4 v + 3.
__device__ __forceinline__ void turn_interleaved(Vec8& x, int v, int rot, const float2* cs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int pair = 4 * v + e;
        if (2 * pair < rot) {
            const float2 a = __bfloat1622float2(x.h[e]);
            const float2 c = cs[pair];
            x.h[e] = __floats2bfloat162_rn(a.x * c.x - a.y * c.y, a.y * c.x + a.x * c.y);
        }
    }
}

__device__ __forceinline__ void turn_half(Vec8& x, Vec8& y, int l, const float2* cs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = __bfloat1622float2(x.h[e]), b = __bfloat1622float2(y.h[e]);
        const float2 c0 = cs[8 * l + 2 * e], c1 = cs[8 * l + 2 * e + 1];
        x.h[e] = __floats2bfloat162_rn(a.x * c0.x - b.x * c0.y, a.y * c1.x - b.y * c1.y);
        y.h[e] = __floats2bfloat162_rn(b.x * c0.x + a.x * c0.y, b.y * c1.x + a.y * c1.y);
    }
}

// Half layout whose halves are not whole vectors: each element's partner is fetched by itself.
__device__ __forceinline__ void turn_half_odd(Vec8& x, const uint16_t* head, int v, int rot,
                                              const float2* cs) {
    const int half = rot / 2;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = 8 * v + e;
        const float own = __bfloat162float(e & 1 ? x.h[e / 2].y : x.h[e / 2].x);
        r[e] = own;
        if (i < rot) {
            const bool first = i < half;
            const int other = first ? i + half : i - half;
            const float o = __uint_as_float(static_cast<uint32_t>(__ldg(head + other)) << 16);
            const float2 c = cs[first ? i : other];
            r[e] = first ? own * c.x - o * c.y : own * c.x + o * c.y;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x.h[e] = __floats2bfloat162_rn(r[2 * e], r[2 * e + 1]);
}

template <int HD, int MODE>
__global__ void __launch_bounds__(kMostThreads) rope_kernel(const RopeParams p) {
    constexpr int kLanes = HD / 16;
    const int kThreads = static_cast<int>(blockDim.x);
    __shared__ float2 cs[128];
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
    for (int base = begin; base < end; base += kThreads * kBatch) {
        Vec8 x[kBatch], y[kBatch];
        const uint16_t* head[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int item = base + u * kThreads + static_cast<int>(threadIdx.x);
            const int h = item / kLanes, l = item % kLanes;
            if (item >= end) break;
            head[u] = h < p.q_heads               ? q + h * HD
                      : h < p.q_heads + p.k_heads ? k + (h - p.q_heads) * HD
                                                  : v + (h - p.q_heads - p.k_heads) * HD;
            int v0, v1;
            lane_vectors<HD, MODE>(l, p.rot, v0, v1);
            x[u] = load8(head[u] + 8 * v0);
            y[u] = load8(head[u] + 8 * v1);
        }
        if (!ready) {
            for (int i = threadIdx.x; turns && i < p.rot / 2; i += kThreads) {
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
            const int item = base + u * kThreads + static_cast<int>(threadIdx.x);
            const int h = item / kLanes, l = item % kLanes;
            if (item >= end) break;
            int v0, v1;
            lane_vectors<HD, MODE>(l, p.rot, v0, v1);
            if (h < p.q_heads + p.k_heads) {
                if constexpr (MODE == kHalf) {
                    if (l < p.rot / 16) turn_half(x[u], y[u], l, cs);
                } else if constexpr (MODE == kInterleaved) {
                    turn_interleaved(x[u], v0, p.rot, cs);
                    turn_interleaved(y[u], v1, p.rot, cs);
                } else {
                    turn_half_odd(x[u], head[u], v0, p.rot, cs);
                    turn_half_odd(y[u], head[u], v1, p.rot, cs);
                }
            }
            auto store = [&](uint16_t* to) {
                *reinterpret_cast<uint4*>(to + 8 * v0) = *reinterpret_cast<const uint4*>(&x[u]);
                *reinterpret_cast<uint4*>(to + 8 * v1) = *reinterpret_cast<const uint4*>(&y[u]);
            };
            if (h < p.q_heads) {
                store(p.Q_out + (token * p.q_heads + h) * HD);
            } else if (h < p.q_heads + p.k_heads) {
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

template <int HD>
auto kernel_for(int mode) {
    return mode == kInterleaved ? rope_kernel<HD, kInterleaved>
           : mode == kHalf      ? rope_kernel<HD, kHalf>
                                : rope_kernel<HD, kHalfOdd>;
}

}  // namespace

hss_status launch_rope(const RopeArgs& r, cudaStream_t stream) {
    const hss_rope_args& a = *r.a;
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    RopeParams p;
    p.Q = r.Q;
    p.K = r.K;
    p.V = r.V;
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
    p.cache_tokens = a.dims.max_blocks * a.dims.block_size;
    p.magnitude = a.magnitude;
    p.rot = a.rot_dim;
    p.q_heads = r.Q_out != nullptr ? a.dims.num_q_heads : 0;
    p.k_heads = r.K_out != nullptr || r.K_cache != nullptr ? a.dims.num_kv_heads : 0;
    p.v_heads = r.V_cache != nullptr ? a.dims.num_kv_heads : 0;
    p.nkv = a.dims.num_kv_heads;
    p.dev_status = a.dev_status;
    p.lib_error = dev->error_word;
    const int mode = a.layout == HSS_ROPE_INTERLEAVED ? kInterleaved
                     : a.rot_dim % 16 == 0            ? kHalf
                                                      : kHalfOdd;
    // A token is one CTA's, unless there are too few tokens to reach every SM: then its items
    // are split over several, down to one item a thread.
    const int items = (p.q_heads + p.k_heads + p.v_heads) * (a.dims.head_dim / 16);
    int64_t splits = (2 * dev->num_sms + a.num_tokens - 1) / a.num_tokens;
    const int most = (items + kMostThreads - 1) / kMostThreads;
    splits = splits < most ? splits : most;
    p.split_items = static_cast<int>((items + splits - 1) / splits);
    const dim3 grid(static_cast<unsigned>(a.num_tokens),
                    static_cast<unsigned>((items + p.split_items - 1) / p.split_items));
    // As many threads as leave each with kBatch items, all of whose loads are then in flight (80
    // heads of 128: 160 threads and four items each, 53 us for 8192 tokens, against 58 us with
    // 256 threads of two or three).  Few tokens are short of threads, not of bandwidth: one item.
    const int each = splits > 1 ? 1 : kBatch;
    int threads = ((p.split_items + each - 1) / each + 31) / 32 * 32;
    threads = threads < 64 ? 64 : (threads > kMostThreads ? kMostThreads : threads);
    auto kern = a.dims.head_dim == 64    ? kernel_for<64>(mode)
                : a.dims.head_dim == 128 ? kernel_for<128>(mode)
                : a.dims.head_dim == 192 ? kernel_for<192>(mode)
                                         : kernel_for<256>(mode);
    if (launch_pdl(kern, grid, dim3(threads), 0, stream, p) != cudaSuccess) return HSS_ERR_CUDA;
    return HSS_OK;
}

}  // namespace hss
