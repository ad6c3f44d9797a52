// attend.cu -- attention of a tree of drafted tokens over the paged cache.
//
// One CTA takes 16 rows (node, query head of one kv head) of a sequence and walks the
// sequence's tokens in tiles of 32 through shared memory, one pass with the running maximum and
// sum of the softmax, everything in fp32.  The block weights come from a second kernel that
// forms the scores of an entry's tokens again and adds exp(s - lse).
#include "ptx.cuh"

namespace hss {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;
constexpr int kTokens = 32;

struct AttendParams {
    const uint16_t* Q;
    const uint16_t* K;
    const uint16_t* V;
    uint16_t* out;
    float* lse;
    const float* weights_in;
    float* weights_out;
    const int32_t* q_offsets;
    const uint64_t* mask;
    const int32_t* table;
    const int32_t* seq_offsets;
    const int32_t* ctx_len;
    int64_t max_blocks;
    int64_t total_blocks;
    int32_t mask_words, num_seqs, max_q, nq, nkv, g, bs;
    float scale, decay;
    int32_t* dev_status;
    int32_t* lib_error;
};

__device__ __forceinline__ float bf(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
}

struct Seq {
    int64_t q0, e0, tokens;
    int nodes, ctx;
};

__device__ __forceinline__ Seq seq_of(const AttendParams& p, int s) {
    Seq x;
    x.q0 = p.q_offsets[s];
    x.nodes = p.q_offsets[s + 1] - static_cast<int>(x.q0);
    if (x.nodes > p.max_q) {
        if (threadIdx.x == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_INVALID_ARGUMENT);
        x.nodes = p.max_q;
    }
    x.e0 = p.seq_offsets[s];
    const int64_t room = (p.seq_offsets[s + 1] - x.e0) * p.bs;
    x.ctx = max(p.ctx_len[s], 0);
    x.tokens = static_cast<int64_t>(x.ctx) + x.nodes;
    if (x.tokens > room) {
        if (threadIdx.x == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        x.tokens = room;
    }
    return x;
}

__device__ __forceinline__ bool sees(const AttendParams& p, const Seq& x, int node, int64_t pos) {
    if (pos >= x.tokens) return false;
    if (pos < x.ctx) return true;
    const int64_t j = pos - x.ctx;
    if (p.mask == nullptr) return j <= node;
    if (j >= 64 * static_cast<int64_t>(p.mask_words)) return false;
    return (p.mask[(x.q0 + node) * p.mask_words + (j >> 6)] >> (j & 63)) & 1;
}

template <int HD>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendParams p) {
    extern __shared__ float smem[];
    float* q = smem;                        // [kRows][HD]
    float* k = q + kRows * HD;              // [kTokens][HD + 1]
    float* v = k + kTokens * (HD + 1);      // [kTokens][HD]
    float* w = v + kTokens * HD;            // [kRows][kTokens]; -1: not seen
    int* good = reinterpret_cast<int*>(w + kRows * kTokens);
    grid_dependency_wait();
    grid_launch_dependents();
    const int tiles = (p.max_q * p.g + kRows - 1) / kRows;
    const int tile = blockIdx.x % tiles;
    const int h = blockIdx.x / tiles % p.nkv;
    const int s = blockIdx.x / tiles / p.nkv;
    const Seq x = seq_of(p, s);
    const int row0 = tile * kRows, rows = x.nodes * p.g;
    if (row0 >= rows) return;
    const int tid = threadIdx.x, r = tid / 8, c = tid % 8;
    const int row = row0 + r, node = row / p.g, head = h * p.g + row % p.g;
    for (int i = tid; i < kRows * HD; i += kThreads) {
        const int rr = row0 + i / HD;
        q[i] = rr < rows ? bf(p.Q[((x.q0 + rr / p.g) * p.nq + h * p.g + rr % p.g) * HD + i % HD])
                         : 0.0f;
    }
    float m = -INFINITY, l = 0.0f, acc[HD / 8];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) acc[i] = 0.0f;
    for (int64_t t0 = 0; t0 < x.tokens; t0 += kTokens) {
        __syncthreads();
        for (int i = tid; i < kTokens * HD; i += kThreads) {
            const int t = i / HD, d = i % HD;
            const int64_t pos = t0 + t;
            const int64_t id = pos < x.tokens ? p.table[x.e0 + pos / p.bs] : -1;
            const bool ok = id >= 0 && id < p.max_blocks;
            if (d == 0) {
                good[t] = ok;
                if (!ok && pos < x.tokens)
                    raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
            }
            const int64_t at = ((id * p.bs + pos % p.bs) * p.nkv + h) * HD + d;
            k[t * (HD + 1) + d] = ok ? bf(p.K[at]) : 0.0f;
            v[t * HD + d] = ok ? bf(p.V[at]) : 0.0f;
        }
        __syncthreads();
        float sc[kTokens / 8], top = m;
#pragma unroll
        for (int i = 0; i < kTokens / 8; ++i) {
            const int t = c + 8 * i;
            float a = 0.0f;
            for (int d = 0; d < HD; ++d) a += q[r * HD + d] * k[t * (HD + 1) + d];
            const bool see = row < rows && good[t] && sees(p, x, node, t0 + t);
            sc[i] = see ? a * p.scale : -INFINITY;
            w[r * kTokens + t] = see ? 0.0f : -1.0f;
            top = fmaxf(top, sc[i]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        const float shrink = expf(m - base);
        float add = 0.0f;
#pragma unroll
        for (int i = 0; i < kTokens / 8; ++i) {
            const int t = c + 8 * i;
            const float e = expf(sc[i] - base);
            if (w[r * kTokens + t] >= 0.0f) {
                w[r * kTokens + t] = e;
                add += e;
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
        l = l * shrink + add;
        m = top;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) acc[i] *= shrink;
        for (int t = 0; t < kTokens; ++t) {
            const float e = w[r * kTokens + t];
            if (e < 0.0f) continue;
#pragma unroll
            for (int i = 0; i < HD / 8; ++i) acc[i] += e * v[t * HD + c + 8 * i];
        }
    }
    if (row < rows) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* o = p.out + ((x.q0 + node) * p.nq + head) * HD;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
            const __nv_bfloat16 y = __float2bfloat16(acc[i] * inv);
            o[c + 8 * i] = __bfloat16_as_ushort(y);
        }
        if (c == 0) p.lse[(x.q0 + node) * p.nq + head] = l == 0.0f ? -INFINITY : m + logf(l);
    }
}

__global__ void __launch_bounds__(kThreads) weights_kernel(const AttendParams p, int hd) {
    __shared__ float part[kThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t e = blockIdx.x;
    int lo = 0, hi = p.num_seqs;  // last s with seq_offsets[s] <= e
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.seq_offsets[mid] <= e) lo = mid; else hi = mid;
    }
    const Seq x = seq_of(p, lo);
    const int64_t id = p.table[e], pos0 = (e - x.e0) * p.bs;
    float sum = 0.0f;
    if (id >= 0 && id < p.max_blocks) {
        const int all = x.nodes * p.nq * p.bs;
        for (int i = threadIdx.x; i < all; i += kThreads) {
            const int t = i % p.bs, hq = i / p.bs % p.nq, node = i / p.bs / p.nq;
            if (!sees(p, x, node, pos0 + t)) continue;
            const uint16_t* q = p.Q + ((x.q0 + node) * p.nq + hq) * hd;
            const uint16_t* k = p.K + ((id * p.bs + t) * p.nkv + hq / p.g) * hd;
            float a = 0.0f;
            for (int d = 0; d < hd; ++d) a += bf(q[d]) * bf(k[d]);
            sum += expf(a * p.scale - p.lse[(x.q0 + node) * p.nq + hq]);
        }
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 32; ++i) sum += part[i];
        const float old = p.weights_in != nullptr ? p.weights_in[e] * p.decay : 0.0f;
        p.weights_out[e] = old + sum;
    }
}

template <int HD>
cudaError_t launch(const AttendParams& p, unsigned grid, cudaStream_t stream) {
    const int smem = (kRows * HD + kTokens * (HD + 1) + kTokens * HD + kRows * kTokens + kTokens) * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        attend_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attend_kernel<HD>, dim3(grid), dim3(kThreads), smem, stream, p);
}

}  // namespace

size_t attend_workspace_bytes(const hss_dims& d, int32_t num_seqs, int32_t max_q,
                              int64_t total_blocks, bool with_weights) {
    (void)total_blocks;
    (void)with_weights;
    return (static_cast<size_t>(num_seqs) * max_q * d.num_q_heads * 4 + 255) / 256 * 256;
}

hss_status launch_attend(const AttendArgs& r, cudaStream_t stream) {
    const hss_attend_args& a = *r.a;
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    AttendParams p;
    p.Q = r.Q;
    p.K = r.K;
    p.V = r.V;
    p.out = r.out;
    p.lse = r.lse != nullptr ? r.lse : static_cast<float*>(a.workspace);
    p.weights_in = r.weights_in;
    p.weights_out = r.weights_out;
    p.q_offsets = a.q_offsets;
    p.mask = a.tree_mask;
    p.table = a.block_table;
    p.seq_offsets = a.seq_offsets;
    p.ctx_len = a.ctx_len;
    p.max_blocks = a.dims.max_blocks;
    p.total_blocks = a.total_blocks;
    p.mask_words = a.mask_words;
    p.num_seqs = a.num_seqs;
    p.max_q = a.max_q;
    p.nq = a.dims.num_q_heads;
    p.nkv = a.dims.num_kv_heads;
    p.g = p.nq / p.nkv;
    p.bs = a.dims.block_size;
    p.scale = a.scale;
    p.decay = a.decay;
    p.dev_status = a.dev_status;
    p.lib_error = dev->error_word;
    const int64_t tiles = (static_cast<int64_t>(a.max_q) * p.g + kRows - 1) / kRows;
    const int64_t grid = tiles * p.nkv * a.num_seqs;
    if (grid > 0x7FFFFFFF) return HSS_ERR_INVALID_ARGUMENT;
    if (a.total_q > 0) {
        const unsigned n = static_cast<unsigned>(grid);
        const cudaError_t e = a.dims.head_dim == 64    ? launch<64>(p, n, stream)
                              : a.dims.head_dim == 128 ? launch<128>(p, n, stream)
                              : a.dims.head_dim == 192 ? launch<192>(p, n, stream)
                                                       : launch<256>(p, n, stream);
        if (e != cudaSuccess) return HSS_ERR_CUDA;
    }
    if (r.weights_out != nullptr &&
        launch_pdl(weights_kernel, dim3(static_cast<unsigned>(a.total_blocks)), dim3(kThreads), 0,
                   stream, p, a.dims.head_dim) != cudaSuccess)
        return HSS_ERR_CUDA;
    return HSS_OK;
}

}  // namespace hss
