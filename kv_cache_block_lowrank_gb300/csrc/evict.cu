// evict.cu -- cut every sequence's block table to its budget by accumulated attention weight.
//
// Per sequence: the key of the last entry to go is found by radix select over order-preserving
// 32-bit keys (11 bits a pass, from the top; a pass that leaves exactly the entries still needed
// ends it), ties going in index order; then one stable pass packs what stays and what goes.
// Integer throughout, so the result is exact.
//
// What bounds it is latency: a sequence's entries are 8 bytes each (2048 blocks: 16 KB).  A
// cluster of 1 to 8 CTAs takes one sequence, its keys in registers (16 a thread, 8192 a CTA;
// longer slices are read again from L2), the passes' histograms summed through distributed
// shared memory, one cluster barrier a pass.  A warp owns 512 consecutive entries and ranks them
// by ballots, so that packing needs one scan over warp totals only.  Every CTA reads all
// sequences' lengths and budgets itself to know where its outputs go: what a sequence loses
// follows from its counts alone.
#include "rank_device.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace hss {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 16;                       // keys per thread and round
constexpr int kRound = kThreads * kKeys;        // entries per CTA and round
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;

struct EvictShared {
    uint32_t hist[2][kBins];
    uint32_t lt_eq[2];  // this CTA's entries below and at the threshold
    uint32_t warp_a[kWarps];
    uint32_t warp_b[kWarps];
    int64_t sums[4][kWarps];
    int64_t pre[4];  // entries kept and lost before this sequence, and in all
    uint32_t digit, below, in_bin;
};

struct Cut {
    int32_t n, lo, hi, lost;
};

__device__ __forceinline__ Cut cut_of(const EvictArgs& e, int s) {
    Cut c;
    c.n = e.seq_offsets[s + 1] - e.seq_offsets[s];
    if (c.n < 0) c.n = 0;
    int64_t hi = static_cast<int64_t>(c.n) - e.keep_last;
    if (e.ctx_len != nullptr) {
        const int32_t whole = max(e.ctx_len[s], 0) / e.block_size;
        hi = min(hi, static_cast<int64_t>(whole));
    }
    c.lo = min(e.keep_first, c.n);
    c.hi = static_cast<int32_t>(max(hi, static_cast<int64_t>(c.lo)));
    const int32_t over = c.n - max(e.budgets[s], 0);
    c.lost = min(max(over, 0), c.hi - c.lo);
    return c;
}

__global__ void __launch_bounds__(kThreads, 1) evict_kernel(const EvictArgs e) {
    __shared__ EvictShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int s = blockIdx.x / cs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();

    // Where this sequence's outputs go, and how much all of them fill.
    int64_t sum[4] = {0, 0, 0, 0};
    for (int i = tid; i < e.num_seqs; i += kThreads) {
        const Cut c = cut_of(e, i);
        if (i < s) {
            sum[0] += c.n - c.lost;
            sum[1] += c.lost;
        }
        sum[2] += c.n - c.lost;
        sum[3] += c.lost;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], m);
        if (lane == 0) sh.sums[k][warp] = sum[k];
    }
    const Cut c = cut_of(e, s);
    const int64_t first = e.seq_offsets[s];
    __syncthreads();
    if (tid < 4) {
        int64_t t = 0;
        for (int w = 0; w < kWarps; ++w) t += sh.sums[tid][w];
        sh.pre[tid] = t;
    }
    __syncthreads();
    const int64_t kept_before = sh.pre[0], lost_before = sh.pre[1];

    // This CTA's slice of the sequence: whole rounds of kRound entries, round q's warp w owning
    // entries (q * kWarps + w) * 512 + 32 j + lane.
    const int rounds = (c.n + kRound * cs - 1) / (kRound * cs);
    const int per_warp = (c.n + kWarps * cs - 1) / (kWarps * cs);  // short slices: fewer a warp
    const int step = rounds > 1 ? 32 * kKeys : (per_warp + 31) / 32 * 32;
    const int slice = rounds * kWarps * step;
    const int slice0 = rank * slice;
    const float* w_in = e.weights + first;
    const int32_t* table = e.table + first;
    uint32_t key[kKeys];
    // (entries that may not go get the largest key and are never counted)
    auto load = [&](int q) {
        const int base = slice0 + (q * kWarps + warp) * step + lane;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            const int i = base + 32 * j;
            const bool in = 32 * j < step && i >= c.lo && i < c.hi;
            key[j] = in ? rankdev::score_key(__ldg(w_in + i)) : 0xFFFFFFFFu;
        }
    };
    // What is packed, all of a round on its way together and ahead of the ranks (one entry after
    // another, each of a thread's 16 waited for its own loads: 8 sequences of 65536 entries 27 us,
    // so 22).
    int32_t id[kKeys];
    float weight[kKeys];
    auto fetch = [&](int q) {
        const int base = slice0 + (q * kWarps + warp) * step + lane;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            const int i = base + 32 * j;
            const bool there = 32 * j < step && i < c.n;
            id[j] = there ? __ldg(table + i) : 0;
            weight[j] = there ? __ldg(w_in + i) : 0.0f;
        }
    };
    auto inside = [&](int q, int j, int& i) {
        i = slice0 + (q * kWarps + warp) * step + 32 * j + lane;
        return 32 * j < step && i >= c.lo && i < c.hi;
    };
    if (c.lost > 0) load(0);
    fetch(0);

    // Radix select of the c.lost-th smallest key.
    uint32_t prefix = 0, need = static_cast<uint32_t>(c.lost);
    int shift = 32;
    if (c.lost > 0 && c.lost < c.hi - c.lo) {
        for (int pass = 0; shift > 0; ++pass) {
            const int bits = min(kDigitBits, shift);
            const int next = shift - bits;
            uint32_t* hist = sh.hist[pass & 1];
            for (int q = 0; q < rounds; ++q) {
                if (rounds > 1) load(q);
#pragma unroll
                for (int j = 0; j < kKeys; ++j) {
                    int i;
                    if (inside(q, j, i) && (shift == 32 || (key[j] >> shift) == prefix))
                        atomicAdd(&hist[(key[j] >> next) & ((1u << bits) - 1)], 1u);
                }
            }
            cluster.sync();
            // Every CTA sums the cluster's histograms: four bins a thread, then a scan.
            uint32_t bin[4] = {0, 0, 0, 0};
            for (int r = 0; r < cs; ++r) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    cluster.map_shared_rank(hist, (rank + r) % cs) + 4 * tid);
                bin[0] += v.x;
                bin[1] += v.y;
                bin[2] += v.z;
                bin[3] += v.w;
            }
            // The other buffer was last read before this barrier: clear it for the next pass.
            for (int i = tid; i < kBins; i += kThreads) sh.hist[(pass & 1) ^ 1][i] = 0;
            const uint32_t mine = bin[0] + bin[1] + bin[2] + bin[3];
            uint32_t scan = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, scan, m);
                if (lane >= m) scan += o;
            }
            if (lane == 31) sh.warp_a[warp] = scan;
            __syncthreads();
            uint32_t before = scan - mine;
            for (int w = 0; w < warp; ++w) before += sh.warp_a[w];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (before < need && need <= before + bin[b]) {
                    sh.digit = 4 * tid + b;
                    sh.below = before;
                    sh.in_bin = bin[b];
                }
                before += bin[b];
            }
            __syncthreads();
            prefix = (shift == 32 ? 0u : prefix << bits) | sh.digit;
            need -= sh.below;
            shift = next;
            const bool done = sh.in_bin == need;
            __syncthreads();
            if (done) break;
        }
    } else if (c.lost > 0) {
        shift = 0;  // every candidate goes
        prefix = 0xFFFFFFFFu;
        need = 0xFFFFFFFFu;
    }

    // Entries of this CTA below the threshold prefix and at it, and of the CTAs before it.
    uint32_t lt = 0, eq = 0;
    if (c.lost > 0) {
        for (int q = 0; q < rounds; ++q) {
            if (rounds > 1) load(q);
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                int i;
                const bool in = inside(q, j, i);
                const uint32_t k = shift == 32 ? 0u : key[j] >> shift;
                lt += in && k < prefix;
                eq += in && k == prefix;
            }
        }
    }
    if (tid == 0) sh.lt_eq[0] = sh.lt_eq[1] = 0;
    __syncthreads();
    lt = __reduce_add_sync(0xffffffffu, lt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0 && (lt | eq)) {
        atomicAdd(&sh.lt_eq[0], lt);
        atomicAdd(&sh.lt_eq[1], eq);
    }
    cluster.sync();
    uint32_t lt_run = 0, eq_run = 0;
    for (int r = 0; r < rank; ++r) {
        const uint32_t* o = cluster.map_shared_rank(sh.lt_eq, r);
        lt_run += o[0];
        eq_run += o[1];
    }

    // Pack, round by round in index order.
    for (int q = 0; q < rounds; ++q) {
        if (rounds > 1 && c.lost > 0) load(q);
        if (q > 0) fetch(q);
        uint32_t wl = 0, we = 0;
        if (c.lost > 0) {
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                int i;
                const bool in = inside(q, j, i);
                const uint32_t k = shift == 32 ? 0u : key[j] >> shift;
                wl += in && k < prefix;
                we += in && k == prefix;
            }
        }
        wl = __reduce_add_sync(0xffffffffu, wl);
        we = __reduce_add_sync(0xffffffffu, we);
        if (lane == 0) {
            sh.warp_a[warp] = wl;
            sh.warp_b[warp] = we;
        }
        __syncthreads();
        uint32_t l = lt_run, t = eq_run;
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t a = sh.warp_a[w], b = sh.warp_b[w];
            if (w < warp) {
                l += a;
                t += b;
            }
            lt_run += a;
            eq_run += b;
        }
        __syncthreads();
        uint32_t lost = l + min(t, need);  // lost before this warp's first entry
        if (c.lost == 0) lost = 0;
        const int base = slice0 + (q * kWarps + warp) * step + lane;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            if (32 * j >= step) break;
            const int i = base + 32 * j;
            const bool in = c.lost > 0 && i >= c.lo && i < c.hi;
            const uint32_t k = shift == 32 ? 0u : key[j] >> shift;
            const uint32_t lanes_before = (1u << lane) - 1u;
            const uint32_t tie = __ballot_sync(0xffffffffu, in && k == prefix);
            const bool goes = in && (k < prefix || (k == prefix &&
                                                    t + __popc(tie & lanes_before) < need));
            const uint32_t going = __ballot_sync(0xffffffffu, goes);
            const uint32_t gone = lost + __popc(going & lanes_before);
            if (i < c.n) {
                if (goes) {
                    e.freed[lost_before + gone] = id[j];
                } else {
                    const int64_t to = kept_before + i - gone;
                    e.new_table[to] = id[j];
                    e.new_weights[to] = weight[j];
                }
            }
            t += __popc(tie);
            lost += __popc(going);
        }
    }

    if (rank == 0 && tid == 0) {
        e.new_offsets[s] = static_cast<int32_t>(kept_before);
        e.freed_offsets[s] = static_cast<int32_t>(lost_before);
        if (e.new_ctx_len != nullptr) e.new_ctx_len[s] = e.ctx_len[s] - c.lost * e.block_size;
        if (s == e.num_seqs - 1) {
            e.new_offsets[s + 1] = static_cast<int32_t>(sh.pre[2]);
            e.freed_offsets[s + 1] = static_cast<int32_t>(sh.pre[3]);
        }
    }
    // The unused ends of the packed arrays, shared out over the grid.
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
    for (int64_t i = sh.pre[2] + at; i < e.total; i += stride) {
        e.new_table[i] = -1;
        e.new_weights[i] = 0.0f;
    }
    for (int64_t i = sh.pre[3] + at; i < e.total; i += stride) e.freed[i] = -1;
    cluster.sync();  // no CTA leaves while another may still read its counts
}

}  // namespace

hss_status launch_evict(const EvictArgs& e, cudaStream_t stream) {
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    // CTAs per sequence: so that an average sequence's keys stay in registers, eight at most.
    const int64_t mean = e.total / e.num_seqs;
    unsigned cs = 1;
    while (cs < 8 && mean > static_cast<int64_t>(cs) * kRound) cs *= 2;
    if (e.num_seqs > 0x7FFFFFFF / static_cast<int>(cs)) return HSS_ERR_INVALID_ARGUMENT;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(e.num_seqs) * cs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, evict_kernel, e) != cudaSuccess) return HSS_ERR_CUDA;
    return HSS_OK;
}

}  // namespace hss
