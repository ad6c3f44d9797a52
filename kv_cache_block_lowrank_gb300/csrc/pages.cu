// pages.cu -- pages shared by sequences: fork, cut back, grow, drop, move to the front, copy.
//
// The plans (whose page goes where) are integer work over tables, sequences and page counts, with a
// few steps that each need all of the one before: counting down what is given up, counting up what
// is kept, settling who keeps a shared page, ranking the free pages.  One cluster of up to eight
// CTAs takes a whole plan, a cluster barrier between the steps, so that one launch does it; ranks
// are ballots within a warp and sums over warps and CTAs (distributed shared memory).  Counts are
// added with integer atomics, whose order does not matter, so the result is the same every time.
// What bounds a plan is latency: six barriers and as many trips to L2, and in a fork each entry's
// search for its sequence, whose numbers are then worked out anew from the inputs (256 sequences with
// 18,000 table entries over 23,000 pages forked 34 us, 8000 entries over 17,000 pages compacted 13).
// In eager calls the caller's host work with its copies is longer (51 us with the allocations, from
// Python).
//
// The copies are a kernel of their own, at the rate of HBM: 4.3 GB of pages compacted, 2.1 GB moved,
// 329 us, 6.5 TB/s.
#include <cooperative_groups.h>

#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace hss {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCtas = 8;
constexpr int kSums = 3;
constexpr int kHeldOffsets = 2048;  // of the new tables, kept in shared memory if they fit

// (a 64-bit division is some hundred instructions, one after another)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

struct PlanShared {
    int64_t warp[kSums][kWarps];
    int64_t cta[kSums];  // this CTA's totals, read by the others
    int32_t offsets[kHeldOffsets];
};

__device__ __forceinline__ int64_t warp_before(int64_t x, int64_t& all) {
    const int lane = threadIdx.x & 31;
    int64_t s = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, s, m);
        if (lane >= m) s += o;
    }
    all = __shfl_sync(0xffffffffu, s, 31);
    return s - x;
}

// Puts the CTA's sum of every thread's x[k] where the other CTAs find it after the next cluster
// barrier, and turns x[k] into what the threads before this one (of the CTA) have.
template <int N>
__device__ __forceinline__ void cta_before(PlanShared& sh, int64_t (&x)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t all;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        x[k] = warp_before(x[k], all);
        if (lane == 0) sh.warp[k][warp] = all;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int64_t mine = lane < kWarps ? sh.warp[k][lane] : 0;
        const int64_t before = warp_before(mine, all);
        x[k] += __shfl_sync(0xffffffffu, before, warp);
        if (threadIdx.x == 0) sh.cta[k] = all;
    }
}

// After the cluster barrier: what the CTAs before this one have, and all of them.
__device__ __forceinline__ void cluster_totals(cg::cluster_group& cluster, PlanShared& sh, int k,
                                               int64_t& before, int64_t& all) {
    before = all = 0;
    const int rank = static_cast<int>(cluster.block_rank());
    for (int r = 0; r < static_cast<int>(cluster.num_blocks()); ++r) {
        const int64_t v = cluster.map_shared_rank(sh.cta, r)[k];
        if (r < rank) before += v;
        all += v;
    }
}

// Pages are ranked warp by warp: a warp's are consecutive, 32 at a time.
struct PageRange {
    int64_t first, last;
    __device__ __forceinline__ PageRange(int64_t pages, int rank, int ctas) {
        const int64_t warps = static_cast<int64_t>(ctas) * kWarps;
        const int64_t each = ((pages + warps - 1) / warps + 31) / 32 * 32;
        first = min(pages, (static_cast<int64_t>(rank) * kWarps + (threadIdx.x >> 5)) * each);
        last = min(pages, first + each);
    }
};

__device__ __forceinline__ int32_t clip(int64_t x) {
    return static_cast<int32_t>(min(x, static_cast<int64_t>(0x7FFFFFFF)));
}

// ------------------------------------------------------------------------------------ fork

struct Heir {
    int64_t from;    // first table entry of the parent
    int64_t length;  // tokens kept
    int64_t kept;    // entries kept
    int64_t n;       // entries in all
    bool writes;     // into its last kept entry, if that is a page
};

__device__ __forceinline__ Heir heir_of(const ForkArgs& f, int i) {
    Heir x;
    const int p = __ldg(f.parents + i);
    int64_t has = 0;
    x.from = 0;
    if (p >= 0 && p < f.num_seqs) {
        x.from = min(max(static_cast<int64_t>(__ldg(f.seq_offsets + p)), int64_t{0}), f.total);
        const int64_t end = min(static_cast<int64_t>(__ldg(f.seq_offsets + p + 1)), f.total);
        has = max(end - x.from, int64_t{0});
    }
    const int64_t room = max(__ldg(f.room + i), 0);
    x.length = min(static_cast<int64_t>(max(__ldg(f.lengths + i), 0)), has * f.block_size);
    x.kept = divide(x.length + f.block_size - 1, f.block_size);
    x.n = divide(x.length + room + f.block_size - 1, f.block_size);
    x.writes = room > 0 && x.length != x.kept * f.block_size;
    return x;
}

// The last sequence whose entries begin at or before e, and where they begin.
__device__ __forceinline__ int owner_of(const ForkArgs& f, const PlanShared& sh, int64_t e,
                                        int64_t& begin) {
    const bool held = f.num_new <= kHeldOffsets;
    int lo = 0, hi = f.num_new - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((held ? sh.offsets[mid] : __ldcg(f.new_offsets + mid)) <= e)
            lo = mid;
        else
            hi = mid - 1;
    }
    begin = held ? sh.offsets[lo] : __ldcg(f.new_offsets + lo);
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const ForkArgs f, int32_t* lib_error) {
    __shared__ PlanShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(ctas) * kThreads;
    const int64_t at = static_cast<int64_t>(rank) * kThreads + threadIdx.x;
    const int64_t pages = f.max_blocks;
    int32_t* free_list = f.workspace;         // [pages]
    int32_t* writers = free_list + pages;     // [pages], of pages that somebody writes into
    int32_t* first_writer = writers + pages;  // [pages]
    int32_t* fresh_before = first_writer + pages;   // [num_new]
    int32_t* copy_before = fresh_before + f.num_new;  // [num_new], -1 - it where a copy is made
    grid_dependency_wait();
    grid_launch_dependents();
    auto raise = [&](int32_t code) { raise_error(f.dev_status, lib_error, code); };
    auto page_ok = [&](int32_t id) { return id >= 0 && id < pages; };
    // A thread's sequences are consecutive, so that sums over threads are offsets.
    const int64_t each = (f.num_new + stride - 1) / stride;
    const int i0 = static_cast<int>(min(at * each, static_cast<int64_t>(f.num_new)));
    const int i1 = static_cast<int>(min(at * each + each, static_cast<int64_t>(f.num_new)));
    // The page that sequence i writes into from its middle on, or -1.
    auto written_page = [&](const Heir& x) -> int32_t {
        if (!x.writes) return -1;
        const int32_t id = __ldg(f.table + x.from + x.kept - 1);
        return page_ok(id) ? id : -1;
    };

    // (nothing is counted up before all is counted down, so a count of 0 here is one too small)
    auto give_up = [&](int32_t id) {
        if (atomicSub(f.new_refs + id, 1) <= 0) raise(HSS_ERR_INVALID_ARGUMENT);
    };

    // Counts as they are; how many entries each sequence gets.
    for (int64_t p = at; p < pages; p += stride) f.new_refs[p] = __ldg(f.refs + p);
    int64_t entries[1] = {0};
    for (int i = i0; i < i1; ++i) {
        const Heir x = heir_of(f, i);
        entries[0] += x.n;
        const int p = __ldg(f.parents + i);
        if (p < -1 || p >= f.num_seqs) raise(HSS_ERR_OUT_OF_RANGE);
        const int32_t page = written_page(x);
        if (page >= 0) {
            writers[page] = 0;
            first_writer[page] = 0x7FFFFFFF;
        }
    }
    cta_before(sh, entries);
    cluster.sync();

    // What is given up; where the new tables begin; who writes into which page.
    int64_t before, new_total;
    cluster_totals(cluster, sh, 0, before, new_total);
    before += entries[0];
    for (int i = i0; i < i1; ++i) {
        f.new_offsets[i] = clip(before);
        const Heir x = heir_of(f, i);
        before += x.n;
        const int32_t page = written_page(x);
        if (page >= 0) {
            atomicAdd(writers + page, 1);
            atomicMin(first_writer + page, i);
        }
    }
    if (at == 0) f.new_offsets[f.num_new] = clip(new_total);
    if (at == 0 && new_total > f.table_room) raise(HSS_ERR_INVALID_ARGUMENT);
    for (int64_t e = at; e < f.total; e += stride) {
        const int32_t id = __ldg(f.table + e);
        if (page_ok(id))
            give_up(id);
        else
            raise(HSS_ERR_OUT_OF_RANGE);
    }
    for (int64_t e = at; e < f.num_released; e += stride) {
        const int32_t id = __ldg(f.released + e);
        if (page_ok(id))
            give_up(id);
        else if (id != -1)
            raise(HSS_ERR_OUT_OF_RANGE);
    }
    cluster.sync();

    // What is kept.
    if (f.num_new <= kHeldOffsets) {
        for (int i = threadIdx.x; i < f.num_new; i += kThreads)
            sh.offsets[i] = __ldcg(f.new_offsets + i);
        __syncthreads();
    }
    const int64_t table_end = min(new_total, f.table_room);
    for (int64_t e = at; e < table_end; e += stride) {
        int64_t begin;
        const int i = owner_of(f, sh, e, begin);
        const Heir x = heir_of(f, i);
        const int64_t j = e - begin;
        if (j < x.kept) {
            const int32_t id = __ldg(f.table + x.from + j);
            if (page_ok(id)) atomicAdd(f.new_refs + id, 1);
        }
    }
    cluster.sync();

    // Who gets a copy; how many fresh pages each needs; how many are free.
    int64_t sums[3] = {0, 0, 0};
    for (int i = i0; i < i1; ++i) {
        const Heir x = heir_of(f, i);
        const int32_t page = written_page(x);
        const bool keeps = page < 0 || (__ldcg(f.new_refs + page) == __ldcg(writers + page) &&
                                        __ldcg(first_writer + page) == i);
        sums[0] += x.n - x.kept + (keeps ? 0 : 1);
        sums[1] += keeps ? 0 : 1;
        copy_before[i] = keeps ? 0 : -1;
    }
    const PageRange range(pages, rank, ctas);
    int64_t free_here = 0;
    for (int64_t p = range.first + lane; p < range.last; p += 32) {
        free_here += __ldcg(f.new_refs + p) == 0;
    }
    sums[2] = free_here;
    cta_before(sh, sums);
    cluster.sync();

    // The free pages by rank; where each sequence's fresh pages and copy come in the lists.
    int64_t fresh, fresh_all, copies, copies_all, free, free_all;
    cluster_totals(cluster, sh, 0, fresh, fresh_all);
    cluster_totals(cluster, sh, 1, copies, copies_all);
    cluster_totals(cluster, sh, 2, free, free_all);
    fresh += sums[0];
    copies += sums[1];
    for (int i = i0; i < i1; ++i) {
        const Heir x = heir_of(f, i);
        const bool copy = copy_before[i] < 0;
        fresh_before[i] = clip(fresh);
        copy_before[i] = copy ? -1 - static_cast<int32_t>(copies) : 0;
        if (copy) {
            f.copy_src[copies] = written_page(x);
            f.copy_dst[copies] = -1;  // (what it stays if the tables do not fit)
        }
        fresh += x.n - x.kept + (copy ? 1 : 0);
        copies += copy ? 1 : 0;
    }
    // (the warp's first thread has what is before the warp)
    free = __shfl_sync(0xffffffffu, free + sums[2], 0);
    for (int64_t p0 = range.first; p0 < range.last; p0 += 32) {
        const bool is = p0 + lane < range.last && __ldcg(f.new_refs + p0 + lane) == 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, is);
        if (is) free_list[free + __popc(mask & ((1u << lane) - 1u))] =
            static_cast<int32_t>(p0 + lane);
        free += __popc(mask);
        if (free >= fresh_all) break;
    }
    cluster.sync();

    // The new tables; and the old pages of the copies lose a reference.  (Not while the free pages are
    // listed: given counts that are too small, a page that was counted as free could then be missing
    // from the list, and a word of it that nobody wrote would be taken for an id.)
    for (int i = i0; i < i1; ++i)
        if (copy_before[i] < 0) atomicSub(f.new_refs + written_page(heir_of(f, i)), 1);
    for (int64_t e = at; e < f.table_room; e += stride) {
        if (e >= table_end) {
            f.new_table[e] = -1;
            continue;
        }
        int64_t begin;
        const int i = owner_of(f, sh, e, begin);
        const Heir x = heir_of(f, i);
        const int64_t j = e - begin;
        const int32_t mark = __ldcg(copy_before + i);
        const int64_t first_fresh = x.kept - (mark < 0 ? 1 : 0);
        int32_t id;
        if (j < first_fresh) {
            id = __ldg(f.table + x.from + j);
        } else {
            const int64_t k = __ldcg(fresh_before + i) + (j - first_fresh);
            id = k < free_all ? __ldcg(free_list + k) : -1;
            if (id >= 0) f.new_refs[id] = 1;
            // (without room for all, pages that the missing entries hold are not known as held)
            if (mark < 0 && j == first_fresh && new_total <= f.table_room)
                f.copy_dst[-1 - mark] = id;
        }
        f.new_table[e] = id;
    }
    for (int64_t i = copies_all + at; i < f.num_new; i += stride) {
        f.copy_src[i] = -1;
        f.copy_dst[i] = -1;
    }
    if (at == 0) {
        const int64_t taken = min(fresh_all, free_all);
        f.counts[0] = clip(new_total);
        f.counts[1] = static_cast<int32_t>(copies_all);
        f.counts[2] = static_cast<int32_t>(pages - free_all + taken);
        f.counts[3] = clip(fresh_all - taken);
        if (fresh_all > free_all) raise(HSS_ERR_OUT_OF_RANGE);
    }
    cluster.sync();  // no CTA leaves while another may still read its sums
}

// ------------------------------------------------------------------------------------ compact

__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(const CompactArgs c, int32_t* lib_error) {
    __shared__ PlanShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(ctas) * kThreads;
    const int64_t at = static_cast<int64_t>(rank) * kThreads + threadIdx.x;
    const int64_t pages = c.max_blocks;
    int32_t* holes = c.workspace;     // [pages], ascending
    int32_t* tops = holes + pages;    // [pages], descending
    int32_t* goes = tops + pages;     // [pages], where a page from `used` on is afterwards
    grid_dependency_wait();
    grid_launch_dependents();

    const PageRange range(pages, rank, ctas);
    int64_t sums[1] = {0};
    for (int64_t p = range.first + lane; p < range.last; p += 32) {
        const int32_t r = __ldg(c.refs + p);
        c.new_refs[p] = r;
        sums[0] += r != 0;
        if (r < 0) raise_error(c.dev_status, lib_error, HSS_ERR_INVALID_ARGUMENT);
    }
    cta_before(sh, sums);
    cluster.sync();

    // Free pages below `used` by rank, used pages from there on by rank from the top.
    int64_t used_before, used;
    cluster_totals(cluster, sh, 0, used_before, used);
    used_before = __shfl_sync(0xffffffffu, used_before + sums[0], 0);
    int64_t holes_here[1] = {0};
    __syncthreads();
    cluster.sync();  // (the totals are about to be written again)
    for (int64_t p0 = range.first; p0 < range.last; p0 += 32) {
        const int64_t p = p0 + lane;
        const bool in = p < range.last;
        const bool is = in && __ldg(c.refs + p) != 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, is);
        const int64_t below = used_before + __popc(mask & ((1u << lane) - 1u));
        if (in && !is && p < used) {
            holes[p - below] = static_cast<int32_t>(p);
            ++holes_here[0];
        }
        if (is && p >= used) {
            tops[used - 1 - below] = static_cast<int32_t>(p);
            goes[p] = static_cast<int32_t>(p);
        }
        used_before += __popc(mask);
    }
    cta_before(sh, holes_here);
    cluster.sync();

    int64_t unused, found;
    cluster_totals(cluster, sh, 0, unused, found);
    const int64_t moves = min(found, c.move_room);
    for (int64_t k = at; k < c.move_room; k += stride) {
        int32_t src = -1, dst = -1;
        if (k < moves) {
            src = __ldcg(tops + k);
            dst = __ldcg(holes + k);
            c.new_refs[dst] = __ldg(c.refs + src);
            c.new_refs[src] = 0;
            goes[src] = dst;
        }
        c.copy_src[k] = src;
        c.copy_dst[k] = dst;
    }
    cluster.sync();

    for (int64_t e = at; e < c.total; e += stride) {
        int32_t id = __ldg(c.table + e);
        if (id >= 0 && id < pages) {
            // (a free page's id, which no table should hold, stays)
            if (id >= used && __ldg(c.refs + id) != 0) id = __ldcg(goes + id);
        } else if (id != -1) {
            raise_error(c.dev_status, lib_error, HSS_ERR_OUT_OF_RANGE);
        }
        c.new_table[e] = id;
    }
    if (at == 0) {
        c.counts[0] = static_cast<int32_t>(moves);
        c.counts[1] = static_cast<int32_t>(used);
        c.counts[2] = moves < found ? __ldcg(tops + moves) + 1 : static_cast<int32_t>(used);
        c.counts[3] = static_cast<int32_t>(found - moves);
    }
    cluster.sync();  // no CTA leaves while another may still read its sums
}

// Launches a plan on one cluster, of as many CTAs as its work gives something to do.
template <typename Args>
hss_status launch_plan(void (*kernel)(Args, int32_t*), const Args& args, int64_t work,
                       cudaStream_t stream) {
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    unsigned ctas = 1;
    while (ctas < kMostCtas && work > static_cast<int64_t>(ctas) * 4 * kThreads) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args, dev->error_word) == cudaSuccess ? HSS_OK
                                                                                  : HSS_ERR_CUDA;
}

// ------------------------------------------------------------------------------------ copies

constexpr int kCopyThreads = 256;
constexpr int kVectors = 4;  // 16-byte vectors in flight per thread
constexpr int64_t kPiece = kCopyThreads * kVectors * 16;  // bytes of a page that a CTA takes at once

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs c, int64_t pieces,
                                                            int32_t* lib_error) {
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t copies = c.max_copies;
    if (c.num_copies != nullptr)
        copies = min(max(static_cast<int64_t>(*c.num_copies), int64_t{0}), copies);
    const int pools = c.pool1 != nullptr ? 2 : 1;
    // A pair's pieces, pools and layers go to neighbouring CTAs.
    const int64_t per_pair = pieces * pools * c.num_layers;
    const int64_t total = copies * per_pair;
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int64_t pair = divide(w, per_pair), in = w - pair * per_pair;
        const int rest = static_cast<int>(divide(in, pieces));
        const int64_t piece = in - rest * pieces;
        const int32_t src = c.src[pair], dst = c.dst[pair];
        if (src < 0 || dst < 0) continue;
        if (src >= c.max_blocks || dst >= c.max_blocks) {
            if (in == 0 && threadIdx.x == 0)
                raise_error(c.dev_status, lib_error, HSS_ERR_OUT_OF_RANGE);
            continue;
        }
        uint8_t* pool = static_cast<uint8_t*>(rest % pools == 0 ? c.pool0 : c.pool1);
        const int64_t layer = static_cast<int64_t>(rest / pools) * c.max_blocks;
        const uint8_t* from = pool + (layer + src) * c.page_bytes;
        uint8_t* to = pool + (layer + dst) * c.page_bytes;
        const int64_t at = piece * kPiece + threadIdx.x * 16;
        uint4 v[kVectors];
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const int64_t o = at + k * (kCopyThreads * 16);
            if (o < c.page_bytes) v[k] = *reinterpret_cast<const uint4*>(from + o);
        }
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const int64_t o = at + k * (kCopyThreads * 16);
            if (o < c.page_bytes) *reinterpret_cast<uint4*>(to + o) = v[k];
        }
    }
}

}  // namespace

size_t fork_workspace_bytes(int32_t num_new, int64_t max_blocks) {
    return (3 * static_cast<size_t>(max_blocks) + 2 * static_cast<size_t>(num_new)) *
           sizeof(int32_t);
}

size_t compact_workspace_bytes(int64_t max_blocks) {
    return 3 * static_cast<size_t>(max_blocks) * sizeof(int32_t);
}

hss_status launch_fork(const ForkArgs& f, cudaStream_t stream) {
    return launch_plan(fork_kernel, f, f.max_blocks + f.total + f.table_room + f.num_released,
                       stream);
}

hss_status launch_compact(const CompactArgs& c, cudaStream_t stream) {
    return launch_plan(compact_kernel, c, c.max_blocks + c.total, stream);
}

hss_status launch_copy_pages(const CopyArgs& c, cudaStream_t stream) {
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    const int64_t pieces = (c.page_bytes + kPiece - 1) / kPiece;
    const int64_t most = c.max_copies * c.num_layers * (c.pool1 != nullptr ? 2 : 1);
    const int64_t resident = 8 * static_cast<int64_t>(dev->num_sms);
    const int64_t grid = most >= resident ? resident : (most * pieces < resident ? most * pieces
                                                                                : resident);
    return launch_pdl(copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0,
                      stream, c, pieces, dev->error_word) == cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

}  // namespace hss
