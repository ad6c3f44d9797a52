// attend_packed.cu -- hss_attend_packed on the host: the workspace and the choice of the kernel.
#include <algorithm>

#include "attend_packed.cuh"

namespace hss {
namespace {

// Ranges of the list, and their rows, that the workspace has room for.
constexpr int kRanges = 4 * packed::kSms;
constexpr int kRangeRows = 8 * kRanges;

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// n-tiles of 8 rows that a CTA takes at once: a tile of the cache is decoded once for all of them,
// and O takes head_dim / 4 of a thread's registers for each.
int n_tiles(const hss_dims& d, int64_t max_q) {
    return max_q * (d.num_q_heads / d.num_kv_heads) <= 8 ? 1 : 2;
}

}  // namespace

size_t attend_packed_workspace_bytes(const hss_dims& d, int32_t, int32_t, int64_t, int32_t,
                                     int32_t) {
    return round_up(kRanges * sizeof(packed::Start)) +
           round_up(2 * kRangeRows * sizeof(float2)) +
           static_cast<size_t>(2 * kRangeRows) * d.head_dim * sizeof(float);
}

hss_status launch_attend_packed(const PackedArgs& a, cudaStream_t stream) {
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    const hss_packed_args& x = *a.a;
    packed::Params p;
    p.Q = a.Q;
    p.cache = a.cache;
    p.out = a.out;
    p.lse = a.lse;
    p.q_offsets = x.q_offsets;
    p.table = x.block_table;
    p.seq_offsets = x.seq_offsets;
    p.ctx_len = x.ctx_len;
    p.max_blocks = x.dims.max_blocks;
    p.total_blocks = x.total_blocks;
    p.num_seqs = x.num_seqs;
    p.max_q = static_cast<int32_t>(std::min<int64_t>(x.max_q, x.total_q));
    p.nq = x.dims.num_q_heads;
    p.nkv = x.dims.num_kv_heads;
    p.g = p.nq / p.nkv;
    p.bs = x.dims.block_size;
    p.window = x.window > 0 ? x.window : 0x7FFFFFFF;
    p.sinks = x.window > 0 ? x.sinks : 0;
    p.c = x.scale * 1.44269504088896341f;
    p.dev_status = x.dev_status;
    p.lib_error = dev->error_word;
    uint8_t* w = static_cast<uint8_t*>(x.workspace);
    p.starts = reinterpret_cast<packed::Start*>(w);
    w += round_up(kRanges * sizeof(packed::Start));
    p.part_ml = reinterpret_cast<float2*>(w);
    w += round_up(2 * kRangeRows * sizeof(float2));
    p.part_o = reinterpret_cast<float*>(w);
    const int n = n_tiles(x.dims, p.max_q);
    switch (x.dims.head_dim) {
        case 64: return packed::launch_head_dim<64>(p, n, stream);
        case 128: return packed::launch_head_dim<128>(p, n, stream);
        case 192: return packed::launch_head_dim<192>(p, n, stream);
        default: return packed::launch_head_dim<256>(p, n, stream);
    }
}

}  // namespace hss
