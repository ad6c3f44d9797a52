// attend_packed.cu -- hss_attend_packed on the host: the workspace and the choice of the kernel.
#include <algorithm>

#include "attend_packed.cuh"

namespace hss {
namespace {

using packed::kSms;

// Ranges of the list of the kernel for few rows, and their rows, that the workspace has room for;
// the kernel for many has a range an SM, of one or two row tiles of 128.
constexpr int kRanges = 2 * kSms;
constexpr int kRangeRows = 16 * kRanges;

// Rows of one sequence and kv head from which on the tensor cores' rows are filled well enough.  (Heads
// of 128, by the kernel for few rows, 16 at a time, and the other.  64 sequences of 2048 tokens and 8 kv
// heads: 24 rows 135 and 162 us, 32 137 and 164, 40 190 and 166, 64 249 and 171; 16 of 4096: 32 76 and
// 88, 40 101 and 91; one of 32768: 32 41 and 51, 40 53 and 51, 64 66 and 53.  With 2 kv heads less is
// there to fill: 16 of 4096 tokens 32 31 and 41, 48 38 and 43, 64 45 and 44; one of 32768 64 30 and 39, 96
// 36 and 41.  16 of 4096, 8 kv heads of 64: 32 57 and 75, 64 94 and 77; of 192: 32 94 and 118, 64 160
// and 129; of 256: 32 162 and 166, 40 221 and 169.)
constexpr int64_t kManyRows = 33;

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

int64_t rows_of(const hss_dims& d, int64_t max_q) {
    return max_q * (d.num_q_heads / d.num_kv_heads);
}
int64_t many_rows(const hss_dims& d) { return d.head_dim <= 128 ? 256 : 128; }

struct Layout {
    size_t starts, ml, o, flags, many_starts, many_ml, many_o, end;
    Layout(const hss_dims& d, bool many) {
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t was = at;
            at += round_up(bytes);
            return was;
        };
        starts = take(kRanges * sizeof(packed::Start));
        ml = take(2 * kRangeRows * sizeof(float2));
        o = take(static_cast<size_t>(2 * kRangeRows) * d.head_dim * sizeof(float));
        flags = take(packed::kMostGuards * sizeof(int32_t));
        const size_t rows = many ? 2 * kSms * many_rows(d) : 0;
        many_starts = take(kSms * sizeof(packed::Start));
        many_ml = take(rows * sizeof(float2));
        many_o = take(rows * d.head_dim * sizeof(float));
        end = at;
    }
};

}  // namespace

size_t attend_packed_workspace_bytes(const hss_dims& d, int32_t, int32_t max_q, int64_t, int32_t,
                                     int32_t) {
    return Layout(d, rows_of(d, max_q) >= kManyRows).end;
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
    p.window = x.window > 0 ? std::min(x.window, packed::kNoWindow) : packed::kNoWindow;
    p.sinks = x.window > 0 ? x.sinks : 0;
    p.c = x.scale * 1.44269504088896341f;
    p.row_tiles = 0;
    p.guard = nullptr;
    p.guards = 0;
    p.dev_status = x.dev_status;
    p.lib_error = dev->error_word;
    const int64_t rows = rows_of(x.dims, p.max_q);
    const bool with_many = rows >= kManyRows;
    const Layout at(x.dims, with_many);
    uint8_t* w = static_cast<uint8_t*>(x.workspace);
    p.starts = reinterpret_cast<packed::Start*>(w + at.starts);
    p.part_ml = reinterpret_cast<float2*>(w + at.ml);
    p.part_o = reinterpret_cast<float*>(w + at.o);
    int32_t* flags = reinterpret_cast<int32_t*>(w + at.flags);
    packed::Params many = p;
    many.starts = reinterpret_cast<packed::Start*>(w + at.many_starts);
    many.part_ml = reinterpret_cast<float2*>(w + at.many_ml);
    many.part_o = reinterpret_cast<float*>(w + at.many_o);
    if (with_many) p.guard = flags;
    const packed::Params* m = with_many ? &many : nullptr;
    const int n = rows <= 8 ? 1 : 2;  // n-tiles of 8 rows that a tile of the cache is decoded for
    switch (x.dims.head_dim) {
        case 64: return packed::launch_head_dim<64>(p, m, n, flags, stream);
        case 128: return packed::launch_head_dim<128>(p, m, n, flags, stream);
        case 192: return packed::launch_head_dim<192>(p, m, n, flags, stream);
        default: return packed::launch_head_dim<256>(p, m, n, flags, stream);
    }
}

}  // namespace hss
