// packed_api.cu -- the C ABI of the packed cache and of shared pages (include/hss.h).  Every check
// runs before anything is enqueued, so a call that returns an error has launched nothing.
#include <algorithm>
#include <cmath>

#include "internal.h"

using namespace hss;

namespace {

constexpr int64_t kMostPages = int64_t{1} << 30;
constexpr int32_t kMostSeqs = 1 << 20;
constexpr float kMostScale = 0x1p100f;  // (the kernels multiply it by what a row was shifted by)

bool misaligned(const void* p, uintptr_t to) {
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

bool bad_stride(int64_t stride, int64_t width) {
    return stride < width || stride % 8 != 0 || stride > (int64_t{1} << 32);
}

bool outside(int64_t x, int64_t most) { return x < 0 || x > most; }

// The checks of hss_pack_kv_tokens and hss_unpack_kv_tokens; *nothing: no work is asked for.
hss_status check_pack(const hss_pack_args* args, const uint16_t* K, const uint16_t* V,
                      const uint8_t* cache, bool* nothing) {
    *nothing = true;
    if (args == nullptr) return HSS_ERR_NULL_POINTER;
    const hss_status st = hss_validate_dims(&args->dims);
    if (st != HSS_OK) return st;
    const int64_t width = static_cast<int64_t>(args->dims.num_kv_heads) * args->dims.head_dim;
    if (outside(args->num_tokens, int64_t{1} << 30) ||
        (K != nullptr && bad_stride(args->k_stride, width)) ||
        (V != nullptr && bad_stride(args->v_stride, width)))
        return HSS_ERR_INVALID_ARGUMENT;
    if (args->num_tokens == 0 || (K == nullptr && V == nullptr)) return HSS_OK;
    if (cache == nullptr || args->slots == nullptr) return HSS_ERR_NULL_POINTER;
    if (misaligned(K, 16) || misaligned(V, 16) || misaligned(cache, 16) ||
        misaligned(args->slots, 8) || misaligned(args->dev_status, 4))
        return HSS_ERR_MISALIGNED;
    *nothing = false;
    return HSS_OK;
}

}  // namespace

extern "C" {

size_t hss_packed_page_bytes(const hss_dims* dims) {
    if (hss_validate_dims(dims) != HSS_OK) return 0;
    return static_cast<size_t>(dims->num_kv_heads) * (dims->block_size / 16) * 18 * dims->head_dim;
}

hss_status hss_pack_kv_tokens(const hss_pack_args* args, const uint16_t* K, const uint16_t* V,
                              uint8_t* cache, void* stream) {
    bool nothing;
    const hss_status st = check_pack(args, K, V, cache, &nothing);
    if (st != HSS_OK || nothing) return st;
    return launch_pack(*args, K, V, cache, static_cast<cudaStream_t>(stream));
}

hss_status hss_unpack_kv_tokens(const hss_pack_args* args, const uint8_t* cache, uint16_t* K,
                                uint16_t* V, void* stream) {
    bool nothing;
    const hss_status st = check_pack(args, K, V, cache, &nothing);
    if (st != HSS_OK || nothing) return st;
    return launch_unpack(*args, cache, K, V, static_cast<cudaStream_t>(stream));
}

size_t hss_attend_packed_workspace_bytes(const hss_dims* dims, int32_t num_seqs, int32_t max_q,
                                         int64_t total_blocks, int32_t window, int32_t sinks) {
    if (hss_validate_dims(dims) != HSS_OK || num_seqs < 0 || max_q < 0 || total_blocks < 0 ||
        window < 0 || sinks < 0)
        return 0;
    return attend_packed_workspace_bytes(*dims, num_seqs, max_q, total_blocks, window, sinks);
}

hss_status hss_attend_packed(const hss_packed_args* args, const uint16_t* Q, const uint8_t* cache,
                             uint16_t* out, float* lse, void* stream) {
    if (args == nullptr) return HSS_ERR_NULL_POINTER;
    const hss_dims& d = args->dims;
    const hss_status st = hss_validate_dims(&d);
    if (st != HSS_OK) return st;
    if (d.num_q_heads / d.num_kv_heads > 128) return HSS_ERR_UNSUPPORTED_SHAPE;
    if (args->num_seqs < 0 || args->max_q < 0 || outside(args->total_q, 0x7FFFFFFF) ||
        outside(args->total_blocks, 0x7FFFFFFF) || args->window < 0 || args->sinks < 0 ||
        args->total_q > static_cast<int64_t>(args->num_seqs) * args->max_q ||
        (args->num_seqs == 0 && args->total_blocks != 0) || !(std::fabs(args->scale) <= kMostScale))
        return HSS_ERR_INVALID_ARGUMENT;
    // (rows of one kv head are counted in 32 bits)
    if (std::min<int64_t>(args->max_q, args->total_q) * (d.num_q_heads / d.num_kv_heads) >
        (int64_t{1} << 30))
        return HSS_ERR_INVALID_ARGUMENT;
    if (args->total_q == 0) return HSS_OK;
    if (args->q_offsets == nullptr || args->seq_offsets == nullptr || args->ctx_len == nullptr ||
        args->workspace == nullptr || (args->total_blocks > 0 && args->block_table == nullptr) ||
        Q == nullptr || cache == nullptr || out == nullptr)
        return HSS_ERR_NULL_POINTER;
    if (misaligned(Q, 16) || misaligned(cache, 16) || misaligned(out, 16) || misaligned(lse, 4) ||
        misaligned(args->workspace, 256) || misaligned(args->q_offsets, 4) ||
        misaligned(args->block_table, 4) || misaligned(args->seq_offsets, 4) ||
        misaligned(args->ctx_len, 4) || misaligned(args->dev_status, 4))
        return HSS_ERR_MISALIGNED;
    const size_t need = attend_packed_workspace_bytes(d, args->num_seqs, args->max_q,
                                                      args->total_blocks, args->window,
                                                      args->sinks);
    if (need == 0) return HSS_ERR_INVALID_ARGUMENT;
    if (args->workspace_bytes < need) return HSS_ERR_WORKSPACE_TOO_SMALL;
    return launch_attend_packed(PackedArgs{args, Q, cache, out, lse},
                                static_cast<cudaStream_t>(stream));
}

size_t hss_fork_pages_workspace_bytes(int32_t num_new, int64_t max_blocks) {
    if (num_new < 0 || outside(max_blocks, kMostPages)) return 0;
    return fork_workspace_bytes(num_new, max_blocks);
}

size_t hss_compact_pages_workspace_bytes(int64_t max_blocks) {
    if (outside(max_blocks, kMostPages)) return 0;
    return compact_workspace_bytes(max_blocks);
}

hss_status hss_fork_pages(const int32_t* block_table, const int32_t* seq_offsets,
                          int32_t num_seqs, int64_t total_blocks, const int32_t* refs,
                          int64_t max_blocks, const int32_t* released, int64_t num_released,
                          const int32_t* parents, const int32_t* lengths, const int32_t* room,
                          int32_t num_new, int32_t block_size, int64_t table_room,
                          int32_t* new_table, int32_t* new_offsets, int32_t* new_refs,
                          int32_t* copy_src, int32_t* copy_dst, int32_t* counts, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, void* stream) {
    if (outside(num_seqs, kMostSeqs) || outside(num_new, kMostSeqs) ||
        outside(total_blocks, kMostPages) || outside(max_blocks, kMostPages) ||
        outside(num_released, kMostPages) || outside(table_room, kMostPages) || block_size < 1 ||
        (num_seqs == 0 && total_blocks != 0))
        return HSS_ERR_INVALID_ARGUMENT;
    if (new_offsets == nullptr || counts == nullptr ||
        (num_seqs > 0 && seq_offsets == nullptr) || (total_blocks > 0 && block_table == nullptr) ||
        (max_blocks > 0 && (refs == nullptr || new_refs == nullptr)) ||
        (num_released > 0 && released == nullptr) || (table_room > 0 && new_table == nullptr) ||
        (num_new > 0 && (parents == nullptr || lengths == nullptr || room == nullptr ||
                         copy_src == nullptr || copy_dst == nullptr)) ||
        (workspace == nullptr && fork_workspace_bytes(num_new, max_blocks) > 0))
        return HSS_ERR_NULL_POINTER;
    const void* all[] = {block_table, seq_offsets, refs,     released, parents,  lengths,
                         room,        new_table,   new_offsets, new_refs, copy_src, copy_dst,
                         counts,      workspace,   dev_status};
    for (const void* p : all)
        if (misaligned(p, 4)) return HSS_ERR_MISALIGNED;
    if (workspace_bytes < fork_workspace_bytes(num_new, max_blocks))
        return HSS_ERR_WORKSPACE_TOO_SMALL;
    return launch_fork(ForkArgs{block_table, seq_offsets, num_seqs, total_blocks, refs, max_blocks,
                                released, num_released, parents, lengths, room, num_new,
                                block_size, table_room, new_table, new_offsets, new_refs, copy_src,
                                copy_dst, counts, static_cast<int32_t*>(workspace), dev_status},
                       static_cast<cudaStream_t>(stream));
}

hss_status hss_compact_pages(const int32_t* block_table, int64_t total_blocks, const int32_t* refs,
                             int64_t max_blocks, int64_t move_room, int32_t* new_table,
                             int32_t* new_refs, int32_t* copy_src, int32_t* copy_dst,
                             int32_t* counts, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream) {
    if (outside(total_blocks, kMostPages) || outside(max_blocks, kMostPages) ||
        outside(move_room, kMostPages))
        return HSS_ERR_INVALID_ARGUMENT;
    if (counts == nullptr ||
        (total_blocks > 0 && (block_table == nullptr || new_table == nullptr)) ||
        (max_blocks > 0 && (refs == nullptr || new_refs == nullptr || workspace == nullptr)) ||
        (move_room > 0 && (copy_src == nullptr || copy_dst == nullptr)))
        return HSS_ERR_NULL_POINTER;
    const void* all[] = {block_table, refs,   new_table, new_refs,  copy_src,
                         copy_dst,    counts, workspace, dev_status};
    for (const void* p : all)
        if (misaligned(p, 4)) return HSS_ERR_MISALIGNED;
    if (workspace_bytes < compact_workspace_bytes(max_blocks)) return HSS_ERR_WORKSPACE_TOO_SMALL;
    return launch_compact(CompactArgs{block_table, total_blocks, refs, max_blocks, move_room,
                                      new_table, new_refs, copy_src, copy_dst, counts,
                                      static_cast<int32_t*>(workspace), dev_status},
                          static_cast<cudaStream_t>(stream));
}

hss_status hss_copy_pages(const int32_t* copy_src, const int32_t* copy_dst,
                          const int32_t* num_copies, int64_t max_copies, void* pool0, void* pool1,
                          int64_t page_bytes, int64_t max_blocks, int32_t num_layers,
                          int32_t* dev_status, void* stream) {
    if (outside(max_copies, kMostPages) || outside(max_blocks, kMostPages) || page_bytes < 16 ||
        page_bytes > kMostPages || page_bytes % 16 != 0 || num_layers < 1 || num_layers > 65535)
        return HSS_ERR_INVALID_ARGUMENT;
    if (max_copies == 0) return HSS_OK;
    if (copy_src == nullptr || copy_dst == nullptr || pool0 == nullptr)
        return HSS_ERR_NULL_POINTER;
    if (misaligned(copy_src, 4) || misaligned(copy_dst, 4) || misaligned(num_copies, 4) ||
        misaligned(pool0, 16) || misaligned(pool1, 16) || misaligned(dev_status, 4))
        return HSS_ERR_MISALIGNED;
    return launch_copy_pages(CopyArgs{copy_src, copy_dst, num_copies, max_copies, pool0, pool1,
                                      page_bytes, max_blocks, num_layers, dev_status},
                             static_cast<cudaStream_t>(stream));
}

}  // extern "C"
