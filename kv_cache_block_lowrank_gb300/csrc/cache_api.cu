// cache_api.cu -- the C ABI of the operators around the paged cache (include/hss.h): rotary
// writes, tree attention, eviction by attention weight.  Every check runs before anything is
// enqueued, so a call that returns an error has launched nothing.
#include <cmath>

#include "internal.h"

using namespace hss;

namespace {

bool misaligned(const void* p, uintptr_t to) {
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

// A tensor of `rows` rows whose strides the call gives: at least `width` apart, 16-byte steps.
bool bad_stride(int64_t stride, int64_t width) {
    return stride < width || stride % 8 != 0 || stride > (int64_t{1} << 32);
}

// The checks of hss_rope_tokens and hss_norm_rope_tokens; *nothing: no work is asked for.
hss_status check_rope(const hss_rope_args& args, const uint16_t* Q, const uint16_t* K,
                      const uint16_t* V, const uint16_t* Q_out, const uint16_t* K_out,
                      const uint16_t* K_cache, const uint16_t* V_cache, bool* nothing) {
    const hss_dims& d = args.dims;
    *nothing = true;
    const hss_status st = hss_validate_dims(&d);
    if (st != HSS_OK) return st;
    if (args.rot_dim < 2 || args.rot_dim % 2 != 0 || args.rot_dim > d.head_dim ||
        (args.layout != HSS_ROPE_HALF && args.layout != HSS_ROPE_INTERLEAVED) ||
        !std::isfinite(args.magnitude) || args.num_tokens < 0 ||
        args.num_tokens > (int64_t{1} << 30))
        return HSS_ERR_INVALID_ARGUMENT;
    if (args.num_tokens == 0) return HSS_OK;
    const bool k_asked = K_out != nullptr || K_cache != nullptr;
    if ((Q_out != nullptr && Q == nullptr) || (k_asked && K == nullptr) ||
        (V_cache != nullptr && V == nullptr))
        return HSS_ERR_NULL_POINTER;
    if ((Q_out != nullptr || k_asked) && (args.turns == nullptr || args.positions == nullptr))
        return HSS_ERR_NULL_POINTER;
    if ((K_cache != nullptr || V_cache != nullptr) && args.slots == nullptr)
        return HSS_ERR_NULL_POINTER;
    if (misaligned(Q, 16) || misaligned(K, 16) || misaligned(V, 16) || misaligned(Q_out, 16) ||
        misaligned(K_out, 16) || misaligned(K_cache, 16) || misaligned(V_cache, 16) ||
        misaligned(args.turns, 8) || misaligned(args.positions, 8) ||
        misaligned(args.slots, 8) || misaligned(args.dev_status, 4))
        return HSS_ERR_MISALIGNED;
    const int64_t hd = d.head_dim;
    if ((Q_out != nullptr && bad_stride(args.q_stride, d.num_q_heads * hd)) ||
        (k_asked && bad_stride(args.k_stride, d.num_kv_heads * hd)) ||
        (V_cache != nullptr && bad_stride(args.v_stride, d.num_kv_heads * hd)))
        return HSS_ERR_INVALID_ARGUMENT;
    *nothing = Q_out == nullptr && !k_asked && V_cache == nullptr;
    return HSS_OK;
}

}  // namespace

extern "C" {

hss_status hss_rope_table(const hss_rope* rope, uint64_t* turns) {
    if (rope == nullptr || turns == nullptr) return HSS_ERR_NULL_POINTER;
    const int rot = rope->rot_dim;
    if (rot < 2 || rot % 2 != 0 || rot > 256) return HSS_ERR_INVALID_ARGUMENT;
    const bool scaled = rope->scaling != HSS_ROPE_SCALE_NONE;
    if (!(rope->base > 0) || !std::isfinite(rope->base)) return HSS_ERR_INVALID_ARGUMENT;
    if (scaled && (!(rope->factor > 0) || !std::isfinite(rope->factor)))
        return HSS_ERR_INVALID_ARGUMENT;
    double base = rope->base;
    const double two_pi = 2.0 * std::acos(-1.0);
    switch (rope->scaling) {
        case HSS_ROPE_SCALE_NONE:
        case HSS_ROPE_SCALE_LINEAR: break;
        case HSS_ROPE_SCALE_BASE:
            if (rot == 2) return HSS_ERR_INVALID_ARGUMENT;
            base *= std::pow(rope->factor, rot / (rot - 2.0));
            // (a base past the range of a double would leave pairs unturned)
            if (!(base > 0) || !std::isfinite(base)) return HSS_ERR_INVALID_ARGUMENT;
            break;
        case HSS_ROPE_SCALE_RAMP:
            if (!(rope->original_ctx > 0) || !std::isfinite(rope->original_ctx) ||
                !std::isfinite(rope->low) || !std::isfinite(rope->high) ||
                !(rope->low < rope->high) || !std::isfinite(rope->high - rope->low))
                return HSS_ERR_INVALID_ARGUMENT;
            break;
        default: return HSS_ERR_INVALID_ARGUMENT;
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (rope->scaling == HSS_ROPE_SCALE_LINEAR) f /= rope->factor;
        if (rope->scaling == HSS_ROPE_SCALE_RAMP) {
            const double n = rope->original_ctx * f / two_pi;
            double w = (n - rope->low) / (rope->high - rope->low);
            w = w < 0 ? 0 : (w > 1 ? 1 : w);
            f = f * w + f / rope->factor * (1.0 - w);
        }
        if (!std::isfinite(f)) return HSS_ERR_INVALID_ARGUMENT;
        // Positions are whole numbers, so whole turns per position drop out.
        const double t = std::rint(std::ldexp(std::fmod(f / two_pi, 1.0), 64));
        turns[i] = t >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(t);
    }
    return HSS_OK;
}

hss_status hss_rope_tokens(const hss_rope_args* args, const uint16_t* Q, const uint16_t* K,
                           const uint16_t* V, uint16_t* Q_out, uint16_t* K_out,
                           uint16_t* K_cache, uint16_t* V_cache, void* stream) {
    if (args == nullptr) return HSS_ERR_NULL_POINTER;
    bool nothing;
    const hss_status st =
        check_rope(*args, Q, K, V, Q_out, K_out, K_cache, V_cache, &nothing);
    if (st != HSS_OK || nothing) return st;
    return launch_rope(RopeArgs{args, Q, K, V, Q_out, K_out, K_cache, V_cache},
                       static_cast<cudaStream_t>(stream));
}

hss_status hss_norm_rope_tokens(const hss_norm_rope_args* args, const uint16_t* Q,
                                const uint16_t* K, const uint16_t* V, const uint16_t* q_weight,
                                const uint16_t* k_weight, uint16_t* Q_out, uint16_t* K_out,
                                uint16_t* K_cache, uint16_t* V_cache, void* stream) {
    if (args == nullptr) return HSS_ERR_NULL_POINTER;
    bool nothing;
    const hss_status st =
        check_rope(args->rope, Q, K, V, Q_out, K_out, K_cache, V_cache, &nothing);
    if (st != HSS_OK) return st;
    const int64_t hd = args->rope.dims.head_dim;
    if (!(args->eps >= 0) || !std::isfinite(args->eps) || !std::isfinite(args->weight_offset) ||
        (args->q_weight_stride != 0 && bad_stride(args->q_weight_stride, hd)) ||
        (args->k_weight_stride != 0 && bad_stride(args->k_weight_stride, hd)))
        return HSS_ERR_INVALID_ARGUMENT;
    if (misaligned(q_weight, 16) || misaligned(k_weight, 16)) return HSS_ERR_MISALIGNED;
    if (nothing) return HSS_OK;
    return launch_norm_rope(NormRopeArgs{args, Q, K, V, q_weight, k_weight, Q_out, K_out, K_cache,
                                         V_cache},
                            static_cast<cudaStream_t>(stream));
}

size_t hss_attend_tree_workspace_bytes(const hss_dims* dims, int32_t num_seqs, int32_t max_q,
                                       int64_t total_blocks, int32_t with_weights) {
    if (hss_validate_dims(dims) != HSS_OK || num_seqs < 0 || max_q < 0 || total_blocks < 0)
        return 0;
    return attend_workspace_bytes(*dims, num_seqs, max_q, total_blocks, with_weights != 0);
}

hss_status hss_attend_tree(const hss_attend_args* args, const uint16_t* Q,
                           const uint16_t* K_cache, const uint16_t* V_cache, uint16_t* out,
                           float* lse, const float* weights_in, float* weights_out,
                           void* stream) {
    if (args == nullptr) return HSS_ERR_NULL_POINTER;
    const hss_dims& d = args->dims;
    const hss_status st = hss_validate_dims(&d);
    if (st != HSS_OK) return st;
    if (d.num_q_heads / d.num_kv_heads > 128) return HSS_ERR_UNSUPPORTED_SHAPE;
    if (args->num_seqs < 0 || args->max_q < 0 || args->total_q < 0 || args->total_blocks < 0 ||
        args->total_blocks > 0x7FFFFFFF || args->total_q > 0x7FFFFFFF ||
        args->total_q > static_cast<int64_t>(args->num_seqs) * args->max_q ||
        (args->num_seqs == 0 && args->total_blocks != 0) || !std::isfinite(args->scale) ||
        !std::isfinite(args->decay) || args->mask_words < 0 ||
        (args->tree_mask != nullptr && args->mask_words < 1))
        return HSS_ERR_INVALID_ARGUMENT;
    const bool rows = args->total_q > 0;
    const bool weigh = weights_out != nullptr && args->total_blocks > 0;
    if (!rows && !weigh) return HSS_OK;
    if (args->q_offsets == nullptr || args->seq_offsets == nullptr || args->ctx_len == nullptr ||
        args->workspace == nullptr || (args->total_blocks > 0 && args->block_table == nullptr) ||
        (rows && (Q == nullptr || K_cache == nullptr || V_cache == nullptr || out == nullptr)))
        return HSS_ERR_NULL_POINTER;
    if (misaligned(Q, 16) || misaligned(K_cache, 16) || misaligned(V_cache, 16) ||
        misaligned(out, 16) || misaligned(lse, 4) || misaligned(weights_in, 4) ||
        misaligned(weights_out, 4) || misaligned(args->tree_mask, 8) ||
        misaligned(args->workspace, 256) || misaligned(args->q_offsets, 4) ||
        misaligned(args->block_table, 4) || misaligned(args->seq_offsets, 4) ||
        misaligned(args->ctx_len, 4) || misaligned(args->dev_status, 4))
        return HSS_ERR_MISALIGNED;
    if (args->workspace_bytes < attend_workspace_bytes(d, args->num_seqs, args->max_q,
                                                       args->total_blocks, weigh))
        return HSS_ERR_WORKSPACE_TOO_SMALL;
    return launch_attend(AttendArgs{args, Q, K_cache, V_cache, out, lse, weights_in,
                                    weigh ? weights_out : nullptr},
                         static_cast<cudaStream_t>(stream));
}

hss_status hss_evict_blocks(const float* weights, const int32_t* block_table,
                            const int32_t* seq_offsets, const int32_t* ctx_len,
                            const int32_t* budgets, int32_t num_seqs, int64_t total_blocks,
                            int32_t block_size, int32_t keep_first, int32_t keep_last,
                            int32_t* new_table, int32_t* new_offsets, float* new_weights,
                            int32_t* new_ctx_len, int32_t* freed, int32_t* freed_offsets,
                            void* stream) {
    if (num_seqs < 0 || total_blocks < 0 || total_blocks > (1 << 30) || block_size < 1 ||
        keep_first < 0 || keep_last < 0 || (num_seqs == 0 && total_blocks != 0))
        return HSS_ERR_INVALID_ARGUMENT;
    if (num_seqs == 0) return HSS_OK;
    if (seq_offsets == nullptr || budgets == nullptr || new_offsets == nullptr ||
        freed_offsets == nullptr || (ctx_len == nullptr) != (new_ctx_len == nullptr))
        return HSS_ERR_NULL_POINTER;
    if (total_blocks > 0 && (weights == nullptr || block_table == nullptr ||
                             new_table == nullptr || new_weights == nullptr || freed == nullptr))
        return HSS_ERR_NULL_POINTER;
    const void* all[] = {weights, block_table, seq_offsets, ctx_len,     budgets, new_table,
                         new_offsets, new_weights, new_ctx_len, freed, freed_offsets};
    for (const void* p : all)
        if (misaligned(p, 4)) return HSS_ERR_MISALIGNED;
    return launch_evict(EvictArgs{weights, block_table, seq_offsets, ctx_len, budgets, num_seqs,
                                  total_blocks, block_size, keep_first, keep_last, new_table,
                                  new_offsets, new_weights, new_ctx_len, freed, freed_offsets},
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
