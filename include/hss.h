/*
 * hss.h -- C ABI of the GB300 (sm_103a) low-rank KV-block predictor.
 *
 * The predictor ("high-speed swap" block predictor, page
 * "metrale_storage/predictor.rs", module docs) keeps, for every key token of
 * every paged KV block, a low-rank copy of the key:
 *
 *     A_g[layer][block][kv_head][token][j] = bf16( sum_d K[token][kv_head][d] * P[d][j] )
 *
 * and scores each block against the current queries as the largest projected
 * dot product Qp . A_g over query heads, query rows and the block's tokens.
 * The lowest-scoring blocks are the eviction victims.
 *
 * Conventions for every call:
 *   - bf16 tensors are passed as uint16_t bit patterns (IEEE binary32 upper
 *     halves); every tensor is dense, row-major, in the layout stated.
 *   - Pointers marked "device" must point to memory of the current CUDA
 *     device; the caller owns every buffer.  The library allocates no memory
 *     and keeps no state between calls other than the per-device kernel set-up
 *     done on first use and one device-resident error word (see
 *     hss_read_device_error).
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     compute call only validates its arguments on the host and enqueues work
 *     on that stream; it returns before the work is done.  Nothing is enqueued
 *     when a call returns an error.
 *   - Argument errors are reported synchronously by the return value.  Errors
 *     that depend on device-resident data (a block id out of range) are
 *     reported through the optional `dev_status` word (device int32): the
 *     kernel stores the first error code into it if it is still HSS_OK; the
 *     caller zeroes it before the call and reads it after synchronising.
 */
#ifndef HSS_H
#define HSS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The seven predictor dimensions (PredictorDims on the predictor page).
 * num_q_heads must be a multiple of num_kv_heads (PredictorDims::validate);
 * query head h reads kv head h / (num_q_heads / num_kv_heads).
 * Shapes the kernels support: head_dim in {64, 128, 192, 256}; r in {16, 32, 64, 128};
 * block_size a multiple of 16 in [16, 256] (the tensor-core scorer: 16 or 32);
 * num_kv_heads <= 64; max_blocks <= 2^31 - 1. */
typedef struct hss_dims {
    int32_t num_layers;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t r;
    int32_t block_size;
    int64_t max_blocks;
} hss_dims;

typedef enum hss_status {
    HSS_OK = 0,
    HSS_ERR_INVALID_DIMS = 1,        /* a dimension is <= 0, or num_q_heads % num_kv_heads != 0 */
    HSS_ERR_OUT_OF_RANGE = 2,        /* layer >= num_layers, or a block id outside [0, max_blocks) */
    HSS_ERR_NULL_POINTER = 3,        /* a required pointer is NULL */
    HSS_ERR_MISALIGNED = 4,          /* a bf16 tensor is not 16-byte aligned */
    HSS_ERR_WORKSPACE_TOO_SMALL = 5, /* a caller workspace (hss_layer_step) or the static
                                        array (hss_layer_step_static) is too small */
    HSS_ERR_UNSUPPORTED_SHAPE = 6,   /* valid dims that no kernel here handles */
    HSS_ERR_CUDA = 7,                /* a CUDA runtime call or a launch failed */
    HSS_ERR_DEVICE_TIMEOUT = 8,      /* a kernel gave up waiting on a pipeline barrier */
    HSS_ERR_INVALID_ARGUMENT = 9     /* a count or size is negative or inconsistent */
} hss_status;

/* Human-readable name of a status code (static storage; never NULL). */
const char* hss_status_string(int32_t status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t hss_version(void);

/* HSS_OK if the dims are valid (PredictorDims::validate) and supported. */
hss_status hss_validate_dims(const hss_dims* dims);

/* Bytes of the per-token low-rank key store A_g,
 * num_layers * max_blocks * num_kv_heads * block_size * r * 2
 * (PredictorDims::a_g_bytes, predictor page); 0 if dims is NULL or invalid. */
size_t hss_a_g_bytes(const hss_dims* dims);

/*
 * Query projection: Qp = Q . P, rounded once to bf16 (round to nearest even).
 * Page "metrale_storage/predictor.rs", Predictor::project_q ("q_proj = q @ P";
 * q is [num_q_heads, head_dim] BF16, q_proj [num_q_heads, r] BF16), extended
 * here to many query rows.
 *
 *   P    device, [head_dim, r] bf16, 16-byte aligned
 *   Q    device, [num_rows, num_q_heads, head_dim] bf16, 16-byte aligned
 *   Qp   device, [num_rows, num_q_heads, r] bf16, 16-byte aligned (output)
 *   num_rows >= 0 query rows (num_rows = 0 enqueues nothing)
 * Accumulation is fp32 on the tensor cores.
 */
hss_status hss_project_q(const hss_dims* dims, const uint16_t* P, const uint16_t* Q,
                         int64_t num_rows, uint16_t* Qp, void* stream);

/*
 * Key projection of whole blocks into A_g:
 *   A_g[layer][block_ids[i]][h][t][j] = bf16( sum_d K[i][t][h][d] * P[d][j] ).
 * Page "metrale_storage/predictor.rs", Predictor::project_kv_block (k_block is
 * [block_size, num_kv_heads, head_dim] BF16, token-major; the A_g slot is
 * [num_kv_heads, block_size, r], head-major; an out-of-range layer or block
 * is an error), batched here over num_blocks blocks per call.
 *
 *   P          device, [head_dim, r] bf16, 16-byte aligned
 *   K          device, [num_blocks, block_size, num_kv_heads, head_dim] bf16,
 *              16-byte aligned
 *   layer      0 <= layer < num_layers, else HSS_ERR_OUT_OF_RANGE
 *   block_ids  device, [num_blocks] int32; ids should be distinct (two
 *              entries with the same id race for the slot).  An id outside
 *              [0, max_blocks) is skipped and sets *dev_status to
 *              HSS_ERR_OUT_OF_RANGE.
 *   A_g        device, [num_layers, max_blocks, num_kv_heads, block_size, r]
 *              bf16, 16-byte aligned; only the addressed slots are written
 *   dev_status device int32 or NULL
 */
hss_status hss_project_kv_blocks(const hss_dims* dims, const uint16_t* P, const uint16_t* K,
                                 int32_t layer, const int32_t* block_ids, int64_t num_blocks,
                                 uint16_t* A_g, int32_t* dev_status, void* stream);

/*
 * Cache write with projection: the page's ingest (Predictor::project_kv_block, launched once
 * per block after a block is written) moved to where the layer's new keys are written, one
 * token at a time.  For every token i with slot s = slots[i] = block * block_size + t:
 *   K_cache[s / block_size][s % block_size][h][:] = K_tok[i][h][:]        (if K_cache != NULL)
 *   A_g[layer][s / block_size][h][s % block_size][:] = bf16(K_tok[i][h] . P)
 * for every kv head h, in one launch.  A decode step (one new token per sequence) thus keeps
 * A_g current without waiting for a block to fill; the rows of positions not yet written
 * keep what they held (score such blocks with a ctx_len mask, hss_score_blocks_masked).
 *   K_tok    device, [num_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned: the layer's
 *            keys of the new tokens
 *   slots    device, [num_tokens] int64, 8-byte aligned.  A negative slot marks a padding
 *            token: nothing is written for it.  A slot >= max_blocks * block_size is skipped
 *            and raises HSS_ERR_OUT_OF_RANGE in *dev_status (if not NULL) and the library's
 *            device error word.  If two tokens name one slot, each 16 bytes of
 *            its rows are one token's or the other's: name it once.
 *   K_cache  device, [max_blocks, block_size, num_kv_heads, head_dim] bf16, 16-byte aligned:
 *            this layer's paged key cache (each block in the page's k_block layout), or NULL
 *            to write A_g only
 *   A_g      as in hss_project_kv_blocks
 * Each A_g row equals what hss_project_kv_blocks writes for that position (the same kernel
 * computes it).  Errors as hss_project_kv_blocks.
 */
hss_status hss_write_kv_tokens(const hss_dims* dims, const uint16_t* P, const uint16_t* K_tok,
                               const int64_t* slots, int64_t num_tokens, uint16_t* K_cache,
                               uint16_t* A_g, int32_t layer, int32_t* dev_status, void* stream);

/* Score kernel choice for hss_score_blocks. */
#define HSS_PATH_AUTO 0    /* decode kernel when rows_per_seq * (num_q_heads/num_kv_heads) <= 16,
                              else the tensor-memory (tcgen05) kernel */
#define HSS_PATH_DECODE 1  /* streaming kernel: warp-level MMA per block, A_g read once */
#define HSS_PATH_TCGEN05 2 /* dense kernel for prefill chunks: tcgen05 MMA, TMEM accumulators */

/*
 * Block scores:
 *   scores[i] = max over query rows, query heads h and tokens t of block
 *               block_table[i] of  sum_j Qp[s][row][h][j] * A_g[layer][block_table[i]][h/g][t][j]
 * for i in sequence s (seq_offsets[s] <= i < seq_offsets[s+1]), g =
 * num_q_heads / num_kv_heads.  No scaling, no masking: every token of the
 * block is scored.  Page "metrale_storage/predictor.rs",
 * Predictor::score_blocks (the max over query heads and tokens of the
 * projected dot product, f32 out); that call scores contiguous slots, which
 * an identity table reproduces.
 *
 *   Qp           device, [num_seqs, rows_per_seq, num_q_heads, r] bf16,
 *                16-byte aligned
 *   rows_per_seq >= 1 query rows per sequence
 *   A_g          device, as in hss_project_kv_blocks
 *   block_table  device, [total_blocks] int32 physical block ids
 *   seq_offsets  device, [num_seqs + 1] int32, non-decreasing,
 *                seq_offsets[0] = 0, seq_offsets[num_seqs] = total_blocks
 *   scores       device, [total_blocks] f32 (output)
 *   path         HSS_PATH_*
 *   dev_status   device int32 or NULL.  A table entry outside
 *                [0, max_blocks) gets score +inf (so it is never a victim)
 *                and sets HSS_ERR_OUT_OF_RANGE.
 * Accumulation is fp32; the result differs from an exact sum by at most
 * about r * 2^-23 * sum_j |Qp_j * A_j|.
 */
hss_status hss_score_blocks(const hss_dims* dims, const uint16_t* Qp, int32_t rows_per_seq,
                            const uint16_t* A_g, int32_t layer, const int32_t* block_table,
                            const int32_t* seq_offsets, int32_t num_seqs, int64_t total_blocks,
                            float* scores, int32_t path, int32_t* dev_status, void* stream);

/*
 * Block scores restricted to visible tokens: hss_score_blocks with two optional masks.
 * Token t of the entry at table position j of sequence s (j counted from seq_offsets[s])
 * sits at position p = j * block_size + t.
 *   ctx_len   device, [num_seqs] int32, or NULL: only tokens with p < ctx_len[s] count
 *             (the tail of a partly filled last block, or blocks past the context);
 *   row_pos0  device, [num_seqs] int32, or NULL: causal mask for a chunk of query rows
 *             whose first row sits at row_pos0[s]; row r sees only p <= row_pos0[s] + r.
 * A block with no visible candidate scores -inf.  Both NULL: exactly hss_score_blocks.
 * The predictor page's scorer takes no lengths or positions (Predictor::score_blocks);
 * these masks are the next step it leaves open.  Seeing a key only from rows at or after
 * its position follows the complete-block count of "metrale_model_layers/layers/
 * qsa_select.rs" (QsaIndexer::prefill_select).
 */
hss_status hss_score_blocks_masked(const hss_dims* dims, const uint16_t* Qp, int32_t rows_per_seq,
                                   const uint16_t* A_g, int32_t layer, const int32_t* block_table,
                                   const int32_t* seq_offsets, int32_t num_seqs,
                                   int64_t total_blocks, const int32_t* ctx_len,
                                   const int32_t* row_pos0, float* scores, int32_t path,
                                   int32_t* dev_status, void* stream);

/* Largest k that hss_rank_victims accepts. */
#define HSS_MAX_VICTIMS 8192

/*
 * Eviction victims: for each sequence s, the min(k, n_s) table entries with
 * the smallest scores, in ascending order of (score, entry index), written as
 * indices into that sequence's own table (0 .. n_s - 1); the rest of the row
 * is -1.  -0 ranks equal to +0; NaN ranks as +inf.  The predictor page says
 * the scores serve only to rank eviction victims (module docs of
 * "metrale_storage/predictor.rs"); the lower-index-first rule for equal scores
 * mirrors the host top-k of "metrale_model_layers/layers/qsa_select.rs".
 *
 *   scores       device, [total_blocks] f32
 *   seq_offsets  device, [num_seqs + 1] int32, as in hss_score_blocks
 *   k            1 <= k <= HSS_MAX_VICTIMS
 *   victims      device, [num_seqs, k] int32 (output)
 * The result is exact (integer output, no tolerance).
 */
hss_status hss_rank_victims(const float* scores, const int32_t* seq_offsets, int32_t num_seqs,
                            int64_t total_blocks, int32_t k, int32_t* victims, void* stream);

/*
 * Per-row block scores (QSA-style selection, the host top-k of the page
 * "metrale_model_layers/layers/qsa_select.rs" done on the GPU, with this predictor's score):
 * for one sequence's chunk of query rows, each row on its own,
 *   scores[row * num_blocks + j] = max over query heads h and the tokens t of block
 *       block_table[j] of  sum_k Qp[row][h][k] * A_g[layer][block_table[j]][h / g][t][k]
 * i.e. the block score of hss_score_blocks without the max over rows.  Runs on the tcgen05
 * scorer (the dense prefill contraction).
 *   Qp           device, [rows, num_q_heads, r] bf16, 16-byte aligned
 *   block_table  device, [num_blocks] int32: the sequence's physical block ids, in order
 *   scores       device, [rows, num_blocks] f32 (output)
 * Supported: g = num_q_heads / num_kv_heads in {1, 2, 4, 8, 16}, block_size 16 or 32, and
 * the tcgen05 scorer's shapes; otherwise HSS_ERR_UNSUPPORTED_SHAPE.  An id outside
 * [0, max_blocks) scores -inf in every row (never selected) and raises HSS_ERR_OUT_OF_RANGE
 * in *dev_status (if not NULL) and the library's device error word.
 */
hss_status hss_score_rows(const hss_dims* dims, const uint16_t* Qp, int32_t rows,
                          const uint16_t* A_g, int32_t layer, const int32_t* block_table,
                          int64_t num_blocks, float* scores, int32_t* dev_status, void* stream);

/*
 * Per-row top-k selection (the host top-k per row of the page
 * "metrale_model_layers/layers/qsa_select.rs", QsaIndexer::prefill_select, on the GPU).
 * Row r of a prefill chunk whose first row sits at position first_pos has seen the blocks
 *   j < complete_r = min(num_blocks, (first_pos + r + 1) / block_size)
 * whole; its list holds the topk of them with the largest scores[r * num_blocks + j],
 * larger first, the lower index first among equal scores (-0 equals +0; NaN ranks like
 * -inf, below every number), as indices j; lists[r * topk + i] = -1 where i >= complete_r.
 *   scores  device, [rows, num_blocks] f32 (e.g. from hss_score_rows)
 *   lists   device, [rows, topk] int32 (output); 1 <= topk <= HSS_MAX_VICTIMS
 * The result is exact (integer output).
 */
hss_status hss_select_rows(const float* scores, int32_t rows, int64_t num_blocks,
                           int64_t first_pos, int32_t block_size, int32_t topk, int32_t* lists,
                           void* stream);

/*
 * One predictor layer call in as few launches as the shape allows: project the newly
 * written blocks into A_g and the query rows into Qp (one launch), score every table
 * entry, and rank the victims of every sequence.  Results are the same as
 *   hss_project_kv_blocks(K_new, new_ids) ; hss_project_q(Q) ; hss_score_blocks(path AUTO) ;
 *   hss_rank_victims
 * on the same stream (the same kernels compute them; the victims are the same words in
 * the same order).  In the decode regime the victim ranking runs inside the scoring kernel:
 * for at most 8 sequences and 4096 blocks in all, when the scoring grid fits on the GPU at
 * once, every CTA publishes its blocks' keys in the workspace, waits until all the call's
 * keys are there (a bounded wait: HSS_ERR_DEVICE_TIMEOUT after 1 s) and places its own blocks
 * by counting the smaller (sequence, score, position) words; otherwise the last CTA to finish
 * a sequence ranks it.  That bounded wait assumes the scoring grid gets the whole GPU: a kernel of
 * another stream that holds SMs for longer than the limit makes the call report
 * HSS_ERR_DEVICE_TIMEOUT (its victims are then wrong; zero the workspace before the next call).
 * This is the fused decode call the predictor page's per-step usage implies (module docs
 * of "metrale_storage/predictor.rs": scores only rank eviction victims).
 *
 *   K_new, new_ids, num_new  blocks written this step (num_new may be 0), as in
 *                            hss_project_kv_blocks
 *   Q                        device, [num_seqs, rows_per_seq, num_q_heads, head_dim] bf16
 *   Qp                       device, [num_seqs, rows_per_seq, num_q_heads, r] bf16 (output),
 *                            or NULL when the caller does not need the projected queries.
 *                            With NULL, the decode scorer projects the queries itself (into
 *                            shared memory; Qp is never stored), so the scoring path has one
 *                            launch fewer: only the new blocks are projected before it, and it
 *                            waits for that projection only where it reads a new block.  NULL
 *                            is accepted when the call takes the decode scorer (rows_per_seq *
 *                            num_q_heads / num_kv_heads <= 16), num_seqs <= 8, and the query
 *                            rows, P and the projected fragments fit the scorer's 96 KiB of
 *                            shared memory (the Llama-3-8B-like decode layer, 32 q / 8 kv
 *                            heads, head_dim 128, r 32, one row, needs 22 KiB); otherwise the
 *                            call returns HSS_ERR_NULL_POINTER.  The scores then come from
 *                            the same fp32-accumulated, bf16-rounded Qp, summed in another
 *                            order, so a Qp element may differ from hss_project_q's by one
 *                            bf16 ulp.
 *   scores, victims          outputs, as in hss_score_blocks / hss_rank_victims
 *   workspace                device, >= hss_layer_step_workspace_bytes(num_seqs) bytes,
 *                            4-byte aligned (16-byte aligned for the in-kernel ranking of
 *                            at most 8 sequences above): that ranking's call number and 32 KiB of
 *                            tagged keys (33024 bytes), then the per-sequence completion
 *                            counters, so calls with different num_seqs may share one
 *                            workspace sized for the largest.  Zero all of it once
 *                            (e.g. cudaMemsetAsync) before its first use, then leave it as
 *                            each call leaves it: the counters return to zero, the call
 *                            number and the keys carry over to the next call (zeroing all
 *                            of it again is also fine; after HSS_ERR_DEVICE_TIMEOUT, do).
 *                            Two calls that share a workspace must not run at the same time
 *                            on the GPU.
 * Errors as in the four calls above; HSS_ERR_WORKSPACE_TOO_SMALL if the workspace is short.
 */
size_t hss_layer_step_workspace_bytes(int32_t num_seqs);

hss_status hss_layer_step(const hss_dims* dims, const uint16_t* P, const uint16_t* K_new,
                          const int32_t* new_ids, int64_t num_new, const uint16_t* Q,
                          int32_t rows_per_seq, uint16_t* Qp, uint16_t* A_g, int32_t layer,
                          const int32_t* block_table, const int32_t* seq_offsets,
                          int32_t num_seqs, int64_t total_blocks, float* scores, int32_t k,
                          int32_t* victims, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, void* stream);

/*
 * hss_layer_step with the arguments that stay the same from call to call bound once in a
 * struct (a serving loop's layer calls differ only in the layer, the new key blocks, the
 * queries, the outputs and the stream): one call is exactly
 *   hss_layer_step(&args->dims, args->P, K_new, args->new_ids, args->num_new, Q,
 *                  args->rows_per_seq, args->Qp, args->A_g, layer, args->block_table,
 *                  args->seq_offsets, args->num_seqs, args->total_blocks, scores, args->k,
 *                  victims, args->workspace, args->workspace_bytes, args->dev_status, stream)
 * with every argument's meaning, layout, ownership and error as there; the struct is read
 * during the call only (the caller keeps it).  A calling convention of this library (the
 * pages have no counterpart): fewer arguments to marshal per call for bindings whose
 * per-argument cost shows beside a 10 us layer call.  HSS_ERR_NULL_POINTER if args is NULL.
 */
typedef struct hss_layer_step_args {
    hss_dims dims;
    const uint16_t* P;
    const int32_t* new_ids;
    int64_t num_new;
    int32_t rows_per_seq;
    uint16_t* Qp;
    uint16_t* A_g;
    const int32_t* block_table;
    const int32_t* seq_offsets;
    int32_t num_seqs;
    int64_t total_blocks;
    int32_t k;
    void* workspace;
    size_t workspace_bytes;
    int32_t* dev_status;
} hss_layer_step_args;

hss_status hss_layer_step_bound(const hss_layer_step_args* args, int32_t layer,
                                const uint16_t* K_new, const uint16_t* Q, float* scores,
                                int32_t* victims, void* stream);

/*
 * hss_layer_step for callers that cannot allocate device memory.  (The predictor pages have
 * no counterpart: this is a calling convention of this library.)
 *
 * hss_layer_step needs a caller-allocated workspace.  Some callers cannot call cudaMalloc
 * there: an engine whose memory arena owns the GPU's memory and allows no allocation after
 * start-up, a library hosted by a process that hands it no allocator, or a caller that only
 * holds raw pointers to its own buffers.  This variant takes no workspace: the completion
 * counters live in a fixed array inside the library, HSS_LAYER_STEP_STATIC_MAX_SEQS int32
 * words and 32.25 KiB more (48.25 KiB) on every GPU that loads it, kept until the process
 * exits.  It allocates
 * nothing and calls no allocating routine.
 *
 *   Arguments and results: as hss_layer_step, without workspace / workspace_bytes; Qp must
 *   not be NULL here (HSS_ERR_NULL_POINTER).
 *   Every argument check runs before anything is enqueued, as for the other calls.
 *   num_seqs > HSS_LAYER_STEP_STATIC_MAX_SEQS  -> HSS_ERR_WORKSPACE_TOO_SMALL, nothing enqueued.
 *   Each call first clears the counters it uses (a memset on `stream`), then runs the same
 *   kernels as hss_layer_step.
 *   The first call on a device looks up the array's device address (cudaGetSymbolAddress);
 *   make that first call before any stream capture on that device.  The address is kept
 *   for the life of the process: after cudaDeviceReset on that device, reload the library
 *   before calling this again (the same holds for the library's error word).
 *   All calls share the one array: calls that overlap on the GPU (on different streams, or
 *   unordered) race and give wrong victims.  Order them on one stream.
 */
#define HSS_LAYER_STEP_STATIC_MAX_SEQS 4096

int32_t hss_layer_step_static_max_seqs(void);

hss_status hss_layer_step_static(const hss_dims* dims, const uint16_t* P, const uint16_t* K_new,
                                 const int32_t* new_ids, int64_t num_new, const uint16_t* Q,
                                 int32_t rows_per_seq, uint16_t* Qp, uint16_t* A_g, int32_t layer,
                                 const int32_t* block_table, const int32_t* seq_offsets,
                                 int32_t num_seqs, int64_t total_blocks, float* scores, int32_t k,
                                 int32_t* victims, int32_t* dev_status, void* stream);

/*
 * Rotary positions (RoFormer's rotary embedding; the predictor pages take keys and queries as
 * they come, so no page has a counterpart).  A head's first rot_dim elements are rotated in
 * pairs, pair i of a token at position pos by the angle
 *     a(pos, i) = 2 pi frac(pos * turns[i] / 2^64),
 * where turns[i] is the pair's frequency as a 64-bit fixed-point fraction of a turn per
 * position.  The product of two whole numbers modulo 2^64 is exact, so an angle is as good as its
 * frequency, which hss_rope_table gives within a few parts in 2^53: at position 2^27 it is off by
 * less than the 1e-7 radians of its rounding to fp32, at 2^40 by up to 1e-3 (a 32-bit frequency
 * times a position of 131072 is off by up to 0.008 radians).  A negative position turns back by the
 * same angle (the transposed rotation, which the gradient of a rotated row needs).
 */
#define HSS_ROPE_HALF 0        /* pair i = elements (i, i + rot_dim / 2) */
#define HSS_ROPE_INTERLEAVED 1 /* pair i = elements (2 i, 2 i + 1) */

/* Frequencies f_i = base^(-2 i / rot_dim) radians per position, for longer contexts scaled as */
#define HSS_ROPE_SCALE_NONE 0   /* f_i */
#define HSS_ROPE_SCALE_LINEAR 1 /* f_i / factor (position interpolation) */
#define HSS_ROPE_SCALE_BASE 2   /* f_i of base * factor^(rot_dim / (rot_dim - 2)); rot_dim > 2 */
#define HSS_ROPE_SCALE_RAMP 3   /* w f_i + (1 - w) f_i / factor, with w going from 0 to 1 as the
                                   turns over the original context, n_i = original_ctx f_i /
                                   (2 pi), go from low to high: w = clamp((n_i - low) /
                                   (high - low), 0, 1) */

typedef struct hss_rope {
    int32_t rot_dim; /* even, 2 .. 256 */
    int32_t scaling; /* HSS_ROPE_SCALE_* */
    double base;     /* > 0 */
    double factor;   /* > 0 (SCALE_NONE ignores it) */
    double original_ctx, low, high; /* SCALE_RAMP only: original_ctx > 0, low < high */
} hss_rope;

/* The table turns[rot_dim / 2] of a rope, computed on the host in double (a host array; the
 * caller copies it to the device once).  HSS_ERR_INVALID_ARGUMENT for values outside the ranges
 * above or not finite, a stretched base or a high - low past the range of a double included. */
hss_status hss_rope_table(const hss_rope* rope, uint64_t* turns);

/* What the layers of one step share in hss_rope_tokens. */
typedef struct hss_rope_args {
    hss_dims dims;
    int32_t rot_dim;          /* even, 2 .. head_dim: elements past it are copied */
    int32_t layout;           /* HSS_ROPE_HALF or HSS_ROPE_INTERLEAVED */
    const uint64_t* turns;    /* device, [rot_dim / 2], 8-byte aligned */
    float magnitude;          /* factor on the rotated elements (1: none) */
    const int64_t* positions; /* device, [num_tokens], any sign */
    const int64_t* slots;     /* device, [num_tokens], as in hss_write_kv_tokens; needed with a
                                 cache, else may be NULL */
    int64_t num_tokens;
    int64_t q_stride, k_stride, v_stride; /* elements from token to token of Q, K and V:
                                             multiples of 8, at least heads * head_dim (the rows of
                                             a fused projection have them all alike) */
    int32_t* dev_status;      /* device int32 or NULL */
} hss_rope_args;

/*
 * Rotate the queries and keys of new tokens and write keys and values into the paged cache, in
 * one launch:
 *   Q_out[i][h]                 = R(positions[i]) Q[i][h]     (every query head)
 *   K_out[i][h]                 = R(positions[i]) K[i][h]     (K_out != NULL; every kv head)
 *   K_cache[slot / bs][slot % bs][h] = the same key           (K_cache != NULL; slot = slots[i])
 *   V_cache[slot / bs][slot % bs][h] = V[i][h]                (V_cache != NULL)
 * with y_a = m (x_a cos - x_b sin), y_b = m (x_b cos + x_a sin) for a pair (a, b), computed in
 * fp32 and rounded once to bf16.
 *   Q, K, V   device, token i's heads at i * stride, dense [heads, head_dim] bf16; 16-byte
 *             aligned.  Each may be NULL if none of its outputs is asked for, and an output
 *             needs its input.
 *   Q_out     device, [num_tokens, num_q_heads, head_dim] bf16, 16-byte aligned, or NULL
 *   K_out     device, [num_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned, or NULL (the
 *             rows hss_write_kv_tokens projects into A_g)
 *   K_cache, V_cache  device, [max_blocks, block_size, num_kv_heads, head_dim] bf16, 16-byte
 *             aligned: this layer's caches, or NULL
 * A negative slot marks padding (the cache is left alone, Q_out and K_out are still written); a
 * slot >= max_blocks * block_size is skipped and raises HSS_ERR_OUT_OF_RANGE in *dev_status and
 * the library's device error word.  If two tokens name one slot, each 16 bytes of its rows are one
 * token's or the other's: name it once.  No output may overlap an input.
 */
hss_status hss_rope_tokens(const hss_rope_args* args, const uint16_t* Q, const uint16_t* K,
                           const uint16_t* V, uint16_t* Q_out, uint16_t* K_out,
                           uint16_t* K_cache, uint16_t* V_cache, void* stream);

/* What the layers of one step share in hss_attend_tree. */
typedef struct hss_attend_args {
    hss_dims dims;
    const int32_t* q_offsets;   /* device, [num_seqs + 1]: sequence s owns the rows
                                   q_offsets[s] .. q_offsets[s + 1] - 1, its tree's nodes */
    int64_t total_q;            /* rows in all, q_offsets[num_seqs] */
    int32_t max_q;              /* at least the largest tree's nodes; the workspace goes by it */
    int32_t mask_words;         /* 64-bit words of a row's mask (tree_mask != NULL: >= 1) */
    const uint64_t* tree_mask;  /* device, [total_q, mask_words], 8-byte aligned, or NULL */
    const int32_t* block_table; /* device, [total_blocks] physical block ids */
    const int32_t* seq_offsets; /* device, [num_seqs + 1], as in hss_score_blocks */
    const int32_t* ctx_len;     /* device, [num_seqs]: cached tokens before the tree */
    int64_t total_blocks;
    int32_t num_seqs;
    float scale;                /* factor on the scores, finite; usually head_dim^-0.5 */
    float decay;                /* factor on weights_in, finite */
    void* workspace;            /* device, 256-byte aligned, hss_attend_tree_workspace_bytes(...);
                                   what it holds does not matter.  Calls that share one must not
                                   run at the same time. */
    size_t workspace_bytes;
    int32_t* dev_status;        /* device int32 or NULL */
} hss_attend_args;

/* Bytes of the workspace: enough for every call with these dims and counts, or smaller ones (0 if a
 * count is negative, the dims are not valid, or the call would be refused as too large: 2^30 tiles
 * of tokens under a row tile, or pieces of a row tile, at most).
 * Without weights it holds what the CTAs have of the rows in fp32, with room for max_q rows of every
 * sequence: max_q as whole row tiles of 128 / (num_q_heads / num_kv_heads) nodes, two by two where
 * there are more than one and head_dim is below 256; twice that where max_q is at most one row tile
 * or head_dim is 256; up to a third more for an odd few row tiles; and at most 42 MB besides.  With
 * weights also five bytes for every 16 tokens that such a row may see, per query head.  64 single
 * tokens over 16k tokens each (32 heads of 128), with weights: 13 MB; 512 rows of 64 heads of 128
 * over 128k tokens: 39 MB, with weights 1.6 GB.
 * It goes by max_q and not by the rows there are: a chunk of 2048 rows among 63 single tokens, all
 * over 4k tokens (64 heads of 128), takes 4.8 GB, with weights 17.4 GB, where a call of the chunk
 * alone takes 95 MB (382 MB) and one of the single tokens 5.5 MB (11 MB).  Call such sequences
 * apart. */
size_t hss_attend_tree_workspace_bytes(const hss_dims* dims, int32_t num_seqs, int32_t max_q,
                                       int64_t total_blocks, int32_t with_weights);

/*
 * Attention of a tree of drafted tokens over the paged cache, and of the single new token of an
 * ordinary decode step (a tree of one node) or a chunk of prompt tokens (a chain).  Sequence s
 * has ctx_len[s] cached tokens, which all its rows see, and then its tree's nodes: node j's key
 * and value are in the cache at position ctx_len[s] + j (write them first, e.g. with
 * hss_rope_tokens).  Row i sees node j if bit j % 64 of tree_mask[row][j / 64] is set (nodes past
 * the mask's words are not seen), or, with tree_mask NULL, if j <= i (a chain).  Position p is
 * token p % block_size of the sequence's table entry p / block_size.  Query head h reads kv
 * head h / (num_q_heads / num_kv_heads).  Over the tokens that a row sees:
 *   lse[row][h] = ln sum_p exp(scale q.k_p)
 *   out[row][h] = sum_p exp(scale q.k_p - lse) v_p
 *   weights_out[e] = decay * weights_in[e] + sum over the sequence's rows, all query heads and
 *                    the tokens p of table entry e of exp(scale q.k_p - lse)
 * A row that sees nothing gets out 0 and lse -inf and adds no weight.  Keys and values that no
 * row of the tree sees, or that lie past the sequence's last token, may hold anything (NaN and
 * infinities included); a node's NaN or infinite value reaches only the rows that see it.
 *   Q        device, [total_q, num_q_heads, head_dim] bf16, 16-byte aligned
 *   K_cache, V_cache  as in hss_rope_tokens
 *   out      device, [total_q, num_q_heads, head_dim] bf16, 16-byte aligned
 *   lse      device, [total_q, num_q_heads] f32, or NULL
 *   weights_in   device, [total_blocks] f32, or NULL (zeros)
 *   weights_out  device, [total_blocks] f32, or NULL (weights_in is then not read); it may be
 *                weights_in
 * Scores, softmax statistics and sums are fp32; the weights exp(s - m) enter the product with V
 * rounded to bf16, the statistics and block weights take them unrounded.  That rounding moves an
 * element of out by at most 2^-9 sum_p exp(s - lse) |v_p|, beside the 2^-9 |out| of its own rounding
 * to bf16; of the outputs' norm the two come to 0.0023 together, where the second alone is 0.0017.
 * Up to three more launches follow the attention itself on the stream (the join of what several
 * CTAs have of a row, and the block weights); a pipeline wait that runs out raises
 * HSS_ERR_DEVICE_TIMEOUT like those of the other kernels.
 * Supported: num_q_heads / num_kv_heads <= 128; num_seqs, max_q >= 0; HSS_ERR_INVALID_ARGUMENT if
 * the counts are too large for hss_attend_tree_workspace_bytes.  Other device-side errors
 * (*dev_status and the library's device error word): a block id outside [0, max_blocks) hides
 * its tokens and raises HSS_ERR_OUT_OF_RANGE; so does a table too short for ctx_len + nodes (the
 * tokens past it are hidden); a negative ctx_len counts as 0; a sequence with more than max_q
 * rows raises HSS_ERR_INVALID_ARGUMENT and its rows past max_q are not written.
 */
hss_status hss_attend_tree(const hss_attend_args* args, const uint16_t* Q,
                           const uint16_t* K_cache, const uint16_t* V_cache, uint16_t* out,
                           float* lse, const float* weights_in, float* weights_out,
                           void* stream);

/*
 * Eviction from the cache by accumulated attention weight: cut every sequence's table to its
 * budget.  Sequence s (n entries) may lose its entries j with
 *   keep_first <= j < n - keep_last
 * and, with ctx_len, whole ones only, j < ctx_len[s] / block_size;
 * of these it loses the max(n - budgets[s], 0) (or all, if there are fewer) with the least
 * (weight, index): -0 equals +0 and NaN ranks as +inf, as in hss_rank_victims.  The entries that
 * stay keep their order:
 *   new_offsets[num_seqs + 1]  the offsets of the shorter tables
 *   new_table, new_weights     [total_blocks] the entries that stay, packed; the rest of the
 *                              arrays is -1 and 0
 *   new_ctx_len[s] = ctx_len[s] - block_size * entries lost   (ctx_len and new_ctx_len both
 *                              given, or both NULL)
 *   freed [total_blocks]       the physical ids that were lost, by sequence and index, packed;
 *                              the rest is -1.  Sequence s's are at freed_offsets[s] ..
 *                              freed_offsets[s + 1] - 1.
 * All arrays are on the device: weights and new_weights f32, the others int32.  No output may
 * overlap an input.  Budgets below 0 count as 0.  block_size > 0, keep_first, keep_last >= 0,
 * total_blocks <= 2^30.
 * The result is exact.
 */
hss_status hss_evict_blocks(const float* weights, const int32_t* block_table,
                            const int32_t* seq_offsets, const int32_t* ctx_len,
                            const int32_t* budgets, int32_t num_seqs, int64_t total_blocks,
                            int32_t block_size, int32_t keep_first, int32_t keep_last,
                            int32_t* new_table, int32_t* new_offsets, float* new_weights,
                            int32_t* new_ctx_len, int32_t* freed, int32_t* freed_offsets,
                            void* stream);

/* What the layers of one step share in hss_norm_rope_tokens. */
typedef struct hss_norm_rope_args {
    hss_rope_args rope;      /* as in hss_rope_tokens */
    int64_t q_weight_stride; /* elements from head to head of the weights: 0 (the heads share one */
    int64_t k_weight_stride; /* row), or a multiple of 8, at least head_dim */
    float eps;               /* >= 0, finite */
    float weight_offset;     /* added to every weight, finite (1 where weights are kept around 0) */
} hss_norm_rope_args;

/*
 * hss_rope_tokens with a root-mean-square norm of every query and key head before the rotation,
 * in the same launch:
 *   y[i] = x[i] / sqrt(mean_j x[j]^2 + eps) * (weight[i] + weight_offset),
 * over the whole head (head_dim elements, the ones past rot_dim too), then rotated and written as
 * there.  Values are not normed.  Norm and rotation are computed in fp32 (weight + weight_offset is off
 * by 2^-24 of the offset at most, and not at all if that is a power of two) and rounded once to bf16;
 * the sum of squares is fp32 too, so that a head whose sum passes 3.4e38 comes out as 0 (small heads
 * lose nothing, with eps 0 either, where a head of zeros alone is NaN, 0 / 0).
 *   q_weight, k_weight  device, [head_dim] or, with a stride, [heads, head_dim] bf16, 16-byte
 *             aligned; NULL: 1 (weight_offset is then not added)
 * The other arguments, the refusals and the device-side errors are those of hss_rope_tokens.
 */
hss_status hss_norm_rope_tokens(const hss_norm_rope_args* args, const uint16_t* Q,
                                const uint16_t* K, const uint16_t* V, const uint16_t* q_weight,
                                const uint16_t* k_weight, uint16_t* Q_out, uint16_t* K_out,
                                uint16_t* K_cache, uint16_t* V_cache, void* stream);

/*
 * A paged cache in 4 bits.  Every 32 consecutive elements of a head share a bf16 scale; an element
 * is a code from -7 to 7 times its group's scale, 4.5 bits an element in all.  A page holds keys
 * and values, in tiles of 16 tokens of one head:
 *     cache[max_blocks][num_kv_heads][block_size / 16][tile]
 * with head_dim = 32 G and a tile of 18 head_dim bytes,
 *     [ codes of K: 8 head_dim bytes | codes of V: 8 head_dim bytes |
 *       scales of K: bf16 [16][G] | scales of V: bf16 [16][G] ],
 * a code being kept as code + 8 in a nibble (the low nibble of a byte first).  Of token t (0 .. 15)
 * and element d the nibble lies
 *   K: in byte t head_dim / 2 + (d % 32 / 8) 4 G + d / 32 * 4 + d % 8 / 2, the low one if d is even
 *   V: in byte ((d / 64) 32 + (d % 8) 4 + t % 8 / 2) 16 + d % 64 / 16 * 4 + t % 2 * 2 + t / 8,
 *      the low one if d % 16 < 8
 * so that a thread of the attention finds its operands of the matrix products side by side, and no
 * byte holds two tokens.  (A nibble of 0 counts as -8; packing writes none.)
 */
/* Bytes of one page: num_kv_heads * block_size / 16 * 18 * head_dim (0 if the dims are invalid). */
size_t hss_packed_page_bytes(const hss_dims* dims);

/* What the layers of one step share in hss_pack_kv_tokens and hss_unpack_kv_tokens. */
typedef struct hss_pack_args {
    hss_dims dims;
    const int64_t* slots;      /* device, [num_tokens], as in hss_write_kv_tokens */
    int64_t num_tokens;
    int64_t k_stride, v_stride; /* elements from token to token of K and V: multiples of 8, at least
                                   num_kv_heads * head_dim */
    int32_t* dev_status;       /* device int32 or NULL */
} hss_pack_args;

/*
 * Write tokens into the packed cache.  Per token, kv head and group of 32 elements x, all in fp32:
 *   scale = bf16(max |x| / 7),  code = max(-7, min(7, rint(x / scale)))    (ties to even)
 * A group whose scale is 0 has codes 0; one with a NaN or an infinity gets the scale NaN, and reads
 * as NaN.  The result is exact: the same bits wherever and with whatever else a token is packed.
 *   K, V      device, token i's heads at i * stride, dense [heads, head_dim] bf16, 16-byte aligned;
 *             either may be NULL (that half of the tokens is then left as it was)
 *   cache     device, one layer's pages, 16-byte aligned
 * A negative slot marks padding; a slot >= max_blocks * block_size is skipped and raises
 * HSS_ERR_OUT_OF_RANGE in *dev_status and the library's device error word.  Name a slot once: what
 * two tokens of one call leave in it is a mixture of both.  (From 4096 tokens of 1024 elements on, K
 * and V together, 16 tokens in a row that fill a tile are packed together: give tokens in the order of
 * their slots.)  No output overlaps an input.
 */
hss_status hss_pack_kv_tokens(const hss_pack_args* args, const uint16_t* K, const uint16_t* V,
                              uint8_t* cache, void* stream);

/*
 * Read tokens back from the packed cache: code * scale, rounded once to bf16 (the keys of a packed
 * cache for hss_project_kv_blocks, or a cache to be packed anew).  K and V are outputs here, laid
 * out as above, and either may be NULL.  Rows of tokens with a negative slot, or one that is out of
 * range (which raises the error), are left as they were.
 */
hss_status hss_unpack_kv_tokens(const hss_pack_args* args, const uint8_t* cache, uint16_t* K,
                                uint16_t* V, void* stream);

/* What the layers of one step share in hss_attend_packed. */
typedef struct hss_packed_args {
    hss_dims dims;
    const int32_t* q_offsets;   /* device, [num_seqs + 1], as in hss_attend_tree */
    int64_t total_q;            /* rows in all, q_offsets[num_seqs] */
    int32_t max_q;              /* at least the most rows of a sequence */
    int32_t window;             /* tokens that a row sees back from its own, >= 1; or 0: all */
    int32_t sinks;              /* first tokens that stay visible behind the window, >= 0 */
    const int32_t* block_table; /* device, [total_blocks] physical block ids */
    const int32_t* seq_offsets; /* device, [num_seqs + 1], as in hss_score_blocks */
    const int32_t* ctx_len;     /* device, [num_seqs]: cached tokens before the rows */
    int64_t total_blocks;
    int32_t num_seqs;
    float scale;                /* factor on the scores, -2^100 .. 2^100; usually head_dim^-0.5 */
    void* workspace;            /* device, 256-byte aligned,
                                   hss_attend_packed_workspace_bytes(...); what it holds does not
                                   matter.  Calls that share one must not run at the same time. */
    size_t workspace_bytes;
    int32_t* dev_status;        /* device int32 or NULL */
} hss_packed_args;

/* Bytes of the workspace: enough for every call with these dims, window and sinks and these counts
 * or smaller ones (0 if a count is negative or the dims are not valid).  It goes by head_dim and by
 * whether there are more than 32 rows of a sequence and kv head together: 5 or 45 MB for head_dim
 * 128, 10 or 50 for 256. */
size_t hss_attend_packed_workspace_bytes(const hss_dims* dims, int32_t num_seqs, int32_t max_q,
                                         int64_t total_blocks, int32_t window, int32_t sinks);

/*
 * Attention over the packed cache: of the new token of a decode step, of a few drafted tokens in a
 * row, or of a chunk of prompt tokens, with an optional sliding window behind which the first
 * tokens stay visible.  Sequence s has ctx_len[s] cached tokens and then its rows' own tokens: row
 * i's is at position ctx_len[s] + i (write them first, with hss_pack_kv_tokens).  It sees the
 * positions
 *   p <= ctx_len[s] + i,  and with a window only those with
 *   p > ctx_len[s] + i - window  or  p < sinks.
 * Position p is token p % block_size of the sequence's table entry p / block_size.  Pages that no
 * row sees are not read, and their entries may hold anything (an evicted page's id).  Query head
 * h reads kv head h / (num_q_heads / num_kv_heads).  Over the tokens that a row sees:
 *   lse[row][h] = ln sum_p exp(scale q.k_p)
 *   out[row][h] = sum_p exp(scale q.k_p - lse) v_p
 * A row that sees nothing (its sequence's table does not reach that far) gets out 0 and lse -inf.
 * Tokens that a row does not see may hold anything, scales of NaN included.
 *   Q        device, [total_q, num_q_heads, head_dim] bf16, 16-byte aligned
 *   cache    device, one layer's pages, 16-byte aligned
 *   out      device, [total_q, num_q_heads, head_dim] bf16, 16-byte aligned
 *   lse      device, [total_q, num_q_heads] f32, or NULL
 * No output overlaps an input.
 * Scores, softmax statistics and sums are fp32: sums over 32 elements of q times codes, scores, and sums
 * over tokens of weights (1 at most) times values have to stay below 3.4e38 (a row with a score above
 * it is NaN).  The statistics take the weights exp(s - m) unrounded; a weight below 2^-118 of the
 * row's largest counts as 0.  Up to 32 rows of a sequence and kv head together (rows times
 * num_q_heads / num_kv_heads, by max_q): a weight times its value's scale enters the product with the
 * codes rounded to bf16; an element of out is off by at most 2^-8 sum_p exp(s - lse) |v_p| for it,
 * beside the rounding of out itself.  More rows run on the tensor cores of tcgen05 with K, V and the weights
 * in fp16: K and V lose nothing, a weight 2^-11 of itself or 2^-32 of the row's largest.  There a scale
 * that fp16 has no place for (above 64, or below 2^-17 but not 0, or not finite; also a query times the
 * factor past 2^108) makes the whole call run by the first method after all, 16 rows at a time: of any
 * sequence's rows, for one group that any of them sees.  That takes three to seven times as long (512
 * rows over 32768 tokens 3.6 ms, not 0.51; 16 chunks of 64 rows over 2000 0.33, not 0.11).
 * A call is one to three launches on the stream: for few rows the attention and, unless contexts are
 * short, the join of what several CTAs have of a row; for many rows the attention, that second
 * attempt, which ends at once if it is not needed, and at most one join for both.  A pipeline wait
 * that runs out raises HSS_ERR_DEVICE_TIMEOUT like those of the other kernels.
 * Single tokens in one call with a chunk of many rows cost as much as row tiles of 128: call them
 * apart.
 * Supported: num_q_heads / num_kv_heads <= 128, at most 2^30 rows of a sequence and kv head
 * together; window, sinks >= 0; positions below 2^31 - 512.  Device-side errors
 * (*dev_status and the library's device error word): a block id outside [0, max_blocks) of a page
 * that a row sees hides its tokens and raises HSS_ERR_OUT_OF_RANGE; so does a table too short for
 * ctx_len + rows (the tokens past it are hidden); a negative ctx_len counts as 0; a sequence with
 * more than max_q rows raises HSS_ERR_INVALID_ARGUMENT and its rows past max_q are not written.
 */
hss_status hss_attend_packed(const hss_packed_args* args, const uint16_t* Q, const uint8_t* cache,
                             uint16_t* out, float* lse, void* stream);

/*
 * Pages that sequences share.  refs[p] counts who holds page p: the table entries that name it, and
 * whoever else the caller counts (a cache of prompt prefixes); 0: the page is free.  The two plans
 * below take the tables and counts as they are and write new ones, so that a call can be repeated;
 * the page copies they ask for are then made by hss_copy_pages, once per cache.
 */

/* Bytes of the workspace of hss_fork_pages and hss_compact_pages (0 if a count is negative). */
size_t hss_fork_pages_workspace_bytes(int32_t num_new, int64_t max_blocks);
size_t hss_compact_pages_workspace_bytes(int64_t max_blocks);

/*
 * The tables of the next step: num_new sequences, each the continuation of one of the present ones.
 * New sequence i keeps the first len_i = min(lengths[i], what its parent's table has room for)
 * tokens of sequence parents[i] (-1: none, len_i = 0) and gets room for room[i] more: its table has
 * ceil((len_i + room[i]) / block_size) entries, of which the first kept_i = ceil(len_i /
 * block_size) are the parent's.  So a sequence can go on (once), be forked (more than once), be cut
 * back (a smaller length), grow, and be dropped (not at all; its pages lose a reference).
 *   A last kept page that is partly filled will be written, if room[i] > 0.  It stays the new
 * sequence's own if all its other references are such sequences too and i is the least of them;
 * otherwise the new sequence gets a fresh page there, and the pair (old page, fresh page) is one of
 * the copies.  The other entries past the kept ones are fresh pages as well.  Fresh pages are those
 * whose count is then 0, handed out by ascending id in the order of (sequence, entry).
 *   block_table, seq_offsets, num_seqs, total_blocks  the present tables, as in hss_score_blocks
 *   refs       [max_blocks] in;  new_refs [max_blocks] out
 *   released   [num_released] page ids that lose one reference besides (what hss_evict_blocks has
 *              freed: entries of -1 are skipped), or NULL with num_released = 0
 *   parents, lengths, room   [num_new]; negative lengths and room count as 0
 *   new_table  [table_room], the tables packed, the rest -1;  new_offsets [num_new + 1]
 *   copy_src, copy_dst  [num_new], the copies by sequence, packed, the rest -1
 *   counts     [4]: entries of the new tables, copies, pages in use, fresh pages that were missing
 * All arrays are on the device and int32, 4-byte aligned; no output overlaps an input.  The result
 * is exact and the same on every run.  Device-side errors, in *dev_status and the library's device
 * error word: a parent outside [-1, num_seqs) counts as -1 and raises HSS_ERR_OUT_OF_RANGE; so does
 * an id outside [0, max_blocks) in a present table or (but for -1) in released, which is counted
 * nowhere and kept as it is.  If there are not enough free pages, the last entries are -1 (a copy
 * to such an entry has copy_dst -1) and HSS_ERR_OUT_OF_RANGE is raised; if the new tables need more
 * than table_room entries, HSS_ERR_INVALID_ARGUMENT is, nothing but counts[0] and new_offsets is
 * then of use, and every copy_dst is -1.  HSS_ERR_INVALID_ARGUMENT is raised as well if a page has a
 * smaller count than the present tables and released give up of it; the page may then be handed out
 * although it is held.
 * num_seqs, num_new <= 2^20, total_blocks, table_room, num_released, max_blocks <= 2^30.
 */
hss_status hss_fork_pages(const int32_t* block_table, const int32_t* seq_offsets,
                          int32_t num_seqs, int64_t total_blocks, const int32_t* refs,
                          int64_t max_blocks, const int32_t* released, int64_t num_released,
                          const int32_t* parents, const int32_t* lengths, const int32_t* room,
                          int32_t num_new, int32_t block_size, int64_t table_room,
                          int32_t* new_table, int32_t* new_offsets, int32_t* new_refs,
                          int32_t* copy_src, int32_t* copy_dst, int32_t* counts, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * Move pages to the front of the pool, so that its end can be given up.  With `used` pages that are
 * not free, the free pages below `used` are filled in ascending order by the used pages from
 * `used` on in descending order, at most move_room of them (the rest of the work is left for
 * another call):
 *   new_table  [total_blocks] the table with the moved ids replaced
 *   new_refs   [max_blocks] the counts moved along
 *   copy_src, copy_dst  [move_room] the moves, in that order, the rest -1
 *   counts     [4]: moves, pages in use, the last used page + 1 after the moves, moves left over
 * Whoever holds ids besides the table (refs counts them) has to follow the moves too.  Arrays,
 * limits are as in hss_fork_pages; an id outside [0, max_blocks) other than -1 is kept and raises
 * HSS_ERR_OUT_OF_RANGE, a negative count raises HSS_ERR_INVALID_ARGUMENT (its page counts as used);
 * move_room <= 2^30.
 */
hss_status hss_compact_pages(const int32_t* block_table, int64_t total_blocks, const int32_t* refs,
                             int64_t max_blocks, int64_t move_room, int32_t* new_table,
                             int32_t* new_refs, int32_t* copy_src, int32_t* copy_dst,
                             int32_t* counts, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream);

/*
 * Copy pages within one or two pools, in every layer of them:
 *   pool[layer][copy_dst[i]] = pool[layer][copy_src[i]]    i < *num_copies, layer < num_layers
 *   copy_src, copy_dst  device, [max_copies] int32; a pair with a negative id is skipped, one with
 *              an id >= max_blocks too, which raises HSS_ERR_OUT_OF_RANGE.  The destinations are
 *              distinct and none of them is a source.
 *   num_copies device int32, or NULL for max_copies (values outside [0, max_copies] are clipped)
 *   pool0, pool1  device, [num_layers][max_blocks][page_bytes], 16-byte aligned (the K and the V
 *              cache); pool1 may be NULL
 *   page_bytes a multiple of 16, 16 .. 2^30
 * max_copies, max_blocks <= 2^30; num_layers <= 65535.
 */
hss_status hss_copy_pages(const int32_t* copy_src, const int32_t* copy_dst,
                          const int32_t* num_copies, int64_t max_copies, void* pool0, void* pool1,
                          int64_t page_bytes, int64_t max_blocks, int32_t num_layers,
                          int32_t* dev_status, void* stream);

/*
 * Failure-detection self-test.  Every pipeline wait in the tensor-core kernels gives up
 * after a time limit and reports HSS_ERR_DEVICE_TIMEOUT instead of hanging the GPU.  This
 * call launches one small kernel whose thread waits, with that same bounded wait, on a
 * barrier nothing arrives on, for limit_ns (1e3 .. 2e9) nanoseconds; the kernel then stores
 * HSS_ERR_DEVICE_TIMEOUT into *dev_status (device int32, which the caller zeroes first) and
 * into the library's error word, and exits.  The context stays usable.
 */
hss_status hss_self_test_wait_timeout(int32_t* dev_status, int64_t limit_ns, void* stream);

/*
 * Failure-detection self-test of hss_layer_step's one-sequence victim ranking.  In that
 * ranking every CTA of the scorer waits until all of the sequence's keys are published, with
 * a bounded wait.  This call runs the decode layer call's scorer on one sequence (one query
 * row, queries projected in the scorer, no new blocks; the arguments as in hss_layer_step)
 * with its last CTA withholding its keys, so that every CTA's wait runs out after limit_ns
 * (1e3 .. 2e9) nanoseconds: HSS_ERR_DEVICE_TIMEOUT is stored into *dev_status and the
 * library's error word, the kernel exits, the context stays usable.  The scores are
 * written; the victims are not meaningful.  Zero the workspace again before the next
 * hss_layer_step on it.  HSS_ERR_UNSUPPORTED_SHAPE (nothing launched) when the shape does not
 * take that ranking (more than 4096 entries, or a grid that does not fit the GPU at once).
 * No page has a counterpart: it tests this library's own wait.
 */
hss_status hss_self_test_spread_wait(const hss_dims* dims, const uint16_t* P, const uint16_t* Q,
                                     uint16_t* A_g, int32_t layer, const int32_t* block_table,
                                     const int32_t* seq_offsets, int64_t total_blocks,
                                     float* scores, int32_t k, int32_t* victims, void* workspace,
                                     size_t workspace_bytes, int64_t limit_ns,
                                     int32_t* dev_status, void* stream);

/*
 * Device-side error word of the current device: the first HSS_ERR_* code a
 * kernel raised since the last read (HSS_ERR_DEVICE_TIMEOUT when a pipeline
 * wait ran out), or HSS_OK.  Synchronises `stream`, copies the word to
 * *status and clears it.
 */
hss_status hss_read_device_error(int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSS_H */
