// attend.cu -- attention of a tree of drafted tokens over the paged cache, on tcgen05.
//
// For one sequence and kv head, the rows are (node, query head of the group) pairs, and
//   S = Q K^T,  P = exp2(c S - m),  O = P V,  l = sum P
// runs over the sequence's tokens in tiles, one pass, with the softmax's running maximum m.  S
// and O are tcgen05 products (M = 128 rows, a row per TMEM lane, so that one thread owns a row's
// maximum and sum and no shuffle is needed); P goes back to tensor memory in bf16 and is the A
// operand of the second product; K is its own K-major operand, V an MN-major one, both as TMA
// leaves them.
//
// Roles of a CTA (12 warps, one CTA per SM):
//   warps 0, 1   TMA: look up the block ids, one box per 16 or more tokens (K and V of one group's
//                tiles each, or one K and one V); warp 0 also brings the queries
//   warps 2, 3   issue the products of one softmax group each, as whole converged warps: with a
//                lone thread's divergent branch every instruction first moved its operands to
//                uniform registers, 60 to 80 cycles each, and a 512-row chunk took 1.8 ms, not 1.4
//   warps 4..11  two softmax groups of four warps.  With at most 128 rows the groups take a
//                sequence's even and odd tiles, each with its own O, m and l (joined later, like
//                any two pieces of a split sequence); with more rows they take two row tiles over
//                the same K and V.  Either way one group's exponentials run under the other
//                group's products.
//
// Split.  All (sequence, batch of row tiles, kv head, tile) units form one list, cut into equal
// contiguous ranges: every SM gets the same work whatever the lengths are.  A range's
// pieces of (sequence, batch, head) leave unnormalised O, m and l in the workspace, and a second
// kernel joins them.  What one group saw from the first tile to the last needs no join: its rows
// go out from here (a prompt of 4096 tokens 574 us, through the workspace 603; 50 trees of 248
// nodes, head_dim 256, 453 against 595).  Row tiles beyond one (large trees, chunks) go to
// neighbouring CTAs that walk the same range in step, so that K and V come from HBM once and from
// L2 to the rest.
//
// Block weights: the softmax thread has the sum of every 16 of its tokens anyway (l is their
// sum); with weights it stores them beside m, and once the rows' lse are known they are scaled by
// exp2(m - lse) and added up over rows and heads.  No score is formed twice, and there are no
// float atomics: the same call gives the same bits.
//
// What bounds it, and what it reaches on GB300 (HBM 6.79 TB/s and 1906 TFLOP/s bf16 measured):
// few rows, the bytes of K and V: 64 sequences of 1k to 16k tokens, 32 query heads on 8 of 128, 380
// us with weights and join, 6.0 TB/s; one sequence of 32k tokens 38 us, of which 20 are its bytes
// and the rest the start (sequence lengths, block ids and the first tiles, one way through memory
// after another, 7 us), the last tiles and the join (8 us).  Many rows, the products and the
// exponentials between them, both near 1400 cycles for a job of 2 x 128 rows by 64 tokens: 512
// rows of 64 heads over 131072 tokens 1.36 ms in the first calls after a pause (1.6 PFLOP/s), 1.47
// to 1.49 ms under the power cap of a long run.  Many short items, what each costs besides its tiles (4 to 5 us): a prompt of 4096
// tokens, 64 heads, 282 us (1 PFLOP/s of what its rows see); 43 chains of 202 nodes over nothing
// 132 us, of which 42 are the bytes of queries and results.
//
// Masked places.  Tokens that all rows see need no mask; a tile that holds others, the end of the
// sequence or a bad block id gets 32 visibility bits per 32 tokens and row.  A zero weight does
// not silence an infinite or NaN value in a matrix product, so before such a tile's second
// product the group clears the values past the end and any non-finite element of a node's
// value, and whoever writes the rows adds those elements to those that do see the node.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "ptx.cuh"

namespace hss {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;          // UMMA M
constexpr int kMetaRing = 16;       // bad-id bits of the tiles in flight
// Flags of pieces with a non-finite value.  A flag is set by any of the group's warps (with two row
// tiles, by the other group's too) and read at the piece's end, with no barrier of its own, so a
// slot must not be set again before every warp has read it.  Pieces count where the group has jobs.
// A warp that is at piece n has seen its scores, which were issued after all products of the
// group's piece n - 1, and those wait for weights from all four warps of the group: they have
// left piece n - 2.  The other group can be one piece further behind: its queries for piece n were
// loaded once its last scores of n - 1 were done, two of which need no weights of n - 1, but all
// products of n - 2: its warps have left piece n - 3.  Three slots would do; four count by a mask
// (with three, 512 rows over 16384 tokens 211 us, so 209).
constexpr int kFlagSlots = 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kCtas = 152;          // GB300's SMs; the workspace does not depend on the device
constexpr float kLazy = 8.0f;       // the maximum may lag by 2^8 before O is rescaled

// A tile of K or V is what one ring stage holds; a job is the 64 tokens that a softmax group
// takes at a time.  TMEM: the score buffers of every group, then every group's O, 512 columns.
// Two score buffers let a group start on its next scores while the product with its last weights
// and the scores after that are on their way; for head_dim 192 there is room for one.
template <int HD, int NQ>
struct Cfg {
    static constexpr int kTile = HD <= 128 ? 128 : 64;
    static constexpr int kJobs = kTile / 64;
    static constexpr int kGroups = HD == 256 ? 1 : 2;
    static constexpr int kBuffers = HD == 192 ? 1 : 2;
    // One softmax group walks all tiles of a row: where a CTA has a whole item, it writes the
    // result itself and the join has nothing to do for it.
    static constexpr bool kWhole = NQ == 2 || kGroups == 1;
    static constexpr int kOCols = kGroups * kBuffers * 64;  // where O begins
    static constexpr int kStageBytes = kTile * HD * 2;
    static constexpr int kQBytes = NQ * kRows * HD * 2;
    static constexpr int kBudget = 232448 - 1024 - 1024 - kQBytes;
    // Two rings.  Groups on tiles of their own: one ring each, K and V in turn.  Otherwise one
    // ring for K and one for V.  Whoever waits on a stage has then seen every earlier use of it
    // complete, which a wait for a phase's parity takes for granted.
    static constexpr bool kOwnTiles = NQ == 1 && kGroups == 2;
    static constexpr int kMost = kBudget / kStageBytes < 12 ? kBudget / kStageBytes : 12;
    static constexpr int kRing0 = kOwnTiles ? kMost / 2 : (kMost + 1) / 2;
    static constexpr int kRing1 = kMost / 2;
    static constexpr int kStages = kRing0 + kRing1;
    static constexpr int kSmemBytes = 2048 + kQBytes + kStages * kStageBytes;
    static_assert(kRing1 >= 2, "two operands in flight");
    static_assert(kOCols + kGroups * HD <= 512, "tensor memory");
    static_assert(kRing0 + 2 <= kMetaRing, "tiles in flight");
};

// Where a CTA's range of the list begins: tile t of (sequence s, batch b, head h).
struct Start {
    int s, b, h, t, item0, total, per;
};

struct AttendParams {
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
    int32_t box;         // tokens per TMA box: the largest power of two that divides bs
    int32_t nodes_tile;  // nodes per row tile, 128 / g
    int32_t members;     // CTAs per group: row tiles (or pairs of them) walked in step
    int32_t groups;
    int32_t rowcap;      // rows of a tile that can be in use
    int32_t ways;        // warps to a task of join_columns, or 0: part_o by row
    float c;             // |scale| log2(e), or 1 for scale 0
    float pre;           // 1, or -1 / 0 for a negative / zero scale: scores are multiplied first
    float decay;
    int32_t* dev_status;
    int32_t* lib_error;
    // workspace
    int32_t* header;     // [0] tiles in all, [1] tiles per group
    Start* starts;       // [groups] where each range begins
    int32_t* seq_tiles;  // [num_seqs] tiles before a sequence
    int32_t* seq_items;  // [num_seqs] (batch, head) items before a sequence
    float* part_o;       // [slot][row][head_dim], or [slot][head_dim][row] with ways
    float2* part_ml;     // [slot][row] (m, l)
    int32_t* part_bad;   // [slot] a node's value was not finite
    float* row_lse;      // [unit row tile][row], log2
    float* sums;         // [tile][member][q tile][16-token granule][row]
    float* sums_m;       // [tile][member][q tile][job][row]
};

struct SeqInfo {
    int q0, nodes, ctx, tokens, e0, end;
    bool cut;  // the table is too short for ctx_len + nodes
};

__device__ __forceinline__ SeqInfo load_seq(const AttendParams& p, int s) {
    SeqInfo x;
    x.q0 = __ldg(p.q_offsets + s);
    x.nodes = __ldg(p.q_offsets + s + 1) - x.q0;
    x.e0 = __ldg(p.seq_offsets + s);
    x.end = __ldg(p.seq_offsets + s + 1);
    x.ctx = max(__ldg(p.ctx_len + s), 0);
    x.nodes = min(max(x.nodes, 0), p.max_q);
    const int64_t room = static_cast<int64_t>(x.end - x.e0) * p.bs;
    const int64_t want = static_cast<int64_t>(x.ctx) + x.nodes;
    x.tokens = static_cast<int>(min(min(room, want), static_cast<int64_t>(0x7FFFFF00)));
    // What the table has no room for is hidden, so that a context past its end is no longer than
    // the tokens (and sums of its length and a node's number stay in 32 bits).
    x.cut = x.tokens < want;
    x.ctx = min(x.ctx, max(x.tokens, 0));
    return x;
}

// Row tiles of a sequence are `span` nodes each (NQ tiles of 128 rows); `members` of them form a
// batch.  A chain's rows see nothing past themselves, so its earlier batches have fewer tiles.
__device__ __forceinline__ int tokens_upto(const AttendParams& p, const SeqInfo& x, int nodes) {
    return max(p.mask == nullptr ? min(x.tokens - x.ctx, nodes) + x.ctx : x.tokens, 0);
}
template <int TILE>
__device__ __forceinline__ int tiles_upto(const AttendParams& p, const SeqInfo& x, int nodes) {
    return max(1, (tokens_upto(p, x, nodes) + TILE - 1) / TILE);
}
// In the list an item is longer than its tiles by what it costs besides (its last product, its
// rows' way out, the next queries), so that ranges of equal length take equal time: one tile of
// 128 tokens, three of 64.  (None, so, and twice that: a prompt of 4096 tokens 496, 448 and 455
// us; 4 of 1000 to 2000 210, 173 and 179; 50 trees of 248 nodes, head_dim 256, 385, 370 and 371.)
template <int TILE>
constexpr int kBeside = TILE == 128 ? 1 : 3;

template <int TILE>
__device__ __forceinline__ int batch_tiles(const AttendParams& p, const SeqInfo& x, int span,
                                           int b) {
    return tiles_upto<TILE>(p, x, min(x.nodes, (b + 1) * p.members * span)) + kBeside<TILE>;
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <int TILE>
__device__ __forceinline__ int seq_tiles(const AttendParams& p, const SeqInfo& x, int span,
                                         int nb) {
    if (p.mask != nullptr || nb == 1)
        return nb * p.nkv * (nb > 0 ? batch_tiles<TILE>(p, x, span, 0) : 0);
    int w = 0;
    for (int b = 0; b < nb; ++b) w += batch_tiles<TILE>(p, x, span, b);
    return w * p.nkv;
}

// One piece of this CTA's range: tiles [ta, ta + n) of (sequence, head) for row tile rt.
struct Segment {
    SeqInfo x;
    int h, rt, ta, n, item;
    int seen;   // tokens that some row of the row tile may see
    bool rows;  // the row tile exists
    int f;      // list index of tile ta
};

template <int TILE>
struct Walk {
    SeqInfo x;
    int s, b, h, t, nb, rts, item0, member, span, f, f1;

    __device__ __forceinline__ void enter(const AttendParams& p) {
        x = load_seq(p, s);
        rts = ceil_div(x.nodes, span);
        nb = ceil_div(rts, p.members);
    }
    __device__ __forceinline__ void begin(const AttendParams& p, const Start& st, int span_nodes) {
        const int group = blockIdx.x / p.members;
        member = blockIdx.x % p.members;
        span = span_nodes;
        f = min(st.total, group * st.per);
        f1 = min(st.total, f + st.per);
        s = st.s;
        b = st.b;
        h = st.h;
        t = st.t;
        item0 = st.item0;
        if (f < f1) enter(p);
    }
    __device__ __forceinline__ bool next(const AttendParams& p, Segment& g) {
        while (f < f1) {
            const int n = nb > 0 ? batch_tiles<TILE>(p, x, span, b) : 0;
            const int real = n - kBeside<TILE>;
            if (t < real) {
                const int take = min(real - t, f1 - f);
                g.x = x;
                g.h = h;
                g.rt = b * p.members + member;
                g.rows = g.rt < rts;
                g.ta = t;
                g.seen = g.rows ? tokens_upto(p, x, min(x.nodes, (g.rt + 1) * span)) : 0;
                const int mine = (g.seen + TILE - 1) / TILE;
                g.n = max(0, min(t + take, mine) - t);
                g.item = item0 + b * p.nkv + h;
                g.f = f;
                f += take;
                t += take;
                return true;
            }
            f += max(n - t, 0);
            t = 0;
            if (++h < p.nkv) continue;
            h = 0;
            if (++b < nb) continue;
            b = 0;
            item0 += nb * p.nkv;
            if (++s >= p.num_seqs) break;
            enter(p);
        }
        return false;
    }
    // Whether the segment that next() gave is all of its item.
    __device__ __forceinline__ bool whole(const AttendParams& p, const Segment& g) const {
        return g.ta == 0 && t == batch_tiles<TILE>(p, x, span, b) - kBeside<TILE>;
    }
};

// A group's jobs in a piece: two per tile, but for a last half tile that nobody sees.
template <class C>
__device__ __forceinline__ int jobs_of(const Segment& g, int group, int& tiles) {
    tiles = C::kOwnTiles ? (g.n - group + 1) / 2 : g.n;
    if (tiles == 0) return 0;
    const int last = g.ta + (C::kOwnTiles ? group + 2 * (tiles - 1) : tiles - 1);
    return tiles * C::kJobs - (C::kJobs == 2 && last * C::kTile + 64 >= g.seen ? 1 : 0);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A bounded wait whose waiting is cheap to leave: the clock and the abort flag are looked at only
// after a run of failed tries.
__device__ __forceinline__ bool wait_phase(uint64_t* b, uint32_t parity,
                                           const volatile int* abort_flag) {
    if (mbar_try_wait(b, parity)) return true;
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(b, parity)) return true;
        if (*abort_flag) return false;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) return false;
    }
}

// Where the K or V of a group's n-th tile (of all tiles, when the groups share them) goes.
template <class C>
__device__ __forceinline__ void place(bool values, int group, uint32_t n, int& stage,
                                      uint32_t& parity) {
    if constexpr (C::kOwnTiles) {
        const uint32_t use = 2 * n + (values ? 1 : 0), round = use / C::kRing0;
        stage = static_cast<int>(use - round * C::kRing0) + group * C::kRing0;
        parity = round & 1;
    } else if (!values) {
        const uint32_t round = n / C::kRing0;
        stage = static_cast<int>(n - round * C::kRing0);
        parity = round & 1;
    } else {
        const uint32_t round = n / C::kRing1;
        stage = static_cast<int>(n - round * C::kRing1) + C::kRing0;
        parity = round & 1;
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// 32 columns of this thread's TMEM lane and their maximum (usable after the wait).
__device__ __forceinline__ float tmem_ldred_values(uint32_t taddr, uint32_t* v) {
    float m;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "%32, [%33];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31]), "=f"(m)
        : "r"(taddr));
    return m;
}

// The wait for TMEM loads, with the uses of what they brought held behind it.
__device__ __forceinline__ void tmem_hold(uint32_t* v) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i])::"memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t* v) {
    tmem_ld_wait();
    tmem_hold(v);
}

// 64 visibility bits of a row for nodes 64 w ..
__device__ __forceinline__ uint64_t node_word(const AttendParams& p, const SeqInfo& x, int node,
                                              int w) {
    if (p.mask == nullptr) {
        const int past = node - 64 * w;  // nodes up to `node` are seen
        return past < 0 ? 0 : (past >= 63 ? ~0ull : (2ull << past) - 1);
    }
    if (w >= p.mask_words) return 0;
    return __ldg(p.mask + (static_cast<int64_t>(x.q0) + node) * p.mask_words + w);
}

// Visibility of the 32 tokens from position p0 on for a row, whose first two words are given.
__device__ __forceinline__ uint32_t visible32(const AttendParams& p, const SeqInfo& x, int node,
                                              int p0, uint64_t word0, uint64_t word1) {
    auto word = [&](int w) {
        return w == 0 ? word0 : (w == 1 ? word1 : node_word(p, x, node, w));
    };
    uint32_t bits;
    const int j0 = p0 - x.ctx;
    if (j0 <= -32) {
        bits = 0xFFFFFFFFu;
    } else if (j0 < 0) {
        bits = (static_cast<uint32_t>(word0) << -j0) | ((1u << -j0) - 1);
    } else {
        const int w = j0 >> 6, sh = j0 & 63;
        uint64_t v = word(w) >> sh;
        if (sh > 32 && 64 * (w + 1) < x.nodes) v |= word(w + 1) << (64 - sh);
        bits = static_cast<uint32_t>(v);
    }
    const int left = x.tokens - p0;
    return left >= 32 ? bits : (left <= 0 ? 0u : bits & ((1u << left) - 1));
}

struct Barriers {
    uint64_t full[12], empty[12];
    uint64_t q_full, q_empty, s_full[4], p_full[4], o_done[4], values;
    uint32_t bad_ids[2][kMetaRing];  // [ring] per tile in flight: 16-token granules with a bad id
    int bad_value[2][kFlagSlots];    // [group][piece mod kFlagSlots]: last piece with such a value
    int abort;
    uint32_t tmem;
    Start start;
    int scan[kThreads / 32];
    int scan_items[kThreads / 32];
};

// A whole item's row from tensor memory (anything, if it has no weight): row `to` of out, lse.
// Four lanes exchange their 64 bytes of a row, so that a store brings them side by side (by 16
// bytes of 32 rows it took 7400 cycles for 256 rows of 128).
template <int HD>
__device__ __forceinline__ void write_whole(const AttendParams& p, const SeqInfo& x, int node,
                                            int h, bool bad, uint32_t o_cols, bool live,
                                            int64_t to, float m, float l, float* row_lse) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int lane = threadIdx.x & 31;
    uint16_t* at[4];  // where the lane's 16 bytes of its neighbours' rows go
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = __shfl_sync(0xffffffffu, live ? to : -1, (lane & ~3) + r);
        at[r] = row < 0 ? nullptr : p.out + row * HD + 8 * (lane & 3);
    }
#pragma unroll 1
    for (int k = 0; k < HD; k += 32) {
        uint32_t o[32], u[4][4];
        __syncwarp();  // (the rows went out lane by lane, the last time)
        tmem_ld_32x32b_x32(o_cols + k, o);
        tmem_ld_wait_for(o);
        if (bad && live) {
            // Non-finite values of the nodes this row sees.
            for (int j = 0; j < x.nodes && x.ctx + j < x.tokens; ++j) {
                if (!((node_word(p, x, node, j >> 6) >> (j & 63)) & 1)) continue;
                const int pos = x.ctx + j;
                const int64_t id = p.table[x.e0 + pos / p.bs];
                if (id < 0 || id >= p.max_blocks) continue;
                const uint16_t* v = p.V + ((id * p.bs + pos % p.bs) * p.nkv + h) * HD + k;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float e = __uint_as_float(static_cast<uint32_t>(v[c]) << 16);
                    if (!isfinite(e)) o[c] = __float_as_uint(__uint_as_float(o[c]) + e);
                }
            }
        }
#pragma unroll
        for (int d = 0; d < 16; ++d)
            u[d / 4][d % 4] = l == 0.0f ? 0u
                                        : pack_bf16x2(__uint_as_float(o[2 * d]) * inv,
                                                      __uint_as_float(o[2 * d + 1]) * inv);
#pragma unroll
        for (int step = 1; step < 4; step *= 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i & step) continue;
                const bool up = (lane & step) != 0;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t give = up ? u[i][d] : u[i + step][d];
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, step);
                    if (up)
                        u[i][d] = got;
                    else
                        u[i + step][d] = got;
                }
            }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (at[r] != nullptr)
                *reinterpret_cast<uint4*>(at[r] + k) =
                    make_uint4(u[r][0], u[r][1], u[r][2], u[r][3]);
    }
    if (!live) return;
    const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
    if (p.lse != nullptr) p.lse[to] = lse2 * 0.693147180559945309f;
    if (row_lse != nullptr) *row_lse = lse2;
}

template <int HD, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const AttendParams p) {
    using C = Cfg<HD, NQ>;
    constexpr int TILE = C::kTile, NG = C::kGroups;
    constexpr int kJobs = C::kJobs, kBuffers = C::kBuffers;
    constexpr int kChunks = HD / 64;  // 128-byte columns of an operand row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sKV = sQ + C::kQBytes;
    Barriers& bar = *reinterpret_cast<Barriers*>(sKV + C::kStages * C::kStageBytes);
    static_assert(sizeof(Barriers) <= 1024, "barrier block");
    // (a shuffle, so that the compiler knows the roles' branches to be the whole warp's)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int span = NQ * p.nodes_tile;

    if (warp == 2) {
        tmem_alloc(&bar.tmem, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], NQ);
        }
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, NG);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
        }
        for (int i = 0; i < 2 * kFlagSlots; ++i) (&bar.bad_value[0][0])[i] = -1;
        mbar_init(&bar.values, 8);
        bar.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // Where this CTA's range of the list begins: a scan of the sequences' tiles.
    {
        const int each = ceil_div(p.num_seqs, kThreads);
        const int s0 = min(static_cast<int>(threadIdx.x) * each, p.num_seqs);
        const int s1 = min(s0 + each, p.num_seqs);
        int tiles = 0;
        int items = 0;
        SeqInfo x;  // (with one sequence a thread, still there for the second look)
        for (int s = s0; s < s1; ++s) {
            x = load_seq(p, s);
            const int nb = ceil_div(ceil_div(x.nodes, span), p.members);
            tiles += seq_tiles<TILE>(p, x, span, nb);
            items += nb * p.nkv;
            if (blockIdx.x == 0) {
                if (__ldg(p.q_offsets + s + 1) - x.q0 > p.max_q)
                    raise_error(p.dev_status, p.lib_error, HSS_ERR_INVALID_ARGUMENT);
                if (x.cut)
                    raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
            }
        }
        int before = tiles;
        int items_before = items;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, before, m);
            const int q = __shfl_up_sync(0xffffffffu, items_before, m);
            if (lane >= m) {
                before += o;
                items_before += q;
            }
        }
        if (lane == 31) {
            bar.scan[warp] = before;
            bar.scan_items[warp] = items_before;
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        before -= tiles;
        items_before -= items;
        int total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                before += bar.scan[w];
                items_before += bar.scan_items[w];
            }
            total += bar.scan[w];
        }
        const int per = ceil_div(total, p.groups);
        if (threadIdx.x == 0) {
            bar.start.total = total;
            bar.start.per = per;
            if (blockIdx.x == 0) {
                p.header[0] = total;
                p.header[1] = per;
            }
        }
        const int f0 = static_cast<int>(blockIdx.x) / p.members * per;
        for (int s = s0; s < s1; ++s) {
            if (each > 1) x = load_seq(p, s);
            const int nb = ceil_div(ceil_div(x.nodes, span), p.members);
            const int n = seq_tiles<TILE>(p, x, span, nb);
            if (blockIdx.x == 0) {
                p.seq_tiles[s] = before;
                p.seq_items[s] = items_before;
            }
            if (before <= f0 && f0 < before + n) {
                int o = f0 - before;
                int b = 0, bt = batch_tiles<TILE>(p, x, span, 0);
                while (o >= bt * p.nkv) {
                    o -= bt * p.nkv;
                    bt = batch_tiles<TILE>(p, x, span, ++b);
                }
                bar.start.s = s;
                bar.start.b = b;
                bar.start.h = o / bt;
                bar.start.t = o % bt;
                bar.start.item0 = items_before;
            }
            before += n;
            items_before += nb * p.nkv;
        }
        if (threadIdx.x == 0 && f0 >= total) bar.start.t = 0;  // no range: not within an item
        __syncthreads();
        if (threadIdx.x == 0 && blockIdx.x % p.members == 0)
            p.starts[blockIdx.x / p.members] = bar.start;
    }
    const uint32_t tmem = bar.tmem;
    volatile int* abort_flag = &bar.abort;
    const int boxes = TILE / p.box;

    Walk<TILE> walk;
    Segment g{};
    // A role that gives up reports it and sends the others home.
    auto give_up = [&]() {
        if (lane == 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp < 4) {
        walk.begin(p, bar.start, span);
        auto wait = [&](uint64_t* b, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_phase(b, parity, abort_flag)) != 0;
        };
        if (warp < 2) {
            // ------------------------------------------------------------ TMA
            // Own tiles: warp w brings K and V of group w's tiles.  Else warp 0 K and warp 1 V.
            constexpr bool own = C::kOwnTiles;
            const int first = own ? warp : 0, step = own ? 2 : 1;
            const bool keys = own || warp == 0, values = own || warp == 1;
            const bool loads = lane < boxes;  // a box per lane
            uint32_t tile = 0, segs = 0;      // issued so far
            bool ok = true;
            // The block id under this lane's box of tile t, read ahead of its use (-1 past the
            // sequence's tokens).
            auto block_of = [&](int t) -> int {
                const int pos = t * TILE + lane * p.box;
                return loads && pos < g.x.tokens ? __ldg(p.table + g.x.e0 + pos / p.bs) : -1;
            };
            auto load = [&](bool v, int group_row) -> bool {
                int st;
                uint32_t par;
                place<C>(v, first, tile, st, par);
                if (!wait(&bar.empty[st], par ^ 1u)) return false;
                if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], C::kStageBytes);
                __syncwarp();
                if (loads)
                    tma_load_5d(sKV + st * C::kStageBytes + lane * p.box * (HD * 2),
                                v ? &map_v : &map_k, &bar.full[st], 0, 0, 0, group_row, g.h);
                __syncwarp();
                return true;
            };
            while (ok && walk.next(p, g)) {
                if (g.n == 0) continue;
                if (warp == 0) {
                    if (segs > 0 && !(ok = wait(&bar.q_empty, (segs - 1) & 1))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.q_full,
                                              NQ * kChunks * 128 * p.g * p.nodes_tile);
                        for (int q = 0; q < NQ; ++q)
                            for (int ch = 0; ch < kChunks; ++ch)
                                tma_load_3d(sQ + q * (kRows * HD * 2) + ch * (kRows * 128), &map_q,
                                            &bar.q_full, ch * 64, g.h * p.g,
                                            g.x.q0 + (g.rt * NQ + q) * p.nodes_tile);
                    }
                    __syncwarp();
                }
                ++segs;
                int id = first < g.n ? block_of(g.ta + first) : -1;
                for (int i = first; i < g.n; i += step, ++tile) {
                    const int ahead = i + step < g.n ? block_of(g.ta + i + step) : -1;
                    const int pos = (g.ta + i) * TILE + lane * p.box;
                    const bool good = id >= 0 && id < p.max_blocks;
                    // groups of 8 tokens; past the cache's last one zeros are read
                    const int group_row =
                        static_cast<int>((good ? static_cast<int64_t>(id) * p.bs + pos % p.bs
                                               : p.max_blocks * p.bs) / 8);
                    if (keys) {
                        // bad ids of the tile, as granules of 16 tokens
                        const bool bad = loads && pos < g.x.tokens && !good;
                        uint32_t bits = __ballot_sync(0xffffffffu, bad);
                        if (bits != 0) {
                            if (bad) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
                            uint32_t grains = 0;
                            for (int k = 0; k < TILE / 16; ++k)
                                grains |= ((bits >> (16 * k / p.box)) & 1u) << k;
                            bits = grains;
                        }
                        // (its stage's barrier publishes it: written before the copies)
                        if (lane == 0) bar.bad_ids[first][tile % kMetaRing] = bits;
                        if (!(ok = load(false, group_row))) break;
                    }
                    if (values && !(ok = load(true, group_row))) break;
                    id = ahead;
                }
            }
            if (!ok) give_up();
            // Nobody leaves before the copies have landed and the products have released what
            // they read: the last use of every stage (after a failure, when the count may be off,
            // every stage gets time to finish the copy that it may be waiting for).
            const int begin = own ? warp * C::kRing0 : (keys ? 0 : C::kRing0);
            const uint32_t depth = keys ? C::kRing0 : C::kRing1;
            const uint32_t uses = own ? 2 * tile : tile;
            for (uint32_t i = 0; i < depth; ++i) {
                if (!ok) {
                    (void)mbar_wait_for(&bar.full[begin + i], 0, 1000000);
                    (void)mbar_wait_for(&bar.full[begin + i], 1, 1000000);
                } else if (uses > i) {
                    const uint32_t par = ((uses - 1 - i) / depth) & 1;  // round of its last use
                    (void)mbar_wait(&bar.full[begin + i], par);
                    (void)mbar_wait(&bar.empty[begin + i], par);
                }
            }
            if (warp == 0 && segs > 0) {
                (void)mbar_wait_for(&bar.q_full, (segs - 1) & 1, ok ? kWaitLimitNs : 1000000);
                if (ok) (void)mbar_wait(&bar.q_empty, (segs - 1) & 1);
            }
        } else if (warp - 2 < NG) {
            // ------------------------------------------------------------ products of group w
            const int w = warp - 2;
            constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, 64);
            constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, HD) | (1u << 16);  // V: MN-major
            constexpr uint32_t kJobBytes = 64 * HD * 2;  // a job's part of a stage
            const uint32_t leader = elect_one();
            // Descriptors: the high words do not change, the low ones by (offset >> 4) only.
            const uint64_t dq = smem_desc_kmajor(smem_u32(sQ), 128) +
                                (NQ == 2 ? w * (kRows * HD * 2 >> 4) : 0);
            const uint64_t dk = smem_desc_128b(smem_u32(sKV), kChunks * 1024, 0);
            const uint64_t dv = smem_desc_128b(smem_u32(sKV), kChunks * 1024, 1024);
            const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
            const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
            const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
            const uint32_t d_s = tmem + w * (kBuffers * 64);
            const uint32_t d_o = tmem + C::kOCols + w * HD;
            uint32_t tile = 0, segs = 0;
            uint32_t taken = 0;  // bit b: parity of buffer b's next weights
            bool ok = true;
            while (ok && walk.next(p, g)) {
                if (g.n == 0) continue;
                if (!(ok = wait(&bar.q_full, segs & 1))) break;
                ++segs;
                int tiles;
                const int jobs = __shfl_sync(0xffffffffu, jobs_of<C>(g, w, tiles), 0);
                if (jobs == 0 && leader) mbar_arrive(&bar.q_empty);
                __syncwarp();
                int sk = 0, sv = 0;  // the stages of the tile that each product is on
                auto stage_of = [&](bool v, int j, int& st) {
                    if (j % kJobs != 0) return;
                    uint32_t par;
                    place<C>(v, w, tile + j / kJobs, st, par);
                    st = __shfl_sync(0xffffffffu, st, 0);
                    ok = ok && wait(&bar.full[st], par);
                };
                auto score = [&](int j) {
                    const int b = kBuffers == 2 ? j & 1 : 0;
                    const uint32_t k =
                        k_lo + ((sk * C::kStageBytes + (j % kJobs) * kJobBytes) >> 4);
#pragma unroll
                    for (int s = 0; s < HD / 16; ++s)
                        umma_bf16_warp(leader, d_s + 64 * b,
                                       q_lo + (s >> 2) * (kRows * 128 >> 4) + 2 * (s & 3), q_hi,
                                       k + (s >> 2) * (1024 >> 4) + 2 * (s & 3), k_hi, idesc_s,
                                       s > 0);
                    umma_commit_warp(leader, &bar.s_full[w * kBuffers + b]);
                };
                auto scored = [&](int j) {  // releases behind the scores
                    if (j % kJobs == kJobs - 1 || j == jobs - 1)
                        umma_commit_warp(leader, &bar.empty[sk]);
                    if (j == jobs - 1) umma_commit_warp(leader, &bar.q_empty);
                };
                for (int j = 0; j < kBuffers && j < jobs && ok; ++j) {
                    stage_of(false, j, sk);
                    if (!ok) break;
                    tc_fence_after_sync();
                    score(j);
                    scored(j);
                }
                for (int j = 0; j < jobs && ok; ++j) {
                    // Everything but the weights is waited for first; nothing comes between the
                    // weights and the scores that go into their buffer, which the group will
                    // wait for, not even the commits that only release stages.
                    const int b = kBuffers == 2 ? j & 1 : 0;
                    const bool more = j + kBuffers < jobs;
                    stage_of(true, j, sv);
                    if (more) stage_of(false, j + kBuffers, sk);
                    ok = ok && wait(&bar.p_full[w * kBuffers + b], (taken >> b) & 1);
                    if (!ok) break;
                    taken ^= 1u << b;
                    tc_fence_after_sync();
                    const uint32_t v =
                        v_lo + ((sv * C::kStageBytes + (j % kJobs) * kJobBytes) >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_bf16_ts_warp(leader, d_o, d_s + 64 * b + 8 * s,
                                          v + s * (2 * kChunks * 1024 >> 4), v_hi, idesc_o,
                                          j > 0 || s > 0);
                    if (more) score(j + kBuffers);
                    // (before the last jobs, the scores just issued will say as much)
                    if (!more) umma_commit_warp(leader, &bar.o_done[w * kBuffers + b]);
                    if (j % kJobs == kJobs - 1 || j == jobs - 1)
                        umma_commit_warp(leader, &bar.empty[sv]);
                    if (more) scored(j + kBuffers);
                }
                tile += tiles;
            }
            if (!ok) give_up();
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int w = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t o_cols = lanes + C::kOCols + w * HD;
        const int gt = quarter * 32 + lane;  // thread of the group
        uint32_t tile = 0, pieces = 0, values = 0;
        // bit b: parity of buffer b's next scores, of its next end of a piece
        uint32_t next = 0, ends = 0;
        bool ok = true;
        walk.begin(p, bar.start, span);
        if (w >= NG) walk.f = walk.f1;
        auto wait = [&](uint64_t* b, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_phase(b, parity, abort_flag)) != 0;
        };
        while (ok && walk.next(p, g)) {
            const SeqInfo& x = g.x;
            const int first = (g.rt * NQ + (NQ == 2 ? w : 0)) * p.nodes_tile;
            const int live = min(max(x.nodes - first, 0), p.nodes_tile) * p.g;
            const bool warp_live = quarter * 32 < live;
            const int node = first + row / p.g;
            float m = -INFINITY, l = 0.0f;
            int tiles;
            const int jobs = jobs_of<C>(g, w, tiles);
            // The row's first two mask words, on their way before they are needed.
            uint64_t word0 = 0, word1 = 0;
            if (row < live && (g.ta + g.n) * TILE > x.ctx) {
                word0 = node_word(p, x, node, 0);
                if (x.nodes > 64) word1 = node_word(p, x, node, 1);
            }
            // Tokens that every row of the CTA sees, and every row of this warp: the context, and
            // of a chain the nodes up to the first row's.  (With all of a chain's tiles masked
            // and their values looked over, a prompt of 4096 tokens took 447 us, so 282.)
            const bool chain = p.mask == nullptr;
            const int open_cta = min(x.ctx + (chain ? g.rt * span + 1 : 0), x.tokens);
            const int open = min(x.ctx + (chain ? first + quarter * 32 / p.g + 1 : 0), x.tokens);
            const int64_t unit0 =
                (static_cast<int64_t>(g.f) * p.members + walk.member) * NQ + (NQ == 2 ? w : 0);
            for (int j = 0; j < jobs; ++j) {
                const int b = kBuffers == 2 ? j & 1 : 0, half = j % kJobs;
                const int ti = C::kOwnTiles ? w + 2 * (j / kJobs) : j / kJobs;
                const int pos0 = (g.ta + ti) * TILE + 64 * half;
                if (!(ok = wait(&bar.s_full[w * kBuffers + b], (next >> b) & 1))) break;
                next ^= 1u << b;
                tc_fence_after_sync();
                const uint32_t bad =
                    *(volatile uint32_t*)&bar.bad_ids[C::kOwnTiles ? w : 0]
                                                     [(tile + j / kJobs) % kMetaRing] >> (4 * half);
                const bool special = pos0 + 64 > open || (bad & 15) != 0 || p.pre != 1.0f;
                if (pos0 + 64 > open_cta) {
                    // Values past the end become zero; so do a node's non-finite elements.
                    int sv;
                    uint32_t par;
                    place<C>(true, w, tile + j / kJobs, sv, par);
                    if (!(ok = wait(&bar.full[sv], par))) break;
                    uint8_t* part = sKV + sv * C::kStageBytes + half * (64 * HD * 2);
                    bool found = false, wrote = false;
                    for (int k = gt + (NQ == 2 ? w * 128 : 0); k < 64 * kChunks;
                         k += NQ == 2 ? 256 : 128) {
                        const int r = k % 64, ch = k / 64;
                        if (pos0 + r < open_cta) continue;
                        uint8_t* at = part + ((r >> 3) * kChunks + ch) * 1024;
                        if (pos0 + r >= x.tokens) {
                            wrote = true;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(
                                    at + swizzled_offset(r & 7, 16 * e, 128)) =
                                    make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 q[8];
                        uint32_t most = 0;  // the largest exponent field, twice in a word
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            q[e] = *reinterpret_cast<const uint4*>(
                                at + swizzled_offset(r & 7, 16 * e, 128));
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            most = __vmaxu2(__vmaxu2(most, __vmaxu2(q[e].x & 0x7FFF7FFFu,
                                                                    q[e].y & 0x7FFF7FFFu)),
                                            __vmaxu2(q[e].z & 0x7FFF7FFFu, q[e].w & 0x7FFF7FFFu));
                        if (max(most & 0xFFFFu, most >> 16) < 0x7F80u) continue;
                        found = true;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint32_t* u = &q[e].x;
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                if ((u[d] & 0x7F80u) == 0x7F80u) u[d] &= 0xFFFF0000u;
                                if ((u[d] & 0x7F800000u) == 0x7F800000u) u[d] &= 0x0000FFFFu;
                            }
                            *reinterpret_cast<uint4*>(at + swizzled_offset(r & 7, 16 * e, 128)) =
                                q[e];
                        }
                    }
                    if (found) {
                        const int piece = static_cast<int>(pieces), slot = piece & (kFlagSlots - 1);
                        *(volatile int*)&bar.bad_value[w][slot] = piece;
                        if (NQ == 2)
                            *(volatile int*)&bar.bad_value[w ^ 1][slot] = piece;
                    }
                    if (wrote || found) fence_proxy_async_smem();
                    __syncwarp();  // what reads tensor memory wants the warp as one
                    if (NQ == 2) {  // both groups read the tile: both wait until all of it is fit
                        if (lane == 0) mbar_arrive(&bar.values);
                        if (!(ok = wait(&bar.values, values & 1))) break;
                        ++values;
                    }
                }
                if (warp_live) {
                    const uint32_t s_cols = lanes + (w * kBuffers + b) * 64;
                    // The job's scores and their maximum in one read.
                    uint32_t v[64];
                    const float top0 = tmem_ldred_values(s_cols, v);
                    float top = tmem_ldred_values(s_cols + 32, v + 32);
                    tmem_ld_wait_for(v);
                    tmem_hold(v + 32);
                    float t0 = top0;
                    order_after_wait(t0);
                    order_after_wait(top);
                    if (!special) {
                        top = fmaxf(top, t0);
                    } else {
                        // What the row does not see goes to -inf.
                        if (p.pre != 1.0f) {
#pragma unroll
                            for (int d = 0; d < 64; ++d)
                                v[d] = __float_as_uint(__uint_as_float(v[d]) * p.pre);
                        }
                        const float seen[2] = {t0, top};
                        top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t bits = 0;
                            if (row < live)
                                bits = visible32(p, x, node, pos0 + 32 * k, word0, word1);
                            if ((bad >> (2 * k)) & 1) bits &= 0xFFFF0000u;
                            if ((bad >> (2 * k)) & 2) bits &= 0x0000FFFFu;
                            if (__all_sync(0xffffffffu, bits == 0xFFFFFFFFu || row >= live) &&
                                p.pre == 1.0f) {
                                top = fmaxf(top, seen[k]);  // (unused rows may hold anything)
                                continue;
                            }
#pragma unroll
                            for (int d = 0; d < 32; ++d) {
                                const float s = (bits >> d) & 1 ? __uint_as_float(v[32 * k + d])
                                                                : -INFINITY;
                                v[32 * k + d] = __float_as_uint(s);
                                top = fmaxf(top, s);
                            }
                        }
                    }
                    top *= p.c;
                    const bool grow = top > m + kLazy || m == -INFINITY;
                    const float m_new = grow ? fmaxf(top, m) : m;
                    if (__any_sync(0xffffffffu, grow && j > 0)) {
                        // The product before has to be done with O.  What was issued after it
                        // tells: with one buffer these scores, with two the next ones.  (A parity
                        // names a phase only if the one before it has completed and the one after
                        // has not: this warp has seen the scores before, and those after wait for
                        // weights that it has not given.)
                        if (kBuffers == 2) {
                            const int o = b ^ 1;
                            ok = j + 1 < jobs ? wait(&bar.s_full[w * 2 + o], (next >> o) & 1)
                                              : wait(&bar.o_done[w * 2 + o], (ends >> o) & 1);
                            if (!ok) break;
                            tc_fence_after_sync();
                        }
                        const float shrink =
                            grow ? (m == -INFINITY ? 0.0f : ex2(m - m_new)) : 1.0f;
                        l *= shrink;
#pragma unroll 1
                        for (int k = 0; k < HD; k += 32) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(o_cols + k, o);
                            tmem_ld_wait_for(o);
#pragma unroll
                            for (int d = 0; d < 32; ++d)
                                o[d] = __float_as_uint(__uint_as_float(o[d]) * shrink);
                            tmem_st_32x32b_x32(o_cols + k, o);
                        }
                    }
                    m = m_new;
                    const float base = m == -INFINITY ? 0.0f : -m;
                    const float2 c2 = make_float2(p.c, p.c), b2 = make_float2(base, base);
                    // The weights, packed to bf16, and their sums over 16 tokens (which stay in
                    // registers until the end: a branch in between would keep the exponentials
                    // of different granules from overlapping).  bf16, because both operands of
                    // a product have one type and V comes as it lies in the cache: an output is
                    // off by up to 2^-9 sum p |v| more for it.  What the rounding leaves, as a
                    // second product, would take that away for half as much tensor time again,
                    // where products and exponentials are what bounds many rows.  The sums take
                    // the weights before the rounding: lse and block weights are theirs.
                    float grain[4];
                    uint32_t packed[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int d = 0; d < 16; d += 2) {
                            float2 e = make_float2(__uint_as_float(v[16 * q + d]),
                                                   __uint_as_float(v[16 * q + d + 1]));
                            e = fma2(e, c2, b2);
                            e.x = ex2(e.x);
                            e.y = ex2(e.y);
                            sum = d == 0 ? e : add2(sum, e);
                            packed[8 * q + d / 2] = pack_bf16x2(e.x, e.y);
                        }
                        grain[q] = sum.x + sum.y;
                    }
                    tmem_st_32x32b_x32(s_cols, packed);
                    tmem_st_wait();
                    l += (grain[0] + grain[1]) + (grain[2] + grain[3]);
                    if (p.sums != nullptr && row < p.rowcap) {
                        const int64_t at =
                            (unit0 + static_cast<int64_t>(ti) * p.members * NQ) * kJobs + half;
                        float* sums = p.sums + at * 4 * p.rowcap + row;
                        p.sums_m[at * p.rowcap + row] = base;
#pragma unroll
                        for (int k = 0; k < 4; ++k) sums[k * p.rowcap] = grain[k];
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[w * kBuffers + b]);
            }
            if (!ok) break;
            // What this piece of the sequence came to.
            if (g.rows && warp_live) {
                const int64_t slot =
                    (static_cast<int64_t>(g.item + blockIdx.x / p.members) * p.members +
                     walk.member) * 2 + w;
                if (jobs > 0) {
                    const int b = kBuffers == 2 ? (jobs - 1) & 1 : 0;  // the last product
                    if (!(ok = wait(&bar.o_done[w * kBuffers + b], (ends >> b) & 1))) break;
                    tc_fence_after_sync();
                }
                const bool bad =
                    jobs > 0 && *(volatile int*)&bar.bad_value[w][pieces & (kFlagSlots - 1)] ==
                                    static_cast<int>(pieces);
                if (C::kWhole && walk.whole(p, g)) {
                    const int64_t to = (static_cast<int64_t>(x.q0) + node) * p.nq + walk.h * p.g +
                                       row % p.g;
                    write_whole<HD>(p, x, node, walk.h, bad, o_cols, row < live, to, m, l,
                                    p.sums == nullptr
                                        ? nullptr
                                        : p.row_lse + ((static_cast<int64_t>(g.item) * p.members +
                                                        walk.member) * NQ +
                                                       (NQ == 2 ? w : 0)) * p.rowcap + row);
                } else if (jobs > 0) {
#pragma unroll 2
                    for (int k = 0; k < HD; k += 32) {
                        uint32_t o[32];
                        __syncwarp();
                        tmem_ld_32x32b_x32(o_cols + k, o);
                        tmem_ld_wait_for(o);
                        if (row < live && p.ways > 0) {
                            float* at = p.part_o + (slot * HD + k) * p.rowcap + row;
#pragma unroll
                            for (int d = 0; d < 32; ++d)
                                at[d * p.rowcap] = __uint_as_float(o[d]);
                        } else if (row < live) {
                            float* at = p.part_o + (slot * p.rowcap + row) * HD + k;
#pragma unroll
                            for (int d = 0; d < 32; d += 4)
                                *reinterpret_cast<uint4*>(at + d) =
                                    make_uint4(o[d], o[d + 1], o[d + 2], o[d + 3]);
                        }
                    }
                }
                tc_fence_before_sync();
                if (row < live) p.part_ml[slot * p.rowcap + row] = make_float2(m, l);
                if (row == 0) p.part_bad[slot] = bad;
            }
            if (C::kOwnTiles ? jobs > 0 : g.n > 0) ++pieces;
            ends ^= jobs > 1 && kBuffers == 2 ? 3u : (jobs > 0 ? 1u : 0u);
            tile += tiles;
        }
        if (!ok) give_up();
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The list position of (batch, head) of a sequence and its length in tiles.
template <int TILE>
__device__ __forceinline__ void item_range(const AttendParams& p, const SeqInfo& x, int span,
                                           int seq0, int b, int h, int& f, int& n) {
    f = seq0;
    n = batch_tiles<TILE>(p, x, span, b);
    if (p.mask != nullptr)
        f += b * p.nkv * n;
    else
        for (int k = 0; k < b; ++k) f += p.nkv * batch_tiles<TILE>(p, x, span, k);
    f += h * n;
}

// Adds the non-finite values of the nodes a row sees.
template <int HD>
__device__ __forceinline__ void add_bad_values(const AttendParams& p, const SeqInfo& x,
                                               int node, int h, float* acc) {
    const int lane = threadIdx.x & 31;
    for (int j = 0; j < x.nodes; ++j) {
        if (x.ctx + j >= x.tokens) break;
        if (!((node_word(p, x, node, j >> 6) >> (j & 63)) & 1)) continue;
        const int pos = x.ctx + j;
        const int64_t id = p.table[x.e0 + pos / p.bs];
        if (id < 0 || id >= p.max_blocks) continue;
        const uint32_t* v = reinterpret_cast<const uint32_t*>(
            p.V + ((id * p.bs + pos % p.bs) * p.nkv + h) * HD);
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            const uint32_t u = v[lane + 32 * i];
            const float lo = __uint_as_float(u << 16);
            const float hi = __uint_as_float(u & 0xFFFF0000u);
            if (!isfinite(lo)) acc[2 * i] += lo;
            if (!isfinite(hi)) acc[2 * i + 1] += hi;
        }
    }
}

// A joined row: out, lse, and for the weights its log2 lse.
template <int HD>
__device__ __forceinline__ void write_row(const AttendParams& p, const SeqInfo& x, int node,
                                          int head, float m, float l, const float* acc,
                                          int64_t lse_at) {
    const int lane = threadIdx.x & 31;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = (static_cast<int64_t>(x.q0) + node) * p.nq + head;
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + at * HD);
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
        to[lane + 32 * i] = l == 0.0f ? 0u : pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0) {
        const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
        if (p.lse != nullptr) p.lse[at] = lse2 * 0.693147180559945309f;
        if (p.sums != nullptr) p.row_lse[lse_at] = lse2;
    }
}

// What a CTA of the join is about: (sequence, row tile, head) and where its pieces are.
struct Unit {
    SeqInfo x;
    int s, rt, h, member, g0, g1;  // groups from g0 to g1 have pieces
    int64_t item;
};

// By number; false if there is nothing to join.
template <int HD, int NQ>
__device__ __forceinline__ bool unit_by_number(const AttendParams& p, int unit, int row_tiles,
                                               Unit& u) {
    using C = Cfg<HD, NQ>;
    u.rt = unit % row_tiles;
    u.h = unit / row_tiles % p.nkv;
    u.s = unit / row_tiles / p.nkv;
    u.x = load_seq(p, u.s);
    const int b = u.rt / p.members, per = p.header[1];
    u.member = u.rt % p.members;
    u.item = p.seq_items[u.s] + b * p.nkv + u.h;
    if (u.rt * NQ * p.nodes_tile >= u.x.nodes) return false;
    int f, n;
    item_range<C::kTile>(p, u.x, NQ * p.nodes_tile, p.seq_tiles[u.s], b, u.h, f, n);
    u.g0 = f / per;
    u.g1 = (f + n - kBeside<C::kTile> - 1) / per;
    return !(C::kWhole && u.g0 == u.g1);
}

// By the end of a group's range and the member: what was cut there.
template <int HD, int NQ>
__device__ __forceinline__ bool unit_by_cut(const AttendParams& p, int number, Unit& u) {
    using C = Cfg<HD, NQ>;
    const int group = 1 + number / p.members, per = p.header[1];
    const Start st = p.starts[group];
    const int f = group * per - st.t;  // the item's first tile
    u.g0 = group - 1;
    if (st.t == 0 || f / per != u.g0) return false;  // not cut here, or here not first
    u.s = st.s;
    u.h = st.h;
    u.x = load_seq(p, u.s);
    const int n = batch_tiles<C::kTile>(p, u.x, NQ * p.nodes_tile, st.b) - kBeside<C::kTile>;
    if (st.t >= n) return false;  // cut behind its tiles
    u.member = number % p.members;
    u.rt = st.b * p.members + u.member;
    u.item = st.item0 + st.b * p.nkv + st.h;
    u.g1 = (f + n - 1) / per;
    return u.rt * NQ * p.nodes_tile < u.x.nodes;
}

// Joins the pieces of the rows.  Few rows: a CTA takes 8 / WPR rows of one (sequence, row tile,
// head), WPR warps to a row, so that the pieces of a row (a long sequence is cut into as many as
// there are CTAs to share it) are on their way together.
template <int HD, int NQ, int WPR>
__device__ __forceinline__ void join_rows(const AttendParams& p, int block, int row_tiles,
                                          int row_parts) {
    using C = Cfg<HD, NQ>;
    constexpr int kEach = HD / 32;  // elements of a row per lane, in pairs
    constexpr int kAtOnce = 32 / kEach;
    constexpr int kPieceWidth = NQ == 1 ? C::kGroups : 1;  // pieces of a row per CTA group
    __shared__ float sh_acc[WPR > 1 ? 8 : 1][HD];
    __shared__ float sh_l[8], sh_top[8];
    const int span = NQ * p.nodes_tile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = block % row_parts;
    Unit u;
    if (!unit_by_number<HD, NQ>(p, block / row_parts, row_tiles, u)) return;
    const SeqInfo& x = u.x;
    const int rt = u.rt, h = u.h, member = u.member, g0 = u.g0;
    const int64_t item = u.item;
    const int sub = warp % WPR;
    const int r = part * (8 / WPR) + warp / WPR;
    const int rows = min(max(x.nodes - rt * span, 0), span) * p.g;
    const bool mine = r < rows;
    const int pieces = mine ? (u.g1 - g0 + 1) * kPieceWidth : 0;
    const int node = rt * span + r / p.g;
    const int qt = NQ == 2 ? r / (p.nodes_tile * p.g) : 0;
    const int lr = r - qt * p.nodes_tile * p.g;
    // piece k of the row -> slot
    auto slot_of = [&](int k) -> int64_t {
        const int grp = k / kPieceWidth;
        const int w = NQ == 2 ? qt : k % kPieceWidth;
        return ((item + g0 + grp) * p.members + member) * 2 + w;
    };
    float top = -INFINITY, l = 0.0f, acc[kEach];
    int bad = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) acc[i] = 0.0f;
    for (int k = sub + WPR * lane; k < pieces; k += 32 * WPR) {
        const int64_t sl = slot_of(k);
        const float2 ml = p.part_ml[sl * p.rowcap + lr];
        if (ml.y != 0.0f) top = fmaxf(top, ml.x);
        bad |= p.part_bad[sl];
    }
    // The first pieces' O is on its way before their weights are known.
    float2 v[kAtOnce][kEach / 2];
    auto fetch = [&](int k0, int here) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            if (q >= here) break;
            const float2* o = reinterpret_cast<const float2*>(
                p.part_o + (slot_of(k0 + WPR * q) * p.rowcap + lr) * HD);
#pragma unroll
            for (int i = 0; i < kEach / 2; ++i) v[q][i] = o[lane + 32 * i];
        }
    };
    fetch(sub, (pieces - sub + WPR - 1) / WPR);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    bad = __any_sync(0xffffffffu, bad);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int k0 = sub; k0 < pieces; k0 += 32 * WPR) {
        float wt = 0.0f;
        if (k0 + WPR * lane < pieces) {
            const float2 ml = p.part_ml[slot_of(k0 + WPR * lane) * p.rowcap + lr];
            wt = ml.y != 0.0f ? exp2f(ml.x - base) : 0.0f;
            l += ml.y != 0.0f ? wt * ml.y : 0.0f;
        }
        const int here = min(32, (pieces - k0 + WPR - 1) / WPR);
        for (int k = 0; k < here; k += kAtOnce) {
            if (k0 != sub || k != 0) fetch(k0 + WPR * k, here - k);
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const float wk = __shfl_sync(0xffffffffu, wt, (k + q) & 31);
                if (k + q >= here || wk == 0.0f) continue;  // without weight O may be anything
#pragma unroll
                for (int i = 0; i < kEach / 2; ++i) {
                    acc[2 * i] += wk * v[q][i].x;
                    acc[2 * i + 1] += wk * v[q][i].y;
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float m = base;
    if constexpr (WPR > 1) {
        // The row's first warp adds up what the others have.
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i)
            *reinterpret_cast<float2*>(&sh_acc[warp][2 * (lane + 32 * i)]) =
                make_float2(acc[2 * i], acc[2 * i + 1]);
        if (lane == 0) {
            sh_l[warp] = l;
            sh_top[warp] = top;
        }
        bad = __syncthreads_or(bad);
        if (sub != 0 || !mine) return;
        float all = -INFINITY;
#pragma unroll
        for (int k = 0; k < WPR; ++k)
            if (sh_l[warp + k] != 0.0f) all = fmaxf(all, sh_top[warp + k]);
        m = all == -INFINITY ? 0.0f : all;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) {
            const float lk = sh_l[warp + k];
            if (lk == 0.0f) continue;
            const float t = sh_top[warp + k];
            const float wk = exp2f((t == -INFINITY ? 0.0f : t) - m);
            l += wk * lk;
#pragma unroll
            for (int i = 0; i < kEach / 2; ++i) {
                const float2 v =
                    *reinterpret_cast<const float2*>(&sh_acc[warp + k][2 * (lane + 32 * i)]);
                acc[2 * i] += wk * v.x;
                acc[2 * i + 1] += wk * v.y;
            }
        }
    }
    if (bad) add_bad_values<HD>(p, x, node, h, acc);
    write_row<HD>(p, x, node, h * p.g + r % p.g, m, l, acc,
                  ((item * p.members + member) * NQ + qt) * p.rowcap + lr);
}

// Many rows: a warp takes four rows of one (sequence, row tile, head) at a time, eight lanes a row
// for its pieces' m and l, so that the loads of several rows are in flight together.
template <int HD>
__device__ __forceinline__ void join_many(const AttendParams& p, int block, int row_tiles,
                                          int row_parts) {
    using C = Cfg<HD, 1>;
    constexpr int kEach = HD / 32;
    constexpr int kPieceWidth = C::kGroups;
    const int span = p.nodes_tile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = block % row_parts;
    const int r0 = part * 32 + warp * 4;
    Unit u;
    if (!(C::kWhole && row_tiles == 0
              ? unit_by_cut<HD, 1>(p, block / row_parts, u)
              : unit_by_number<HD, 1>(p, block / row_parts, row_tiles, u)))
        return;
    const SeqInfo& x = u.x;
    const int rt = u.rt, h = u.h, member = u.member, g0 = u.g0;
    const int64_t item = u.item;
    const int rows = min(max(x.nodes - rt * span, 0), span) * p.g;
    if (r0 >= rows) return;
    const int pieces = (u.g1 - g0 + 1) * kPieceWidth;
    auto place_of = [&](int r, int k) -> int64_t {  // row r's piece k, in rows of the workspace
        return (((item + g0 + k / kPieceWidth) * p.members + member) * 2 + k % kPieceWidth) *
                   p.rowcap + r;
    };
    // m of the row: lane 8 q + i looks at pieces i, i + 8, ... of row r0 + q
    const int my_row = min(r0 + lane / 8, rows - 1);
    float top = -INFINITY, l = 0.0f;
    int bad = 0;
    for (int k = lane % 8; k < pieces; k += 8) {
        const int64_t at = place_of(my_row, k);
        const float2 ml = p.part_ml[at];
        bad |= p.part_bad[at / p.rowcap];
        if (ml.y != 0.0f) top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.0f : top;
    float acc[4][kEach];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[q][i] = 0.0f;
    for (int k0 = 0; k0 < pieces; k0 += 8) {
        float wt = 0.0f;
        if (k0 + lane % 8 < pieces) {
            const float2 ml = p.part_ml[place_of(my_row, k0 + lane % 8)];
            wt = ml.y != 0.0f ? exp2f(ml.x - base) : 0.0f;
            l += ml.y != 0.0f ? wt * ml.y : 0.0f;
        }
        const int here = min(8, pieces - k0);
        for (int k = 0; k < here; ++k) {
            float2 v[4][kEach / 2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2* o = reinterpret_cast<const float2*>(
                    p.part_o + place_of(min(r0 + q, rows - 1), k0 + k) * HD);
#pragma unroll
                for (int i = 0; i < kEach / 2; ++i) v[q][i] = __ldcg(o + lane + 32 * i);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float wk = __shfl_sync(0xffffffffu, wt, 8 * q + k);
                if (wk == 0.0f) continue;  // without weight O may be anything
#pragma unroll
                for (int i = 0; i < kEach / 2; ++i) {
                    acc[q][2 * i] += wk * v[q][i].x;
                    acc[q][2 * i + 1] += wk * v[q][i].y;
                }
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const bool any_bad = __any_sync(0xffffffffu, bad) != 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = r0 + q;
        const float lq = __shfl_sync(0xffffffffu, l, 8 * q);
        const float mq = __shfl_sync(0xffffffffu, base, 8 * q);
        if (r >= rows) break;
        const int node = rt * span + r / p.g;
        if (any_bad) add_bad_values<HD>(p, x, node, h, acc[q]);
        write_row<HD>(p, x, node, h * p.g + r % p.g, mq, lq, acc[q],
                      (item * p.members + member) * p.rowcap + r);
    }
}

// Many rows, part_o by column: a task of 32 rows (one a lane, so that reads are whole lines) by
// kJoinCols columns, its pieces split over p.ways warps that put their sums together in shared
// memory, from where the rows go out with their columns side by side.  (32 columns to a task take
// 126 registers, half the warps: 41 trees of 76 nodes 65 us, with 16 columns 44.)
constexpr int kJoinCols = 16;

template <int HD, int NQ>
__device__ __forceinline__ void join_columns(const AttendParams& p, int block, int row_tiles,
                                             int row_parts) {
    using C = Cfg<HD, NQ>;
    constexpr int kPieceWidth = NQ == 1 ? C::kGroups : 1;
    __shared__ float sums[8][32][kJoinCols + 1];
    __shared__ float2 stats[8][32];
    __shared__ int flags[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ways = p.ways;
    const int way = warp % ways, task = (block % row_parts * 8 + warp) / ways;
    const int cb = task % (HD / kJoinCols), r32 = task / (HD / kJoinCols) % ceil_div(p.rowcap, 32);
    const int qt = task / (HD / kJoinCols) / ceil_div(p.rowcap, 32);
    Unit u;
    if (!(C::kWhole && row_tiles == 0
              ? unit_by_cut<HD, NQ>(p, block / row_parts, u)
              : unit_by_number<HD, NQ>(p, block / row_parts, row_tiles, u)))
        return;
    const SeqInfo& x = u.x;
    const int rt = u.rt, h = u.h, member = u.member, g0 = u.g0;
    const int64_t item = u.item;
    const int first = (rt * NQ + qt) * p.nodes_tile;  // node of the tile's first row
    const int rows = qt < NQ ? min(max(x.nodes - first, 0), p.nodes_tile) * p.g : 0;
    auto slot_of = [&](int k) -> int64_t {
        return ((item + g0 + k / kPieceWidth) * p.members + member) * 2 +
               (NQ == 2 ? qt : k % kPieceWidth);
    };
    if (r32 * 32 < rows) {
        const int pieces = (u.g1 - g0 + 1) * kPieceWidth;
        const int lr = min(r32 * 32 + lane, rows - 1);
        float top = -INFINITY, l = 0.0f, acc[kJoinCols];
        int bad = 0;
#pragma unroll
        for (int c = 0; c < kJoinCols; ++c) acc[c] = 0.0f;
#pragma unroll 2
        for (int k = way; k < pieces; k += ways) {
            const int64_t sl = slot_of(k);
            const float2 ml = p.part_ml[sl * p.rowcap + lr];
            bad |= p.part_bad[sl];
            const float* o = p.part_o + (sl * HD + cb * kJoinCols) * p.rowcap + lr;
            float v[kJoinCols];
#pragma unroll
            for (int c = 0; c < kJoinCols; ++c) v[c] = o[c * p.rowcap];
            if (ml.y == 0.0f) continue;  // without weight O may be anything
            const float m = fmaxf(top, ml.x);
            const float shrink = exp2f(top - m), wt = exp2f(ml.x - m);
            top = m;
            l = l * shrink + wt * ml.y;
#pragma unroll
            for (int c = 0; c < kJoinCols; ++c) acc[c] = acc[c] * shrink + wt * v[c];
        }
#pragma unroll
        for (int c = 0; c < kJoinCols; ++c) sums[warp][lane][c] = acc[c];
        stats[warp][lane] = make_float2(top, l);
        if (lane == 0) flags[warp] = bad;
    }
    __syncthreads();
    // Eight columns of a row to a lane; the task's warps take rows in turn.
    const int w0 = warp - way;
    constexpr int kLanes = kJoinCols / 8;
    for (int r0 = way * (32 / kLanes); r0 < 32; r0 += ways * (32 / kLanes)) {
        const int r = r0 + lane / kLanes, at = r32 * 32 + r, col = lane % kLanes * 8;
        if (at >= rows) break;
        float top = -INFINITY;
        int bad = 0;
        for (int w = w0; w < w0 + ways; ++w) {
            top = fmaxf(top, stats[w][r].x);
            bad |= flags[w];
        }
        float l = 0.0f, acc[8] = {};
        for (int w = w0; w < w0 + ways; ++w) {
            const float2 ml = stats[w][r];
            if (ml.y == 0.0f) continue;
            const float wt = exp2f(ml.x - top);
            l += wt * ml.y;
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] += wt * sums[w][r][col + c];
        }
        const int node = first + at / p.g;
        if (bad) {
            // Non-finite values of the nodes this row sees.
            for (int j = 0; j < x.nodes && x.ctx + j < x.tokens; ++j) {
                if (!((node_word(p, x, node, j >> 6) >> (j & 63)) & 1)) continue;
                const int pos = x.ctx + j;
                const int64_t id = p.table[x.e0 + pos / p.bs];
                if (id < 0 || id >= p.max_blocks) continue;
                const uint16_t* v =
                    p.V + ((id * p.bs + pos % p.bs) * p.nkv + h) * HD + cb * kJoinCols + col;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float e = __uint_as_float(static_cast<uint32_t>(v[c]) << 16);
                    if (!isfinite(e)) acc[c] += e;
                }
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] = l == 0.0f ? 0u : pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
        uint16_t* to = p.out +
                       ((static_cast<int64_t>(x.q0) + node) * p.nq + h * p.g + at % p.g) * HD +
                       cb * kJoinCols + col;
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        if (cb == 0 && col == 0) {
            const float lse2 = l == 0.0f ? -INFINITY : top + log2f(l);
            if (p.lse != nullptr)
                p.lse[(static_cast<int64_t>(x.q0) + node) * p.nq + h * p.g + at % p.g] =
                    lse2 * 0.693147180559945309f;
            if (p.sums != nullptr)
                p.row_lse[((item * p.members + member) * NQ + qt) * p.rowcap + at] = lse2;
        }
    }
}

template <int HD, int NQ, int WPR>
__global__ void __launch_bounds__(256, 3) join_kernel(const AttendParams p, int row_tiles,
                                                   int row_parts) {
    grid_dependency_wait();
    grid_launch_dependents();
    if constexpr (WPR > 1)
        join_rows<HD, NQ, WPR>(p, blockIdx.x, row_tiles, row_parts);
    else if (NQ == 2 || p.ways > 0)
        join_columns<HD, NQ>(p, blockIdx.x, row_tiles, row_parts);
    else
        join_many<HD>(p, blockIdx.x, row_tiles, row_parts);
}

// Few rows: the weights of kEntries table entries from e on of a sequence, by one warp: the sums
// of their granules over heads and rows (over the lanes), each scaled by its row's exp2(m - lse),
// with row r of head h's log2 lse at lse[h * rows + r].  Several entries at once, because what an
// entry costs is the way of its loads.
constexpr int kEntries = 4;

template <int HD>
__device__ __forceinline__ void entry_weights(const AttendParams& p, const SeqInfo& x, int seq0,
                                              int64_t e, const float* lse_of) {
    using C = Cfg<HD, 1>;
    constexpr int TILE = C::kTile, kGran = TILE / 16, kJobs = C::kJobs;
    const int lane = threadIdx.x & 31;
    const int grains = p.bs / 16;
    const int64_t gr0 = (e - x.e0) * grains;  // first granule of the first entry
    float sum[kEntries];
#pragma unroll
    for (int q = 0; q < kEntries; ++q) sum[q] = 0.0f;
    const int seen = ceil_div(tokens_upto(p, x, x.nodes), 16);
    const int rows = x.nodes * p.g;
    const int n = batch_tiles<TILE>(p, x, p.nodes_tile, 0);  // (one batch)
    for (int i = lane; i < rows * p.nkv; i += 32) {
        const int h = i / rows, r = i - h * rows;
        const float lse = lse_of[i];
        for (int k = 0; k < grains; ++k) {
            float m[kEntries], part[kEntries];
#pragma unroll
            for (int q = 0; q < kEntries; ++q) {
                const int64_t gr = gr0 + q * grains + k;
                part[q] = 0.0f;
                if (gr >= seen) continue;
                const int t = static_cast<int>(gr) / kGran, in = static_cast<int>(gr) % kGran;
                const int64_t at = seq0 + h * n + t;
                m[q] = p.sums_m[(at * kJobs + in / 4) * p.rowcap + r];
                part[q] = p.sums[(at * kGran + in) * p.rowcap + r];
            }
#pragma unroll
            for (int q = 0; q < kEntries; ++q)  // (without weight m may be anything)
                if (part[q] != 0.0f && lse != -INFINITY) sum[q] += part[q] * exp2f(-m[q] - lse);
        }
    }
#pragma unroll
    for (int q = 0; q < kEntries; ++q) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], o);
        if (lane == q && e + q < x.end)
            p.weights_out[e + q] =
                (p.weights_in != nullptr ? p.weights_in[e + q] * p.decay : 0.0f) + sum[q];
    }
}

// Many rows: first, every job's four granule sums over its row tile's rows, once the join has left
// the rows' lse.  A CTA takes a share of the jobs of one (sequence, head, row tile), a warp per
// job, its lanes on the rows (whose lse stay in registers), so that everything is read in whole
// lines.  The totals take the place of the first row's sums.
template <int HD, int NQ>
__global__ void __launch_bounds__(256) grains_kernel(const AttendParams p, int row_tiles,
                                                     int shares) {
    using C = Cfg<HD, NQ>;
    constexpr int TILE = C::kTile, kJobs = C::kJobs;
    const int span = NQ * p.nodes_tile;
    grid_dependency_wait();
    grid_launch_dependents();
    const int share = blockIdx.x % shares, unit = blockIdx.x / shares;
    const int qt = unit % NQ, rt = unit / NQ % row_tiles;
    const int h = unit / NQ / row_tiles % p.nkv, s = unit / NQ / row_tiles / p.nkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SeqInfo x = load_seq(p, s);
    const int first = (rt * NQ + qt) * p.nodes_tile;
    const int rows = min(max(x.nodes - first, 0), p.nodes_tile) * p.g;
    if (rows == 0) return;
    const int b = rt / p.members, member = rt % p.members;
    int f, n;
    item_range<TILE>(p, x, span, p.seq_tiles[s], b, h, f, n);
    const int jobs = ceil_div(tokens_upto(p, x, min(x.nodes, (rt + 1) * span)), 64);
    const int64_t lse_at =
        ((static_cast<int64_t>(p.seq_items[s] + b * p.nkv + h) * p.members + member) * NQ + qt) *
        p.rowcap;
    float lse[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = lane + 32 * q;
        lse[q] = r < rows ? p.row_lse[lse_at + r] : -INFINITY;
    }
    for (int j = share * 8 + warp; j < jobs; j += shares * 8) {
        const int64_t at = ((static_cast<int64_t>(f + j / kJobs) * p.members + member) * NQ + qt) *
                               kJobs + j % kJobs;
        float* sums = p.sums + at * 4 * p.rowcap;
        float m[4], part[4][4], total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = lane + 32 * q;
            m[q] = r < rows ? p.sums_m[at * p.rowcap + r] : 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) part[q][k] = r < rows ? sums[k * p.rowcap + r] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float scale = exp2f(-m[q] - lse[q]);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // (without weight m may be anything)
                if (part[q][k] != 0.0f && lse[q] != -INFINITY) total[k] += part[q][k] * scale;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                total[k] += __shfl_xor_sync(0xffffffffu, total[k], o);
        __syncwarp();
        if (lane < 4) sums[lane * p.rowcap] = lane == 0   ? total[0]
                                              : lane == 1 ? total[1]
                                              : lane == 2 ? total[2]
                                                          : total[3];
    }
}

// Then an entry's weight is the sum of its granules' totals over heads and row tiles: a warp per
// entry, its lanes on the (granule, head, row tile) triples.
template <int HD, int NQ>
__global__ void __launch_bounds__(256) weights_kernel(const AttendParams p, int shares,
                                                      int ways) {
    using C = Cfg<HD, NQ>;
    constexpr int TILE = C::kTile, kGran = TILE / 16;
    const int span = NQ * p.nodes_tile;
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x / shares, share = blockIdx.x % shares;
    const SeqInfo x = load_seq(p, s);
    const int seq0 = p.seq_tiles[s];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rts = ceil_div(x.nodes, span), grains = p.bs / 16;
    const int tiles = ceil_div(x.nodes, p.nodes_tile);  // row tiles with rows in use
    const int at_once = 8 / ways, way = warp % ways;
    __shared__ float parts[8];
    for (int64_t e0 = x.e0 + share * at_once; e0 < x.end; e0 += shares * at_once) {
        const int64_t e = e0 + warp / ways;
        float sum = 0.0f;
        for (int i = way * 32 + lane; e < x.end && i < grains * p.nkv * rts * NQ;
             i += ways * 32) {
            const int qt = i % NQ, rt = i / NQ % rts, h = i / NQ / rts % p.nkv;
            const int64_t gr = (e - x.e0) * grains + i / NQ / rts / p.nkv;
            const int seen = ceil_div(tokens_upto(p, x, min(x.nodes, (rt + 1) * span)), 16);
            if (gr >= seen || rt * NQ + qt >= tiles) continue;
            int f, n;
            item_range<TILE>(p, x, span, seq0, rt / p.members, h, f, n);
            const int t = static_cast<int>(gr) / kGran, in = static_cast<int>(gr) % kGran;
            const int64_t at =
                (static_cast<int64_t>(f + t) * p.members + rt % p.members) * NQ + qt;
            sum += p.sums[(at * kGran + in) * p.rowcap];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (ways > 1) {
            __syncthreads();
            if (lane == 0) parts[warp] = sum;
            __syncthreads();
            for (int k = 1; way == 0 && k < ways; ++k) sum += parts[warp + k];
        }
        if (lane == 0 && way == 0 && e < x.end)
            p.weights_out[e] = (p.weights_in != nullptr ? p.weights_in[e] * p.decay : 0.0f) + sum;
    }
}

// Join and weights in one launch, for one row tile (NQ 1, one member): the first CTAs join, the
// others each take a share of one sequence's entries and work the rows' lse out for themselves
// from the pieces' m and l, which for a few rows is quicker than waiting for the join.
constexpr int kFewRows = 256;  // rows of a sequence, nodes times query heads

template <int HD, int WPR>
__global__ void __launch_bounds__(256, 3) finish_kernel(const AttendParams p, int row_tiles,
                                                        int row_parts, int join_ctas,
                                                        int shares) {
    using C = Cfg<HD, 1>;
    __shared__ float sh_lse[kFewRows];
    grid_dependency_wait();
    grid_launch_dependents();
    if (static_cast<int>(blockIdx.x) < join_ctas) {
        if constexpr (WPR > 1)
            join_rows<HD, 1, WPR>(p, blockIdx.x, 1, row_parts);
        else if (p.ways > 0)
            join_columns<HD, 1>(p, blockIdx.x, row_tiles, row_parts);
        else
            join_many<HD>(p, blockIdx.x, row_tiles, row_parts);
        return;
    }
    const int s = (blockIdx.x - join_ctas) / shares, share = (blockIdx.x - join_ctas) % shares;
    const int warp = threadIdx.x >> 5;
    const SeqInfo x = load_seq(p, s);
    const int seq0 = p.seq_tiles[s], per = p.header[1];
    const int item0 = p.seq_items[s];
    const int rows = x.nodes * p.g;  // of a head
    const int entries = x.end - x.e0;
    if (share * 8 * kEntries >= entries) return;
    const int n = batch_tiles<C::kTile>(p, x, p.nodes_tile, 0);  // (one batch)
    // lse of row i = (head, row): as many lanes to a row as keep the CTA busy
    const int all = rows * p.nkv;
    const int lanes = all <= 8 ? 32 : all <= 16 ? 16 : all <= 32 ? 8 : all <= 64 ? 4 : 1;
    const int per_pass = 256 / lanes;
    for (int i0 = 0; i0 < all; i0 += per_pass) {
        const int i = i0 + static_cast<int>(threadIdx.x) / lanes, at = threadIdx.x % lanes;
        float top = -INFINITY, l = 0.0f;
        if (i < all && n > 0) {
            const int h = i / rows, lr = i % rows;
            const int f = seq0 + h * n;
            const int g0 = f / per, g1 = (f + n - kBeside<C::kTile> - 1) / per;
            const int pieces = (g1 - g0 + 1) * C::kGroups;
            for (int k0 = at; k0 < pieces; k0 += 8 * lanes) {
                float2 ml[8];
                float m = top;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int k = k0 + q * lanes;
                    ml[q] = make_float2(-INFINITY, 0.0f);
                    if (k >= pieces) continue;
                    const int64_t slot =
                        static_cast<int64_t>(item0 + h + g0 + k / C::kGroups) * 2 + k % C::kGroups;
                    ml[q] = p.part_ml[slot * p.rowcap + lr];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (ml[q].y != 0.0f) m = fmaxf(m, ml[q].x);
                l = l != 0.0f ? l * exp2f(top - m) : 0.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (ml[q].y != 0.0f) l += ml[q].y * exp2f(ml[q].x - m);
                top = m;
            }
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const float ot = __shfl_xor_sync(0xffffffffu, top, o);
            const float ol = __shfl_xor_sync(0xffffffffu, l, o);
            const float m = fmaxf(top, ot);
            l = (l != 0.0f ? l * exp2f(top - m) : 0.0f) + (ol != 0.0f ? ol * exp2f(ot - m) : 0.0f);
            top = m;
        }
        if (i < all && at == 0) sh_lse[i] = l == 0.0f ? -INFINITY : top + log2f(l);
    }
    __syncthreads();
    for (int64_t e = x.e0 + (share * 8 + warp) * kEntries; e < x.end; e += shares * 8 * kEntries)
        entry_weights<HD>(p, x, seq0, e, sh_lse);
}

// ------------------------------------------------------------------------------------- host

// How a call is cut up; everything the workspace depends on.
struct Plan {
    int nq_tiles;    // row tiles per CTA: 1 or 2
    int nodes_tile;  // nodes per row tile
    int row_tiles;   // row tiles (or pairs) of the largest tree
    int members, groups;
    int rowcap;
    int tile;
    bool few;        // few rows in all: a CTA joins one
    int tasks, ways;  // of join_columns: a unit's tasks and the warps to each, 0 for part_o by row
    bool fits;  // few enough slots and tiles for 32-bit positions, and CTAs for a grid
    int64_t slots, tiles, units;
    // The grids behind the attention itself.
    int parts;                // CTAs of a unit that is joined
    int join_tiles;           // row_tiles, or 0: the join goes by the cuts of the list
    int shares, entry_ways;   // CTAs to a sequence's entries, warps to one
    int grain_shares;         // CTAs to a unit's jobs
    int64_t join_ctas, finish_ctas, grain_ctas;  // finish_ctas 0: join and weights by themselves
    size_t header, starts, seq_tiles, seq_items, part_o, part_ml, part_bad, row_lse, sums, sums_m,
        bytes;
};

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// The plan without its split: what does not depend on the members of a group.
Plan row_plan(const hss_dims& d, int32_t max_q) {
    Plan p = {};
    const int g = d.num_q_heads / d.num_kv_heads;
    p.nodes_tile = kRows / g;
    p.tile = d.head_dim <= 128 ? 128 : 64;
    p.nq_tiles = max_q > p.nodes_tile && d.head_dim < 256 ? 2 : 1;
    const int span = p.nq_tiles * p.nodes_tile;
    // (max_q may be anything up to 2^31 - 1)
    p.row_tiles = static_cast<int>(std::max<int64_t>(1, (int64_t{max_q} + span - 1) / span));
    p.rowcap = std::min(kRows, g * std::min(max_q, p.nodes_tile));
    return p;
}

constexpr int kMostMembers = 19;  // kCtas / 8

// Only numbers of members that leave no batch emptier than it must be: the workspace has room for
// every member of every batch (16 row tiles by 15 members would be two batches, 30 row tiles).
bool members_allowed(int row_tiles, int r) {
    const int batches = (row_tiles - 1) / r + 1;
    return r == (row_tiles - 1) / batches + 1;
}

// Members of a group, row tiles in step: many read K and V less often, few leave fewer CTAs
// waiting (in a last batch that is not full, in the upper rows of a chain, in groups that do not
// fill the GPU).  The estimate adds up the tiles that a sequence's batches walk, at 1500 cycles for
// 64 tokens under two row tiles and 1050 under one, with as many as three tiles' time for what an
// item costs besides, against the bytes at the memory's rate; the sequences' nodes are taken to lie
// evenly about their mean.  Measured, in us: 8 trees of 33 nodes, head_dim 256, by 1 member 577, by
// 3 410; 32 prompts of 512 tokens by 8 252, by 2 200; a prompt of 4096 by 2 508, by 8 496; 16
// prompts of 100 to 300 by 5 102, by 2 82.
int members_for(const Plan& p, const hss_dims& d, int32_t num_seqs, int32_t max_q, int64_t total_q,
                int64_t total_blocks, bool chain) {
    if (p.row_tiles == 1) return 1;
    const double seqs = std::max(num_seqs, 1);
    const double nodes = std::min<double>(total_q / seqs, max_q);
    const double fewest = std::max(1.0, 2.0 * nodes - max_q);
    const double context =
        std::max(0.0, (total_blocks / seqs - 0.5) * d.block_size - nodes) / p.tile;
    const int span = p.nq_tiles * p.nodes_tile;
    const double cycles = (p.nq_tiles == 2 ? 1500.0 : 1050.0) * (p.tile / 64);
    const double bytes = p.tile * d.head_dim * 4.0 / 3570.0;  // in cycles: 6.79 TB/s at 1.9 GHz
    double best = INFINITY;
    int members = 1;
    for (int r = 1; r <= std::min(p.row_tiles, kMostMembers); ++r) {
        if (!members_allowed(p.row_tiles, r)) continue;
        double tiles = 0.0;
        for (int i = 0; i < 4; ++i) {
            const double n = max_q - (max_q - fewest) * i / 3.0;
            const double batches = std::ceil(n / (static_cast<double>(span) * r));
            const double last = batches * span * r - n;  // nodes that the last one lacks
            const double seen = chain ? span * r * batches * (batches + 1.0) / 2.0 - last
                                      : batches * n;
            tiles += batches * (context + 3.0) + seen / p.tile;
        }
        const double compute = tiles / (kCtas / r) * cycles, memory = tiles * bytes;
        const double cost = std::max(compute, 1.2 * memory) + 0.3 * memory;
        if (cost <= best) {
            best = cost;
            members = r;
        }
    }
    return members;
}

// The grids of the join and of the weights, once the rows' part of the plan is there.
void plan_grids(Plan& p, const hss_dims& d, int32_t num_seqs, int32_t max_q, int64_t total_blocks,
                bool with_weights) {
    const int g = d.num_q_heads / d.num_kv_heads, grains = d.block_size / 16;
    const bool whole = p.nq_tiles == 2 || d.head_dim == 256;  // as Cfg::kWhole
    const int unit_rows = std::min(max_q, p.nq_tiles * p.nodes_tile) * g;
    const int64_t units = static_cast<int64_t>(p.row_tiles) * d.num_kv_heads * num_seqs;
    p.parts = p.few ? unit_rows : p.ways > 0 ? (p.tasks * p.ways + 7) / 8 : (unit_rows + 31) / 32;
    // What one group saw whole needs no join: where there are more units than cuts of the list, the
    // join goes by the cuts (43 chains of 202 nodes, 2064 units and 144 cuts: 60 us by unit, 4 by
    // cut; 3 trees of 31 to 95 nodes, 6 units and 150 cuts: 11 and 18).
    const int64_t cuts = static_cast<int64_t>(p.groups - 1) * p.members;
    const bool by_cut = whole && !p.few && cuts < units;
    p.join_ctas = (by_cut ? cuts : units) * p.parts;
    p.join_tiles = by_cut ? 0 : p.row_tiles;
    // Join and weights in one launch while a lane has few (row, granule) pairs of an entry to look
    // at in turn (36 sequences of 23 nodes, 14 heads and blocks of 32 tokens, 22 pairs, took 80 us
    // this way and 43 us through the granules' totals).
    const int64_t seq_rows = static_cast<int64_t>(max_q) * d.num_q_heads;
    const bool few_each = p.nq_tiles == 1 && p.row_tiles == 1 && with_weights &&
                          seq_rows <= kFewRows && (seq_rows + 31) / 32 * grains <= 8;
    // Warps to an entry: one for every 32 of its (granule, row tile, head) sums.  (8 trees of 81 to
    // 245 nodes of 128 heads: 32 us with one warp an entry, 9 with eight.)
    const int64_t each = static_cast<int64_t>(grains) * d.num_kv_heads * p.row_tiles * p.nq_tiles;
    p.entry_ways = 1;
    while (p.entry_ways < 8 && p.entry_ways * 32 < each) p.entry_ways *= 2;
    // CTAs to a sequence's entries: an even share of all entries in one pass, if the sequences
    // are alike, within what the GPU holds at once.
    const int64_t seqs = std::max(num_seqs, 1);
    const int64_t per_cta = few_each ? 8 * kEntries : 8 / p.entry_ways;
    const int64_t even = (total_blocks / seqs + per_cta) / per_cta;
    p.shares = static_cast<int>(std::min(even, std::max<int64_t>(1, 8 * kCtas / seqs)));
    p.finish_ctas = few_each ? p.join_ctas + static_cast<int64_t>(num_seqs) * p.shares : 0;
    // Shares of a unit's jobs: two passes over all warps that the GPU holds.
    const int64_t grain_units = units * p.nq_tiles;
    const int64_t jobs = total_blocks * d.block_size / 64 / seqs + 1;
    p.grain_shares = static_cast<int>(std::max<int64_t>(
        1, std::min((jobs + 7) / 8, 8 * kCtas / std::max<int64_t>(grain_units, 1))));
    p.grain_ctas = with_weights ? grain_units * p.grain_shares : 0;
}

Plan make_plan(const hss_dims& d, int32_t num_seqs, int32_t max_q, int64_t total_blocks,
               bool with_weights, int members) {
    Plan p = row_plan(d, max_q);
    const int g = d.num_q_heads / d.num_kv_heads;
    const int span = p.nq_tiles * p.nodes_tile;
    p.members = members;
    p.groups = std::max(1, kCtas / p.members);
    const int64_t batches = (int64_t{p.row_tiles} + p.members - 1) / p.members;
    const int beside = p.tile == 128 ? kBeside<128> : kBeside<64>;
    {
        // In floating point first: the products of the largest counts pass 64 bits.
        const double items = static_cast<double>(batches) * d.num_kv_heads * num_seqs;
        const double slots = (items + p.groups) * p.members * 2;
        const double tiles = static_cast<double>(batches) * d.num_kv_heads *
                             (static_cast<double>(total_blocks) * d.block_size / p.tile +
                              (1.0 + beside) * num_seqs);
        p.fits = slots <= (1 << 30) && tiles <= (1 << 30);
        if (!p.fits) return p;
    }
    // A CTA joins a row while that leaves SMs free (a lone sequence's 32 rows of 38 pieces).
    const int64_t units = static_cast<int64_t>(p.row_tiles) * d.num_kv_heads * num_seqs;
    p.few = units * std::min(max_q, span) * g <= 2 * kCtas;
    // A thread has a row of O to store.  By column a warp's 32 rows are a line a store, by row 32
    // lines that get 16 bytes each; but a join of few rows finds a row's columns quicker by row.
    // By row and by column: 32 rows of 8 heads of 64 sequences 52 and 55 us, 64 rows of 8 heads of
    // one sequence 61 and 43, a prompt of 4096 tokens 730 and 603.
    p.tasks = p.nq_tiles * ((p.rowcap + 31) / 32) * (d.head_dim / kJoinCols);
    p.ways = 0;
    if (!p.few && p.rowcap > 32) {
        // Warps to a task while there are pieces for them and the GPU has room.
        const int width = p.nq_tiles == 1 && d.head_dim < 256 ? 2 : 1;  // softmax groups to a row
        const int64_t pieces = (p.groups * p.members + units - 1) / units * width + 1;
        const int64_t cut = width == 2 ? units : std::min(units, int64_t{p.groups} * p.members);
        for (p.ways = 1; p.ways < 8 && p.ways < pieces && cut * p.tasks * p.ways < 32 * kCtas;)
            p.ways *= 2;
    }
    const int64_t items = batches * d.num_kv_heads * num_seqs;
    p.units = items * p.members * p.nq_tiles;
    p.slots = (items + p.groups) * p.members * 2;
    p.tiles = batches * d.num_kv_heads *
              (total_blocks * d.block_size / p.tile + int64_t{1 + beside} * num_seqs);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    p.header = take(8);
    p.starts = take(p.groups * sizeof(Start));
    p.seq_tiles = take(static_cast<size_t>(num_seqs) * 4);
    p.seq_items = take(static_cast<size_t>(num_seqs) * 4);
    p.part_bad = take(static_cast<size_t>(p.slots) * 4);
    p.part_ml = take(static_cast<size_t>(p.slots) * p.rowcap * 8);
    p.part_o = take(static_cast<size_t>(p.slots) * p.rowcap * d.head_dim * 4);
    p.row_lse = p.sums = p.sums_m = 0;
    if (with_weights) {
        const size_t lanes = static_cast<size_t>(p.tiles) * p.members * p.nq_tiles * p.rowcap;
        p.row_lse = take(static_cast<size_t>(p.units) * p.rowcap * 4);
        p.sums_m = take(lanes * (p.tile / 64) * 4);
        p.sums = take(lanes * (p.tile / 16) * 4);
    }
    p.bytes = at;
    plan_grids(p, d, num_seqs, max_q, total_blocks, with_weights);
    p.fits = p.join_ctas <= 0x7FFFFFFF && p.finish_ctas <= 0x7FFFFFFF &&
             p.grain_ctas <= 0x7FFFFFFF;
    if (!p.fits) p.bytes = 0;
    return p;
}

bool encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const uint16_t* base,
            int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<uint16_t*>(base), dims,
               strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_attr_mu;
bool g_attr_set[64][8] = {};

template <int HD, int NQ>
hss_status launch_all(const AttendParams& p, const Plan& plan, const CUtensorMap& mq,
                      const CUtensorMap& mk, const CUtensorMap& mv, int device, int which,
                      bool rows, cudaStream_t stream) {
    using C = Cfg<HD, NQ>;
    {
        std::lock_guard<std::mutex> lk(g_attr_mu);
        if (!g_attr_set[device & 63][which]) {
            if (cudaFuncSetAttribute(attend_kernel<HD, NQ>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmemBytes) != cudaSuccess)
                return HSS_ERR_CUDA;
            g_attr_set[device & 63][which] = true;
        }
    }
    if (launch_pdl(attend_kernel<HD, NQ>, dim3(plan.groups * plan.members), dim3(kThreads),
                   C::kSmemBytes, stream, mq, mk, mv, p) != cudaSuccess)
        return HSS_ERR_CUDA;
    if constexpr (NQ == 1) {
        if (rows && plan.finish_ctas > 0) {
            auto finish = plan.few ? finish_kernel<HD, 8> : finish_kernel<HD, 1>;
            if (launch_pdl(finish, dim3(static_cast<unsigned>(plan.finish_ctas)), dim3(256), 0,
                           stream, p, plan.join_tiles, plan.parts,
                           static_cast<int>(plan.join_ctas), plan.shares) != cudaSuccess)
                return HSS_ERR_CUDA;
            return HSS_OK;
        }
    }
    if (rows && plan.join_ctas > 0) {
        auto join = plan.few ? join_kernel<HD, NQ, 8> : join_kernel<HD, NQ, 1>;
        if (launch_pdl(join, dim3(static_cast<unsigned>(plan.join_ctas)), dim3(256), 0, stream, p,
                       plan.join_tiles, plan.parts) != cudaSuccess)
            return HSS_ERR_CUDA;
    }
    if (p.weights_out == nullptr) return HSS_OK;
    if (rows && launch_pdl(grains_kernel<HD, NQ>, dim3(static_cast<unsigned>(plan.grain_ctas)),
                           dim3(256), 0, stream, p, plan.row_tiles, plan.grain_shares) !=
                    cudaSuccess)
        return HSS_ERR_CUDA;
    // (without rows this is all, with the shares of a call that has some)
    if (launch_pdl(weights_kernel<HD, NQ>, dim3(static_cast<unsigned>(p.num_seqs * plan.shares)),
                   dim3(256), 0, stream, p, plan.shares, plan.entry_ways) != cudaSuccess)
        return HSS_ERR_CUDA;
    return HSS_OK;
}

}  // namespace

size_t attend_workspace_bytes(const hss_dims& d, int32_t num_seqs, int32_t max_q,
                              int64_t total_blocks, bool with_weights) {
    // (the members depend on more than the sizes given here)
    size_t most = 0;
    const int row_tiles = row_plan(d, max_q).row_tiles;
    for (int r = 1; r <= std::min(row_tiles, kMostMembers); ++r)
        if (members_allowed(row_tiles, r))
            most = std::max(most,
                            make_plan(d, num_seqs, max_q, total_blocks, with_weights, r).bytes);
    return most;
}

hss_status launch_attend(const AttendArgs& r, cudaStream_t stream) {
    const hss_attend_args& a = *r.a;
    const hss_dims& d = a.dims;
    const bool weigh = r.weights_out != nullptr;
    const int members = members_for(row_plan(d, a.max_q), d, a.num_seqs, a.max_q, a.total_q,
                                    a.total_blocks, a.tree_mask == nullptr);
    const Plan plan = make_plan(d, a.num_seqs, a.max_q, a.total_blocks, weigh, members);
    if (!plan.fits) return HSS_ERR_INVALID_ARGUMENT;
    const DeviceInfo* dev = current_device_info();
    if (dev == nullptr) return HSS_ERR_CUDA;
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return HSS_ERR_CUDA;
    AttendParams p;
    p.V = r.V;
    p.out = r.out;
    p.lse = r.lse;
    p.weights_in = r.weights_in;
    p.weights_out = r.weights_out;
    p.q_offsets = a.q_offsets;
    p.mask = a.tree_mask;
    p.table = a.block_table;
    p.seq_offsets = a.seq_offsets;
    p.ctx_len = a.ctx_len;
    p.max_blocks = d.max_blocks;
    p.total_blocks = a.total_blocks;
    p.mask_words = a.mask_words;
    p.num_seqs = a.num_seqs;
    p.max_q = a.max_q;
    p.nq = d.num_q_heads;
    p.nkv = d.num_kv_heads;
    p.g = p.nq / p.nkv;
    p.bs = d.block_size;
    p.box = std::min(d.block_size & -d.block_size, plan.tile);
    p.nodes_tile = plan.nodes_tile;
    p.members = plan.members;
    p.groups = plan.groups;
    p.rowcap = plan.rowcap;
    p.ways = plan.ways;
    p.c = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.44269504088896340736f;
    p.pre = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    p.decay = a.decay;
    p.dev_status = a.dev_status;
    p.lib_error = dev->error_word;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.header = reinterpret_cast<int32_t*>(ws + plan.header);
    p.starts = reinterpret_cast<Start*>(ws + plan.starts);
    p.seq_tiles = reinterpret_cast<int32_t*>(ws + plan.seq_tiles);
    p.seq_items = reinterpret_cast<int32_t*>(ws + plan.seq_items);
    p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml);
    p.part_bad = reinterpret_cast<int32_t*>(ws + plan.part_bad);
    p.row_lse = weigh ? reinterpret_cast<float*>(ws + plan.row_lse) : nullptr;
    p.sums = weigh ? reinterpret_cast<float*>(ws + plan.sums) : nullptr;
    p.sums_m = weigh ? reinterpret_cast<float*>(ws + plan.sums_m) : nullptr;
    const bool rows = a.total_q > 0;

    // Without rows nothing is loaded, but the maps have to be well formed.
    CUtensorMap mq, mk, mv;
    const uint16_t* some = reinterpret_cast<const uint16_t*>(a.workspace);
    const cuuint64_t hd = d.head_dim;
    {
        const cuuint64_t dims[3] = {hd, static_cast<cuuint64_t>(p.nq),
                                    static_cast<cuuint64_t>(std::max<int64_t>(a.total_q, 1))};
        const cuuint64_t strides[2] = {hd * 2, hd * 2 * p.nq};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.g),
                                   static_cast<cuuint32_t>(p.nodes_tile)};
        if (!encode(enc, &mq, rows ? r.Q : some, 3, dims, strides, box)) return HSS_ERR_CUDA;
    }
    {
        // 64 elements x 8 tokens x the head's 64-element columns x groups of 8 tokens x heads: a
        // box of 16 or more tokens lands as 8-row atoms, a group's columns side by side, so that
        // one copy brings whole rows and the atoms of an operand column stay evenly spaced.
        const cuuint64_t token = hd * 2 * p.nkv;
        const cuuint64_t groups = static_cast<cuuint64_t>(d.max_blocks) * p.bs / 8;
        if (groups > 0x7FFFFFFF) return HSS_ERR_UNSUPPORTED_SHAPE;
        const cuuint64_t dims[5] = {64, 8, hd / 64, groups, static_cast<cuuint64_t>(p.nkv)};
        const cuuint64_t strides[4] = {token, 128, token * 8, hd * 2};
        const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(hd / 64),
                                   static_cast<cuuint32_t>(p.box / 8), 1};
        if (!encode(enc, &mk, rows ? r.K : some, 5, dims, strides, box) ||
            !encode(enc, &mv, rows ? r.V : some, 5, dims, strides, box))
            return HSS_ERR_CUDA;
    }
    const int dv = dev->device;
    if (plan.nq_tiles == 2) {
        switch (d.head_dim) {
            case 64: return launch_all<64, 2>(p, plan, mq, mk, mv, dv, 0, rows, stream);
            case 128: return launch_all<128, 2>(p, plan, mq, mk, mv, dv, 1, rows, stream);
            default: return launch_all<192, 2>(p, plan, mq, mk, mv, dv, 2, rows, stream);
        }
    }
    switch (d.head_dim) {
        case 64: return launch_all<64, 1>(p, plan, mq, mk, mv, dv, 3, rows, stream);
        case 128: return launch_all<128, 1>(p, plan, mq, mk, mv, dv, 4, rows, stream);
        case 192: return launch_all<192, 1>(p, plan, mq, mk, mv, dv, 5, rows, stream);
        default: return launch_all<256, 1>(p, plan, mq, mk, mv, dv, 6, rows, stream);
    }
}

}  // namespace hss
