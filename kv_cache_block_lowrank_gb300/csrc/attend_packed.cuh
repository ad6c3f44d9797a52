// attend_packed.cuh -- attention of few rows over the packed cache: one pass over 4-bit tiles with
// warp-level matrix products; and the join that many rows (attend_packed_tc.cuh) share.
//
// A row is a (query row, query head of the group) pair; the rows of one sequence that share a kv
// head are taken R = 8 NT at a time.  Over the tokens they see, in tiles of 16,
//   S^T = K Q^T,  P = exp2(c S - m),  O^T = V^T P^T,  l = sum P
// with mma.m16n8k16: tokens (of V^T: elements) are the 16 rows of the product and query rows its 8
// columns, so that K and V, which are what there is much of, are the operand that goes from packed
// words straight into registers, and eight query rows fill an instruction.  (tcgen05 would want
// 128 rows and its operands in shared memory, where this kernel keeps nothing but the packed bytes.)
// A group's scale multiplies what the group adds to S, and for V the weight of its token: P is
// scaled, rounded to bf16 and transposed (movmatrix) once for each group of 32 elements.
//
// m is 8 above a row's maximum (in powers of two) and lags: it is one for the whole warp and a row, and
// moves only when a score passes it, so that a tile costs a vote and no shuffles.
//
// Split.  All (sequence, row tile, kv head, tile) form one list, cut into equal contiguous ranges, a
// CTA each (two to an SM).  Within a CTA the warps take the tiles of a unit (sequence, row tile,
// head) in turn, each with a ring of its own that its asynchronous copies fill, and put m, l and O
// together in shared memory at the unit's end or the range's.  What a range does not have whole goes
// to the workspace and a second kernel joins it.  Short units are not cut, and if all are short there
// is no list: a CTA takes a unit.
//
// What bounds it, and what it reaches on GB300 (HBM 6.8 TB/s measured): the latency of its own
// instructions.  A tile of 16 tokens of one head takes 312 of them for its 2304 bytes; the cache's
// bandwidth would leave time for 390 if every slot were used, but the 12 warps an SM that registers
// leave room for (168 each, 18 % of the warps there can be) use 55 % of the issue slots and wait for
// their own results most (ncu).  More warps with fewer registers each spill and were slower (16: 154 us
// where 12 took 145).  64 sequences of 1k to 16k tokens, 32 query heads on 8 of 128: 145 us, 4.4 TB/s;
// 152 sequences of 4096 tokens 157 us (a copy of an earlier version without its arithmetic, 116).  One
// of 32768 tokens 22.7 us: its tiles are 5.6 at HBM's rate, the rest is one way through memory after
// another (lengths, block ids, first tiles, pieces, join).  One of 500 tokens 11 us.
// What helped, on those 64 sequences: nibbles into the products without shifts for half of them,
// exact as bf16 counts them (240 to 193 us), scores begun with what the nibbles' 8 comes to, two tiles
// a step and twelve warps (160), cp.async without barriers in place of bulk copies (the same step),
// and units that weigh more than their tiles (143).
#pragma once

#include <algorithm>
#include <type_traits>

#include "packed.cuh"

namespace hss {
namespace packed {

constexpr int kSms = 152;          // GB300's; the workspace does not depend on the device
constexpr float kLazy = 8.0f;
constexpr int32_t kNoWindow = 0x7FFFFF00;
// Short contexts (as far as the host can tell: by the pages of the whole batch or by the window, so that
// many short sequences without a window are listed) of not too many units: a
// CTA takes a unit, and there is neither a list nor a join.  (32 heads on 8 of 128; with the list and
// so: one sequence of 500 tokens 14.4 and 11.2 us, of 2000 14.4 and 20.5; windows of 500 tokens of 16
// sequences 19.3 and 12.3, of 64 29.8 and 23.0, of 256 77 and 83; of 2000 tokens of 16 24.7 and 20.7.)
__host__ __device__ constexpr bool by_units(int64_t tiles, int64_t units) {
    return units <= 1024 && tiles <= (units >= 128 ? 128 : 64);
}
// The same for many rows, up to as many units as there are flags for.  (8 heads on 2 of 128: one
// sequence of 12 rows over 500 tokens 28 us with the list and 23 so, over 1500 29 and 43; 16 of 200
// rows over 1500 tokens, which is 128 units, 93 and 55.)
constexpr int kMostGuards = 2048;
__host__ __device__ constexpr bool many_by_units(int64_t tiles, int64_t units) {
    return units <= kMostGuards && tiles <= (units >= 100 ? 256 : 40);
}
// A unit this short is not cut: the range that it begins in takes all of it.  (Cut and so: 64 single
// tokens over 300 tokens 24.9 and 21.5 us, 16 chunks of 200 rows over 500 70 and 43.  A few units of
// twice this length are better cut: one chunk of 12 rows over 1500 tokens 29 and 45.)
template <int UNIT>
constexpr int kUncut = UNIT == 1 ? 48 : 20;
// In the list a unit is longer than its tiles by what it costs besides (its first loads, the warps'
// meeting, its rows' way out), so that ranges of equal length take equal time: in tiles here, in
// jobs of four for many rows.  (0, 16, 32, 64, 128 and 256: 64 sequences of 1k to 16k tokens 162, 153,
// 145, 144, 149 and 159 us; 16 windows of 4093 tokens with an empty sequence among them 63, 42, 35, 37,
// 41 and 48; 300 sequences of 300 to 1000 tokens 108, 97, 94, 94, 98 and 102; 32 of 1k to 8k with 4 kv
// heads of 256 56, 51, 52, 56, 62 and 74.  Many rows, 0, 3, 6, 12, 24 and 48: 512 rows over 32768
// tokens 512, 515, 512, 513, 512 and 531; 16 chunks of 200 over 2000 238, 230, 230, 222, 217 and 218; 40
// of 10 to 40 rows over 50 to 6000 tokens 246, 236, 208, 174, 162 and 182; 4 of 100 to 300 over 2k to
// 8k, heads of 256, 203, 193, 189, 190, 208 and 242: ragged chunks of 128 would rather have 12.)
template <int UNIT>
constexpr int kBeside = UNIT == 1 ? 32 : 6;
constexpr int kScanWarps = 20;      // of the largest CTA that looks for its range
constexpr int kRowWarps = 6;         // of a CTA that takes few rows
constexpr int kMostSlots = 4;       // of a warp's ring
constexpr int kControlBytes = 2048;  // barriers, and from 512 on the warps' walks

struct Start {
    int64_t total, per;  // the list's length, of a range
    int64_t t, cost;     // where the CTA's range begins in a unit, and the unit's length
    int32_t s, rt, h;
    int32_t q0, r0, live;  // the sequence's first query row, the unit's rows of it
};

struct Params {
    const uint16_t* Q;
    const uint8_t* cache;
    uint16_t* out;
    float* lse;
    const int32_t* q_offsets;
    const int32_t* table;
    const int32_t* seq_offsets;
    const int32_t* ctx_len;
    int64_t max_blocks;
    int64_t total_blocks;
    int32_t num_seqs, max_q, nq, nkv, g, bs;
    int32_t window;  // kNoWindow at most, which is none
    int32_t sinks;   // 0 without a window
    int32_t row_tiles;  // 0: the list; else a CTA takes a unit of this many row tiles a sequence
    float c;         // scale log2(e)
    int32_t* dev_status;
    int32_t* lib_error;
    // workspace
    Start* starts;    // [ranges]
    float2* part_ml;  // [2 ranges][R] (m, l)
    float* part_o;    // [2 ranges][R][head_dim]
    const int32_t* guard;  // [guards] or null: nothing is done if all are 0
    int32_t guards;
};

template <int HD, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    // Few rows: nibbles go into the products as they are (see raw_codes), two tiles at a time.
    static constexpr bool kRaw = NT == 1 && HD <= 128;
    static constexpr int kWarps = kRaw ? kRowWarps : 4;
    static constexpr int kTiles = kRaw ? 2 : 1;  // of a step, and of a ring's slot
    static constexpr int kCtas = 2;   // of an SM
    static constexpr int kRanges = kSms * kCtas;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kOStride = HD + 4;  // floats of a row of O in shared memory
    static constexpr int kOBytes = kWarps * kRows * kOStride * 4;
    static constexpr int kMlBytes = kWarps * kRows * 8;
    static constexpr int kSlotBytes = kTiles * Tile<HD>::kBytes;
    // (of the SM's 228 KB a CTA costs 1 KB besides, and its start may not be aligned)
    static constexpr int kBudget =
        233472 / kCtas - 1024 - 128 - kControlBytes - kOBytes - kMlBytes;
    static constexpr int kFits = kBudget / (kWarps * kSlotBytes);
    static constexpr int kSlots = kFits < kMostSlots ? kFits : kMostSlots;
    static constexpr int kSmemBytes =
        128 + kControlBytes + kOBytes + kMlBytes + kWarps * kSlots * kSlotBytes;
    static_assert(kSlots >= 2, "tiles in flight");
};

struct SeqInfo {
    int q0, rows, ctx, tokens;
    int64_t e0;
    bool cut;  // the table is too short for ctx_len + rows
};

__device__ __forceinline__ SeqInfo load_seq(const Params& p, int s) {
    SeqInfo x;
    x.q0 = __ldg(p.q_offsets + s);
    x.rows = min(max(__ldg(p.q_offsets + s + 1) - x.q0, 0), p.max_q);
    const int64_t e0 = __ldg(p.seq_offsets + s), end = __ldg(p.seq_offsets + s + 1);
    x.e0 = min(max(e0, int64_t{0}), p.total_blocks);
    const int64_t room = max(min(end, p.total_blocks) - x.e0, int64_t{0}) * p.bs;
    x.ctx = min(max(__ldg(p.ctx_len + s), 0), 0x7FFFFE00 - p.max_q);
    const int64_t want = static_cast<int64_t>(x.ctx) + x.rows;
    x.tokens = static_cast<int>(min(room, want));
    x.cut = room < want;
    return x;
}

// What is wrong with a sequence.
__device__ __forceinline__ void report(const Params& p, int s, const SeqInfo& x) {
    if (__ldg(p.q_offsets + s + 1) - x.q0 > p.max_q)
        raise_error(p.dev_status, p.lib_error, HSS_ERR_INVALID_ARGUMENT);
    if (x.cut && x.rows > 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
}

// What a row tile sees: tiles [0, sinks) and [w0, end).
struct View {
    int r0, live;        // its first row (of the sequence and kv head) and how many there are
    int at0, at1;        // positions of its first and last row
    int sinks, w0, end;  // tiles
    __device__ __forceinline__ int tiles() const { return sinks + end - w0; }
    // (a row tile that sees nothing still has its result to write)
    template <int UNIT>
    __device__ __forceinline__ int cost() const {
        return max((tiles() + UNIT - 1) / UNIT, 1);
    }
    __device__ __forceinline__ int tile(int k) const { return k < sinks ? k : w0 + (k - sinks); }
};

template <int R>
__device__ __forceinline__ View view_of(const Params& p, const SeqInfo& x, int rt) {
    View v;
    v.r0 = rt * R;
    v.live = min(x.rows * p.g - v.r0, R);
    v.at0 = x.ctx + v.r0 / p.g;
    v.at1 = x.ctx + (v.r0 + v.live - 1) / p.g;
    const int tokens = min(x.tokens, v.at1 + 1);
    v.end = (tokens + 15) >> 4;
    v.sinks = min((p.sinks >> 4) + ((p.sinks & 15) != 0 ? 1 : 0), v.end);
    // (at0 + 1 - window does not overflow: at0 >= 0)
    v.w0 = min(max(v.sinks, max(v.at0 + 1 - p.window, 0) >> 4), v.end);
    return v;
}

template <int R>
__device__ __forceinline__ int row_tiles(const Params& p, const SeqInfo& x) {
    return (x.rows * p.g + R - 1) / R;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The pieces of a CTA's range, one unit (or the range's part of it) after another; the list counts
// UNIT tiles as one.
template <int R, int UNIT>
struct Walk {
    SeqInfo x;
    View v;
    int s, rt, rts, h;
    int k, n;  // the piece: tiles [k, k + n) of the unit's view, from UNIT t on
    bool whole;
    int64_t f, f1;
    int t;

    __device__ __forceinline__ void begin(const Params& p, const Start& st, const SeqInfo& seq,
                                          const View& view) {
        f = min(st.total, blockIdx.x * st.per);
        f1 = min(st.total, f + st.per);
        s = st.s;
        rt = st.rt;
        h = st.h;
        t = static_cast<int>(st.t);
        x = seq;
        v = view;
        rts = row_tiles<R>(p, x);
    }
    // One unit and no list.
    __device__ __forceinline__ void begin_unit(const Params& p, int unit) {
        h = unit % p.nkv;
        rt = unit / p.nkv % p.row_tiles;
        s = unit / p.nkv / p.row_tiles;
        x = load_seq(p, s);
        rts = row_tiles<R>(p, x);
        t = 0;
        f = f1 = 0;
        if (rt < rts) {
            v = view_of<R>(p, x, rt);
            f1 = v.cost<UNIT>();
        }
    }
    __device__ __forceinline__ bool next(const Params& p) {
        while (f < f1) {
            const int all = v.cost<UNIT>();
            const bool uncut = all <= kUncut<UNIT>;
            if (t < all && !(uncut && t > 0)) {
                const int take =
                    uncut ? all : static_cast<int>(min(static_cast<int64_t>(all - t), f1 - f));
                k = UNIT * t;
                n = max(min(UNIT * (t + take), v.tiles()) - k, 0);
                whole = take == all;
                t += take;
                f += take;
                return true;
            }
            f += all + kBeside<UNIT> - t;
            t = 0;
            if (++h >= p.nkv) {
                h = 0;
                if (++rt >= rts) {
                    rt = 0;
                    do {
                        if (++s >= p.num_seqs) return false;
                        x = load_seq(p, s);
                        rts = row_tiles<R>(p, x);
                    } while (rts == 0);
                }
                v = view_of<R>(p, x, rt);
            }
        }
        return false;
    }
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// The codes of a word as bf16, nibbles j and j + 4 in out[j]: those of j = 0 and 2 divided by 64,
// those of 1 and 3 by 4.  The low eight bits of a bf16, the last of its exponent among them, count in
// steps of 2^-133 from 0 on, so that a nibble in either half of them needs no shift and no
// exponent put above it: times 2^127, less 8, in one exact operation.
__device__ __forceinline__ uint32_t code_fma(uint32_t nibbles, uint32_t minus) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(nibbles), "r"(0x7F007F00u), "r"(minus));
    return d;
}
__device__ __forceinline__ void codes_of(uint32_t (&out)[4], uint32_t w) {
    const uint32_t t = w >> 8;
    out[0] = code_fma(w & 0x000F000Fu, 0xBE00BE00u);  // (-1/8, -1/8)
    out[1] = code_fma(w & 0x00F000F0u, 0xC000C000u);  // (-2, -2)
    out[2] = code_fma(t & 0x000F000Fu, 0xBE00BE00u);
    out[3] = code_fma(t & 0x00F000F0u, 0xC000C000u);
}
// Nibbles as they are, bf16 in steps of 2^-133 (the tensor cores take such numbers as well as
// others): those of j = 1 and 3 sixteen times as large.  What multiplies them is scaled up by a
// power of two, and their 8 is taken away by a product with these:
__device__ __forceinline__ void raw_codes(uint32_t (&out)[4], uint32_t w) {
    const uint32_t t = w >> 8;
    out[0] = w & 0x000F000Fu;
    out[1] = w & 0x00F000F0u;
    out[2] = t & 0x000F000Fu;
    out[3] = t & 0x00F000F0u;
}
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;
// 2^x, -126 <= x <= 127.
__device__ __forceinline__ float pow2(int x) { return __int_as_float((x + 127) << 23); }
__device__ __forceinline__ uint32_t times2(uint32_t two, float f) {
    __nv_bfloat162 d = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&two),
                               __floats2bfloat162_rn(f, f));
    return *reinterpret_cast<uint32_t*>(&d);
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* at) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(at + 4 * i);
            w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(at + 4 * i);
            w[i] = u.x, w[i + 1] = u.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(at + 4 * i);
    }
}

// Group i of the scales in packed pairs.
template <int N>
__device__ __forceinline__ float scale_at(const uint32_t (&w)[N], int i) {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

struct alignas(8) Control {
    uint64_t arrived, merged;  // the warps' parts of a piece are there; are joined
    int abort;
    Start start;
    SeqInfo seq;  // of the unit where the range begins
    View view;
    int64_t scan[kScanWarps];
    alignas(8) float rest[kRowWarps][8];  // [warp][row] a part of a factor that is past fp32
};
static_assert(sizeof(Control) <= 512, "control block");

// Where every CTA's range begins, from a scan of the sequences' lengths.
template <int R, int UNIT, int THREADS>
__device__ __forceinline__ void find_start(const Params& p, Control& ctl, int64_t least) {
    static_assert(THREADS % 32 == 0 && THREADS / 32 <= kScanWarps, "a sum for every warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int each = (p.num_seqs + THREADS - 1) / THREADS;
    const int s0 = min(static_cast<int>(threadIdx.x) * each, p.num_seqs);
    const int s1 = min(s0 + each, p.num_seqs);
    auto length = [&](const SeqInfo& x) -> int64_t {
        const int n = row_tiles<R>(p, x);
        int64_t sum = 0;
        for (int rt = 0; rt < n; ++rt) sum += view_of<R>(p, x, rt).template cost<UNIT>() + kBeside<UNIT>;
        return sum * p.nkv;
    };
    int64_t mine = 0;
    SeqInfo x;  // (with one sequence a thread, still there for the second look)
    for (int s = s0; s < s1; ++s) {
        x = load_seq(p, s);
        mine += length(x);
        if (blockIdx.x == 0) report(p, s, x);
    }
    int64_t before = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, before, m);
        if (lane >= m) before += o;
    }
    if (lane == 31) ctl.scan[warp] = before;
    __syncthreads();
    before -= mine;
    int64_t total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += ctl.scan[w];
        total += ctl.scan[w];
    }
    const int64_t per = max(divide(total + gridDim.x - 1, gridDim.x), least);
    const int64_t f0 = blockIdx.x * per;
    if (threadIdx.x == 0) {
        ctl.start.total = total;
        ctl.start.per = per;
        if (f0 >= total) ctl.start.t = 0;  // no range: not within a unit
    }
    for (int s = s0; s < s1; ++s) {
        if (each > 1) x = load_seq(p, s);
        const int64_t n = length(x);
        if (before <= f0 && f0 < before + n) {
            int64_t o = f0 - before;
            int rt = 0;
            View v = view_of<R>(p, x, 0);
            while (o >= static_cast<int64_t>(v.cost<UNIT>() + kBeside<UNIT>) * p.nkv) {
                o -= static_cast<int64_t>(v.cost<UNIT>() + kBeside<UNIT>) * p.nkv;
                v = view_of<R>(p, x, ++rt);
            }
            const int64_t h = divide(o, v.cost<UNIT>() + kBeside<UNIT>);
            ctl.start.s = s;
            ctl.start.rt = rt;
            ctl.start.h = static_cast<int>(h);
            ctl.start.t = o - h * (v.cost<UNIT>() + kBeside<UNIT>);
            ctl.start.cost = v.cost<UNIT>();
            ctl.start.q0 = x.q0;
            ctl.start.r0 = v.r0;
            ctl.start.live = v.live;
            ctl.seq = x;
            ctl.view = v;
        }
        before += n;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.starts[blockIdx.x] = ctl.start;
}

// Whether the kernel has something to do (see Params::guard).
__device__ __forceinline__ bool wanted(const Params& p) {
    if (p.guard == nullptr) return true;
    int any = 0;
    for (int i = threadIdx.x; i < p.guards; i += blockDim.x) any |= p.guard[i];
    return __syncthreads_or(any) != 0;
}

// A finished row: out and lse.
template <int HD>
__device__ __forceinline__ void write_row(const Params& p, int q0, int r, int h, float m, float l,
                                          const float2 (&acc)[HD / 64]) {
    const int lane = threadIdx.x & 31;
    const int64_t at = (static_cast<int64_t>(q0) + r / p.g) * p.nq + h * p.g + r % p.g;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + at * HD);
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
        to[lane + 32 * i] = l == 0.0f ? 0u : pack_bf16x2(acc[i].x * inv, acc[i].y * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

template <int HD, int NT>
__global__ void __launch_bounds__(Shape<HD, NT>::kThreads, Shape<HD, NT>::kCtas)
    attend_kernel(const Params p) {
    using S = Shape<HD, NT>;
    using T = Tile<HD>;
    constexpr int R = S::kRows, W = S::kWarps, NG = T::kGroups, TT = S::kTiles;
    constexpr bool RAW = S::kRaw;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                               ~static_cast<uintptr_t>(127));
    Control& ctl = *reinterpret_cast<Control*>(smem);
    float* sh_o = reinterpret_cast<float*>(smem + kControlBytes);  // [W][R][kOStride]
    float2* sh_ml = reinterpret_cast<float2*>(smem + kControlBytes + S::kOBytes);  // [W][R]
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* ring =
        smem + kControlBytes + S::kOBytes + S::kMlBytes + warp * S::kSlots * S::kSlotBytes;
    // Where the warp's copies and its products are in the range (in shared memory: few of the
    // numbers are needed from tile to tile, and registers are short).
    static_assert(2 * W * sizeof(Walk<R, 1>) <= kControlBytes - 512, "walks");
    Walk<R, 1>& ahead = reinterpret_cast<Walk<R, 1>*>(smem + 512)[2 * warp];
    Walk<R, 1>& walk = reinterpret_cast<Walk<R, 1>*>(smem + 512)[2 * warp + 1];
    auto advance = [&](Walk<R, 1>& w) {
        __syncwarp();
        bool got = false;
        if (lane == 0) got = w.next(p);
        __syncwarp();
        return __shfl_sync(0xffffffffu, static_cast<int>(got), 0) != 0;
    };

    if (threadIdx.x == 0) {
        mbar_init(&ctl.arrived, W);
        mbar_init(&ctl.merged, W);
        ctl.abort = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    if (!wanted(p)) return;
    if (p.row_tiles == 0) {
        find_start<R, 1, S::kThreads>(p, ctl, TT * W);
        if (lane == 0) {
            ahead.begin(p, ctl.start, ctl.seq, ctl.view);
            walk.begin(p, ctl.start, ctl.seq, ctl.view);
        }
    } else if (lane == 0) {
        walk.begin_unit(p, blockIdx.x);
        ahead = walk;
        if (warp == 0 && walk.h == 0 && walk.rt == 0) report(p, walk.s, walk.x);
    }
    volatile int* abort_flag = &ctl.abort;

    // ---- the copies, a ring ahead of the products
    bool more = advance(ahead);
    int ahead_n = ahead.n;
    int ahead_k = TT * warp;  // the warp's tiles of the piece: TT of every TT W
    int ahead_j = 0;          // how many of them are issued
    int fill = 0;             // slot of the next copy
    uint32_t there = 0;       // bit TT * slot + k: the slot's tile k is there to be seen
    int64_t places = 0;       // lane i: where the i-th next of them lies, or -1
    auto issue = [&]() {
        while (more && ahead_k >= ahead_n) {
            more = advance(ahead);
            ahead_n = ahead.n;
            ahead_k = TT * warp;
            ahead_j = 0;
        }
        if (more) {
            if (ahead_j % 32 == 0) {
                const int k = ahead_k + lane / TT * (TT * W) + lane % TT;
                places = -1;
                if (k < ahead_n) {
                    const int pos = ahead.v.tile(ahead.k + k) * 16;
                    const int entry = pos / p.bs;
                    const int id = __ldg(p.table + ahead.x.e0 + entry);
                    if (id >= 0 && id < p.max_blocks)
                        places = ((static_cast<int64_t>(id) * p.nkv + ahead.h) * (p.bs / 16) +
                                  (pos - entry * p.bs) / 16) * T::kBytes;
                    else
                        raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
                }
            }
            uint32_t have = 0;
#pragma unroll
            for (int u = 0; u < TT; ++u) {
                const int64_t place = __shfl_sync(0xffffffffu, places, ahead_j % 32 + u);
                if (place < 0) continue;
                have |= 1u << u;
                const uint8_t* from = p.cache + place + 16 * lane;
                uint8_t* to = ring + fill * S::kSlotBytes + u * T::kBytes + 16 * lane;
#pragma unroll
                for (int i = 0; i < T::kBytes; i += 512)
                    if (i + 512 <= T::kBytes || i + 16 * lane < T::kBytes)
                        cp_async_16(to + i, from + i);
            }
            there = (there & ~(((1u << TT) - 1) << (TT * fill))) | have << (TT * fill);
            fill = fill + 1 == S::kSlots ? 0 : fill + 1;
            ahead_j += TT;
            ahead_k += TT * W;
        }
        cp_async_commit();  // (a group for every step, be it empty)
    };
    for (int i = 0; i < S::kSlots; ++i) issue();

    // ---- the products
    uint32_t pieces = 0;
    int slot = 0;
    bool ok = true;
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t eight_k[4] = {kMinus8, kMinus8, kMinus128, kMinus128};
    while (ok && advance(walk)) {
        const View& v = walk.v;
        const int tiles = walk.n, sinks = v.sinks, k_first = walk.k, w0 = v.w0 - sinks;
        const int tokens = walk.x.tokens;
        // Q as the second operand of the first product: column g of n-tile i is row 8 i + g.
        uint32_t q[NT][NG][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int r = v.r0 + 8 * i + g;
            const uint16_t* row =
                p.Q + ((static_cast<int64_t>(walk.x.q0) + r / p.g) * p.nq + walk.h * p.g + r % p.g) *
                          HD + 8 * c;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (8 * i + g < v.live) u = __ldg(reinterpret_cast<const uint4*>(row + 32 * G));
                q[i][G][0] = __byte_perm(u.x, u.z, 0x5410);  // elements 0, 4
                q[i][G][1] = __byte_perm(u.x, u.z, 0x7632);  // 1, 5
                q[i][G][2] = __byte_perm(u.y, u.w, 0x5410);  // 2, 6
                q[i][G][3] = __byte_perm(u.y, u.w, 0x7632);  // 3, 7
            }
        }
        // What a sum of products times scales is multiplied with, of rows 2 c and 2 c + 1.
        float factor[NT][2];
        float first[RAW ? NG : 1][4];  // what the sums begin with
        bool far = false;  // factors in two parts, the first in shared memory
        if constexpr (RAW) {
            // A row times 2^n, so that its largest element lies at 2^119: products with steps of
            // 2^-133 are then ordinary numbers.
            uint32_t most = 0;
#pragma unroll
            for (int G = 0; G < NG; ++G)
#pragma unroll
                for (int k = 0; k < 4; ++k) most = __vmaxu2(most, q[0][G][k] & 0x7FFF7FFFu);
            most = max(most & 0xFFFFu, most >> 16);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int n = 246 - max(static_cast<int>(most >> 7), 1);
            const int n1 = min(n, 120), n2 = n - n1;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q[0][G][k] = times2(times2(q[0][G][k], pow2(n1)),
                                        pow2(n2 - (k & 1 ? 4 : 0)));
                float d[4];
                mma(d, eight_k, q[0][G][0], q[0][G][1], zero);
                mma(first[G], eight_k, q[0][G][2], q[0][G][3], d);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 133 - __shfl_sync(0xffffffffu, n, 4 * (2 * c + e));
                factor[0][e] = p.c * pow2(min(m, 127)) * pow2(max(m - 127, 0));
                far |= isinf(factor[0][e]);
            }
            // A row that large (from 2^117 on, with the usual scale) times small keys may have scores
            // of ordinary size.  (|c| <= 2^101, so that neither part is past fp32.)
            far = __any_sync(0xffffffffu, far);
            if (far) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = 133 - __shfl_sync(0xffffffffu, n, 4 * (2 * c + e));
                    factor[0][e] = pow2(max(m - 26, 0));
                    if (g == 0) ctl.rest[warp][2 * c + e] = p.c * pow2(min(m, 26));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    q[i][G][1] = times2(q[i][G][1], 0.0625f);  // (as codes_of has them)
                    q[i][G][3] = times2(q[i][G][3], 0.0625f);
                }
                factor[i][0] = factor[i][1] = p.c * 64.0f;
            }
        }
        const int open_end = min(v.at0, tokens - 1) - 15;  // the last open tile's position
        const int window_end = v.at1 - p.window;
        int at[NT][2];  // positions of rows 8 i + 2 c and the next
        // What is taken from a row's scores (0 before there is a maximum), and the score that moves it:
        // 8 above the maximum when it was last looked at, so that no weight is above 1 and its product
        // with a scale is never past the scale.
        float base[NT][2], limit[NT][2];
        float l[NT][2], o[NT][HD / 16][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c + e;
                at[i][e] = r < v.live ? walk.x.ctx + (v.r0 + r) / p.g : -1;
                base[i][e] = 0.0f;
                limit[i][e] = -INFINITY;
                l[i][e] = 0.0f;
            }
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][d][e] = 0.0f;
        }
        // A slot's tiles, at positions p0[]; OPEN: every row sees all of them.
        auto step = [&](const uint8_t* slot_at, const int* p0, int have, auto open_tag) {
            constexpr bool OPEN = decltype(open_tag)::value;
            // Scores: token g and rows 2 c, 2 c + 1; token g + 8 and the same.
            float s[TT][NT][4];
#pragma unroll
            for (int u = 0; u < TT; ++u) {
                const uint8_t* tile = slot_at + u * T::kBytes;
                uint32_t k0[NG], k1[NG], ks0[NG / 2], ks1[NG / 2];
                load_words(k0, tile + g * (HD / 2) + c * 4 * NG);
                load_words(k1, tile + (g + 8) * (HD / 2) + c * 4 * NG);
                load_words(ks0, tile + key_scale<HD>(0, 0) + g * 2 * NG);
                load_words(ks1, tile + key_scale<HD>(8, 0) + g * 2 * NG);
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    uint32_t x0[4], x1[4];
                    if constexpr (RAW) {
                        raw_codes(x0, k0[G]);
                        raw_codes(x1, k1[G]);
                    } else {
                        codes_of(x0, k0[G]);
                        codes_of(x1, k1[G]);
                    }
                    const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]};
                    const uint32_t a1[4] = {x0[2], x1[2], x0[3], x1[3]};
                    const float f0 = scale_at(ks0, G), f1 = scale_at(ks1, G);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float d0[4], d[4];
                        if constexpr (RAW)
                            mma(d0, a0, q[i][G][0], q[i][G][1], first[G]);
                        else
                            mma(d0, a0, q[i][G][0], q[i][G][1], zero);
                        mma(d, a1, q[i][G][2], q[i][G][3], d0);
                        s[u][i][0] = G == 0 ? d[0] * f0 : fmaf(d[0], f0, s[u][i][0]);
                        s[u][i][1] = G == 0 ? d[1] * f0 : fmaf(d[1], f0, s[u][i][1]);
                        s[u][i][2] = G == 0 ? d[2] * f1 : fmaf(d[2], f1, s[u][i][2]);
                        s[u][i][3] = G == 0 ? d[3] * f1 : fmaf(d[3], f1, s[u][i][3]);
                    }
                }
            }
            if (RAW && far) {
                const float2 rest = *reinterpret_cast<const float2*>(&ctl.rest[warp][2 * c]);
#pragma unroll
                for (int u = 0; u < TT; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][0][e] *= e & 1 ? rest.y : rest.x;
            }
            // What a row does not see goes to -inf, and its weight below to a plain 0.
            uint32_t hidden = 0;  // bit 4 (NT u + i) + e: s[u][i][e]
            bool grow = false;
            float top[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int u = 0; u < TT; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[u][i][e] *= factor[i][e & 1];
                        if constexpr (!OPEN) {
                            const int pos = p0[u] + g + 8 * (e >> 1), own = at[i][e & 1];
                            const bool see = ((have >> u) & 1) && pos <= own && pos < tokens &&
                                             (pos < p.sinks || pos > own - p.window);
                            if (!see) {
                                s[u][i][e] = -INFINITY;
                                hidden |= 1u << (4 * (NT * u + i) + e);
                            }
                        }
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[i][e] = fmaxf(s[0][i][e], s[0][i][e + 2]);
                    if constexpr (TT == 2)
                        top[i][e] = fmaxf(top[i][e], fmaxf(s[TT - 1][i][e], s[TT - 1][i][e + 2]));
                    grow |= top[i][e] > limit[i][e];
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = top[i][e];
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1)
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, k));
                        // (the same for all lanes of the row; the limit is -inf before any score)
                        const bool none = limit[i][e] == -INFINITY;
                        if (t > (none ? -INFINITY : base[i][e] - kLazy)) {
                            const float shrink = none ? 0.0f : ex2(base[i][e] - (t + kLazy));
                            l[i][e] *= shrink;
#pragma unroll
                            for (int d = 0; d < HD / 16; ++d) {
                                o[i][d][e] *= shrink;
                                o[i][d][e + 2] *= shrink;
                            }
                            base[i][e] = limit[i][e] = t + kLazy;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < TT; ++u) {
                const uint8_t* tile = slot_at + u * T::kBytes;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[u][i][e] = ex2(s[u][i][e] - base[i][e & 1]);
                        l[i][e & 1] += s[u][i][e];
                    }
                uint32_t vs0[NG / 2], vs1[NG / 2];
                load_words(vs0, tile + value_scale<HD>(0, 0) + g * 2 * NG);
                load_words(vs1, tile + value_scale<HD>(8, 0) + g * 2 * NG);
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    // A group's weights: the token's weight by its scale, rounded to bf16 because
                    // both operands of a product have one type (an output is off by up to
                    // 2^-8 sum p |v| for it), rows over tokens turned to tokens over rows.
                    const float f0 = scale_at(vs0, G), f1 = scale_at(vs1, G);
                    uint32_t b[NT][2];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float y[4] = {s[u][i][0] * f0, s[u][i][1] * f0, s[u][i][2] * f1,
                                      s[u][i][3] * f1};
                        if constexpr (!OPEN) {  // (a hidden token's scale may be anything)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((hidden >> (4 * (NT * u + i) + e)) & 1) y[e] = 0.0f;
                        }
                        b[i][0] = transpose8x8(pack_bf16x2(y[0], y[1]));
                        b[i][1] = transpose8x8(pack_bf16x2(y[2], y[3]));
                    }
                    // elements 32 G .. + 31: two products' rows, two words of the lane's four
                    const uint2 w = *reinterpret_cast<const uint2*>(
                        tile + T::kCodes + (G / 2 * 32 + lane) * 16 + G % 2 * 8);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[4];
                        codes_of(a, h ? w.y : w.x);
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            mma(o[i][2 * G + h], a, b[i][0], b[i][1], o[i][2 * G + h]);
                    }
                }
            }
        };
        // Steps from open0 on, up to open1, are seen whole by every row: tiles behind the sinks'
        // whose tokens come after the last row's window begins and not after the first row.
        const int open0 = max(sinks, window_end < 0 ? 0 : window_end / 16 + 1 - w0) - k_first;
        const int open1 = min((open_end < 0 ? 0 : open_end / 16 + 1) - w0 - k_first, tiles) - TT + 1;
        for (int j = TT * warp; j < tiles; j += TT * W) {
            cp_async_wait_group<S::kSlots - 1>();
            __syncwarp();  // every lane's copies are there
            const uint8_t* slot_at = ring + slot * S::kSlotBytes;
            const int have = static_cast<int>(there >> (TT * slot)) & ((1 << TT) - 1);
            int p0[TT];
            if (j >= open0 && j < open1 && have == (1 << TT) - 1) {
                step(slot_at, p0, have, std::true_type{});
            } else if (have != 0) {
#pragma unroll
                for (int u = 0; u < TT; ++u) {
                    const int k = k_first + j + u;
                    p0[u] = (k < sinks ? k : w0 + k) * 16;
                }
                step(slot_at, p0, have, std::false_type{});
            }
            __syncwarp();  // the slot has been read
            issue();
            slot = slot + 1 == S::kSlots ? 0 : slot + 1;
        }

        // ---- the piece's end: the warps put together what they have
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 4; k < 32; k <<= 1)
                    l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], k);
        if (pieces > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.merged, (pieces - 1) & 1)) != 0;
            if (!ok) break;
        }
        float* mine = sh_o + warp * R * S::kOStride;
        const bool some = walk.n > TT * warp;  // else O is not looked at
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c + e;
                if (g == 0) sh_ml[warp * R + r] = make_float2(base[i][e], l[i][e]);
                if (some && r < v.live) {
#pragma unroll
                    for (int d = 0; d < HD / 16; ++d) {
                        // (codes_of divides by 64 and 4)
                        mine[r * S::kOStride + 16 * d + g] =
                            o[i][d][e] * 64.0f;
                        mine[r * S::kOStride + 16 * d + g + 8] =
                            o[i][d][e + 2] * 4.0f;
                    }
                }
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.arrived);
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.arrived, pieces & 1)) != 0;
        if (!ok) break;
        const int64_t part = 2 * blockIdx.x + (walk.k > 0 ? 0 : 1);
        for (int r = warp; r < v.live; r += W) {
            float top = -INFINITY, sum = 0.0f;
            for (int w = 0; w < W; ++w) {
                const float2 ml = sh_ml[w * R + r];
                if (ml.y != 0.0f) top = fmaxf(top, ml.x);
            }
            const float top_or_0 = top == -INFINITY ? 0.0f : top;
            float2 acc[HD / 64];
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
            for (int w = 0; w < W; ++w) {
                const float2 ml = sh_ml[w * R + r];
                if (ml.y == 0.0f) continue;
                const float wt = ex2(ml.x - top_or_0);
                sum = fmaf(wt, ml.y, sum);
                const float* from = sh_o + (w * R + r) * S::kOStride;
#pragma unroll
                for (int i = 0; i < HD / 64; ++i) {
                    const float2 y = *reinterpret_cast<const float2*>(from + 2 * lane + 64 * i);
                    acc[i].x = fmaf(wt, y.x, acc[i].x);
                    acc[i].y = fmaf(wt, y.y, acc[i].y);
                }
            }
            if (walk.whole) {
                write_row<HD>(p, walk.x.q0, v.r0 + r, walk.h, top_or_0, sum, acc);
            } else {
                float* to = p.part_o + (part * R + r) * HD;
#pragma unroll
                for (int i = 0; i < HD / 64; ++i)
                    *reinterpret_cast<float2*>(to + 2 * lane + 64 * i) = acc[i];
                if (lane == 0) p.part_ml[part * R + r] = make_float2(top, sum);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.merged);
        ++pieces;
    }
    if (!ok) {
        if (lane == 0 && *abort_flag == 0)
            raise_error(p.dev_status, p.lib_error, HSS_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    }
    cp_async_wait_group<0>();  // nobody leaves before its copies have landed
    __syncthreads();
}

// Joins the pieces of the units that were cut: CTA (x, y) looks at the cut before range x + 1, takes
// the unit there if this is its first cut, and of it every gridDim.y-th ROWS rows.  A long sequence is
// cut into as many pieces as there are ranges to share it, so what costs is the way of their loads: a warp a
// row finds the pieces' weights, while four elements of a row to a thread and a share of the pieces
// are on their way already, a dozen pieces at a time.
constexpr int kJoinThreads = 512;
constexpr int kJoinPieces = 128;

template <int HD, int R, int UNIT>
__device__ __forceinline__ void join_pieces(const Params& p) {
    constexpr int V = HD / 4, kAtOnce = 12;
    // Few rows: eight, and many pieces.  Many rows: as many as there are threads for, few pieces.
    constexpr int ROWS = R <= 16 ? 8 : kJoinThreads / V;
    constexpr int kWarpRows = (ROWS + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
    __shared__ float weight[ROWS][kJoinPieces];
    __shared__ float shrink[ROWS], top_of[ROWS], sum_of[ROWS];
    __shared__ float4 parts[kJoinThreads];
    const int range = blockIdx.x + 1;
    const Start st = p.starts[range];
    // (no cut, or behind the tiles, or in a unit that is not cut)
    if (st.t == 0 || st.t >= st.cost || st.cost <= kUncut<UNIT>) return;
    const int64_t f = range * st.per - st.t;  // the unit's first tile
    if (divide(f, st.per) != range - 1) return;
    const int count = static_cast<int>(divide(f + st.cost - 1, st.per)) - range + 2;
    for (int r0 = ROWS * blockIdx.y; r0 < st.live; r0 += ROWS * gridDim.y) {
        const int rows = min(st.live - r0, ROWS);
        // piece 0 is the end of range - 1, piece k the beginning of range + k - 1
        auto part = [&](int k, int r) -> int64_t {
            return (k == 0 ? 2 * (range - 1) + 1 : 2 * (range + k - 1)) * static_cast<int64_t>(R) +
                   r0 + r;
        };
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int shares = kJoinThreads / (rows * V);
        const int share = threadIdx.x / (rows * V), at = threadIdx.x % (rows * V);
        const int row = at / V, col = at % V * 4;
        float4 v[kAtOnce], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto fetch = [&](int k0, int end) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int k = k0 + i * shares;
                if (share < shares && k < end)
                    v[i] = *reinterpret_cast<const float4*>(p.part_o + part(k, row) * HD + col);
            }
        };
        float top[kWarpRows], sum[kWarpRows];  // of the warp's rows
#pragma unroll
        for (int n = 0; n < kWarpRows; ++n) {
            top[n] = -INFINITY;
            sum[n] = 0.0f;
        }
        for (int c0 = 0; c0 < count; c0 += kJoinPieces) {
            const int end = min(count, c0 + kJoinPieces);
            fetch(c0 + share, end);
#pragma unroll
            for (int n = 0; n < kWarpRows; ++n) {
                const int r = warp + n * (kJoinThreads / 32);
                if (r >= rows) break;
                float2 ml[kJoinPieces / 32];
                float most = top[n];
#pragma unroll
                for (int i = 0; i < kJoinPieces / 32; ++i) {
                    const int k = c0 + 32 * i + lane;
                    ml[i] = k < end ? p.part_ml[part(k, r)] : make_float2(0.0f, 0.0f);
                    if (ml[i].y != 0.0f) most = fmaxf(most, ml[i].x);
                }
#pragma unroll
                for (int m = 1; m < 32; m <<= 1)
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
                const float base = most == -INFINITY ? 0.0f : most;
                const float less = top[n] == -INFINITY ? 0.0f : ex2(top[n] - base);
                float here = 0.0f;
#pragma unroll
                for (int i = 0; i < kJoinPieces / 32; ++i) {
                    const float w = ml[i].y != 0.0f ? ex2(ml[i].x - base) : 0.0f;
                    if (ml[i].y != 0.0f) here = fmaf(w, ml[i].y, here);
                    weight[r][32 * i + lane] = w;
                }
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) here += __shfl_xor_sync(0xffffffffu, here, m);
                sum[n] = fmaf(sum[n], less, here);
                top[n] = most;
                if (lane == 0) {
                    shrink[r] = less;
                    top_of[r] = base;
                    sum_of[r] = sum[n];
                }
            }
            __syncthreads();
            if (share < shares) {
                const float less = shrink[row];
                acc.x *= less, acc.y *= less, acc.z *= less, acc.w *= less;
                for (int k0 = c0 + share; k0 < end; k0 += kAtOnce * shares) {
                    if (k0 != c0 + share) fetch(k0, end);
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const int k = k0 + i * shares;
                        if (k >= end) break;
                        const float w = weight[row][k - c0];
                        if (w == 0.0f) continue;  // (without weight O may be anything)
                        acc.x = fmaf(w, v[i].x, acc.x);
                        acc.y = fmaf(w, v[i].y, acc.y);
                        acc.z = fmaf(w, v[i].z, acc.z);
                        acc.w = fmaf(w, v[i].w, acc.w);
                    }
                }
            }
            __syncthreads();
        }
        parts[threadIdx.x] = acc;
        __syncthreads();
        if (share == 0) {
            for (int k = 1; k < shares; ++k) {
                const float4 o = parts[threadIdx.x + k * rows * V];
                acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
            }
            const float l = sum_of[row], inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int r = st.r0 + r0 + row;
            const int64_t to = (static_cast<int64_t>(st.q0) + r / p.g) * p.nq + st.h * p.g + r % p.g;
            uint2 u = make_uint2(0, 0);
            if (l != 0.0f)
                u = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                               pack_bf16x2(acc.z * inv, acc.w * inv));
            *reinterpret_cast<uint2*>(p.out + to * HD + col) = u;
            if (col == 0 && p.lse != nullptr)
                p.lse[to] = l == 0.0f ? -INFINITY : (top_of[row] + log2f(l)) * 0.693147180559945309f;
        }
        __syncthreads();  // (what the next rows write has been read)
    }
}

template <int HD, int R>
__global__ void __launch_bounds__(kJoinThreads, 1) join_kernel(const Params p) {
    grid_dependency_wait();
    grid_launch_dependents();
    join_pieces<HD, R, 1>(p);
}

// The most tiles that a unit can have, as far as the host can tell.
inline int64_t tiles_bound(const Params& p) {
    const int64_t tiles = (p.total_blocks * p.bs + 15) / 16;
    if (p.window >= kNoWindow) return tiles;
    return std::min<int64_t>(tiles,
                             (static_cast<int64_t>(p.window) + p.sinks + p.max_q) / 16 + 4);
}
inline int64_t row_tiles_bound(const Params& p, int rows) {
    return (static_cast<int64_t>(p.max_q) * p.g + rows - 1) / rows;
}

// The attention of few rows without its join, which *joined says is needed.
template <int HD, int NT>
hss_status launch_few(const Params& args, bool* joined, cudaStream_t stream) {
    using S = Shape<HD, NT>;
    auto kern = attend_kernel<HD, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes) !=
        cudaSuccess)
        return HSS_ERR_CUDA;
    Params p = args;
    const int64_t row_tiles = row_tiles_bound(p, S::kRows);
    const int64_t units = p.num_seqs * row_tiles * p.nkv;
    *joined = !by_units(tiles_bound(p), units);
    p.row_tiles = *joined ? 0 : static_cast<int32_t>(row_tiles);
    const dim3 grid(*joined ? S::kRanges : static_cast<unsigned>(units));
    return launch_pdl(kern, grid, dim3(S::kThreads), S::kSmemBytes, stream, p) == cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

template <int HD, int NT>
hss_status launch_rows(const Params& p, cudaStream_t stream) {
    bool joined;
    const hss_status st = launch_few<HD, NT>(p, &joined, stream);
    if (st != HSS_OK || !joined) return st;
    return launch_pdl(join_kernel<HD, 8 * NT>, dim3(Shape<HD, NT>::kRanges - 1, NT),
                      dim3(kJoinThreads), 0, stream, p) == cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

// Of each head_dim's unit.  With `many` the kernel for many rows comes first (attend_packed_tc.cuh),
// and p, for few, is guarded by the flags that it writes.
template <int HD>
hss_status launch_head_dim(const Params& p, const Params* many, int n_tiles, int32_t* flags,
                           cudaStream_t stream);

}  // namespace packed
}  // namespace hss
