// attend_packed.cuh -- attention of few rows over the packed cache: one pass over 4-bit tiles with
// warp-level matrix products.
//
// A row is a (query row, query head of the group) pair; the rows of one sequence that share a kv
// head are taken R = 8 NT at a time.  Over the tokens they see, in tiles of 16,
//   S^T = K Q^T,  P = exp2(c S - m),  O^T = V^T P^T,  l = sum P
// with mma.m16n8k16: tokens (of V^T: elements) are the 16 rows of the product and query rows its 8
// columns, so that K and V, which are what there is much of, are the operand that goes from packed
// words straight into registers, and eight query rows fill an instruction.  Four bits become bf16
// by placing a nibble under the exponent of 128 and subtracting 136, exactly.  A group's scale
// multiplies what the group adds to S, and for V the weight of its token: P is scaled, rounded to
// bf16 and transposed (movmatrix) once for each group of 32 elements.
//
// The maximum m lags: it is one for the whole warp and a row, and moves only when a score passes it
// by 2^8, so that a tile costs a vote and no shuffles.
//
// Split.  All (sequence, row tile, kv head, tile) form one list, cut into equal contiguous ranges, a
// CTA each.  Within a CTA the warps take the tiles of a unit (sequence, row tile, head) in turn,
// each with a ring of its own that bulk copies fill (a tile is contiguous), and put m, l and O
// together in shared memory at the unit's end or the range's.  What a range does not have whole
// goes to the workspace and a second kernel joins it.
#pragma once

#include "packed.cuh"

namespace hss {
namespace packed {

constexpr int kGrid = 152;         // GB300's SMs; the workspace does not depend on the device
constexpr float kLazy = 8.0f;

struct Start {
    int64_t total, per;  // the list's length, of a range
    int64_t t, cost;     // where the CTA's range begins in a unit, and the unit's length
    int32_t s, rt, h, pad;
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
    int32_t window;  // 0x7FFFFFFF: none
    int32_t sinks;   // 0 without a window
    float c;         // scale log2(e)
    int32_t* dev_status;
    int32_t* lib_error;
    // workspace
    Start* starts;    // [kGrid]
    float2* part_ml;  // [2 kGrid][R] (m, l)
    float* part_o;    // [2 kGrid][R][head_dim]
};

template <int HD, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kOStride = HD + 4;  // floats of a row of O in shared memory
    static constexpr int kOBytes = kWarps * kRows * kOStride * 4;
    static constexpr int kMlBytes = kWarps * kRows * 8;
    static constexpr int kTileBytes = Tile<HD>::kBytes;
    static constexpr int kBudget = 232448 - 1024 - 2048 - kOBytes - kMlBytes;
    static constexpr int kFits = kBudget / (kWarps * kTileBytes);
    static constexpr int kSlots = kFits < 16 ? kFits : 16;  // of a warp's ring
    static constexpr int kSmemBytes =
        1024 + 2048 + kOBytes + kMlBytes + kWarps * kSlots * kTileBytes;
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

// What a row tile sees: tiles [0, sinks) and [w0, end).
struct View {
    int r0, live;        // its first row (of the sequence and kv head) and how many there are
    int at0, at1;        // positions of its first and last row
    int sinks, w0, end;  // tiles
    __device__ __forceinline__ int tiles() const { return sinks + end - w0; }
    // (a row tile that sees nothing still has its result to write)
    __device__ __forceinline__ int cost() const { return max(tiles(), 1); }
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

// The pieces of a CTA's range, one unit (or the range's part of it) after another.
template <int R>
struct Walk {
    SeqInfo x;
    View v;
    int s, rt, rts, h;
    int k, n;  // the piece: tiles [k, k + n) of the unit's view
    bool whole;
    int64_t f, f1;
    int t;

    __device__ __forceinline__ void begin(const Params& p, const Start& st) {
        f = min(st.total, blockIdx.x * st.per);
        f1 = min(st.total, f + st.per);
        s = st.s;
        rt = st.rt;
        h = st.h;
        t = static_cast<int>(st.t);
        if (f < f1) {
            x = load_seq(p, s);
            rts = row_tiles<R>(p, x);
            v = view_of<R>(p, x, rt);
        }
    }
    __device__ __forceinline__ bool next(const Params& p) {
        if (f >= f1) return false;
        // (t is past the unit's end only after a piece)
        while (t >= v.cost()) {
            t = 0;
            if (++h < p.nkv) break;
            h = 0;
            if (++rt >= rts) {
                rt = 0;
                do {
                    if (++s >= p.num_seqs) {
                        f = f1;
                        return false;
                    }
                    x = load_seq(p, s);
                    rts = row_tiles<R>(p, x);
                } while (rts == 0);
            }
            v = view_of<R>(p, x, rt);
        }
        const int take = static_cast<int>(min(static_cast<int64_t>(v.cost() - t), f1 - f));
        k = t;
        n = max(min(t + take, v.tiles()) - t, 0);
        whole = take == v.cost();
        t += take;
        f += take;
        return true;
    }
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Nibbles j and j + 4 of a word, less 8, as two bf16.
__device__ __forceinline__ uint32_t two_codes(uint32_t w, int j) {
    const uint32_t u = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;  // 128 + nibble
    const uint32_t k136 = 0x43084308u;
    __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                               *reinterpret_cast<const __nv_bfloat162*>(&k136));
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
    uint64_t full[8 * 16];     // [warp][slot]
    uint64_t arrived, merged;  // the warps' parts of a piece are there; are joined
    int bad[8 * 16];           // [warp][slot] the tile's block id is out of range
    int abort;
    Start start;
    int64_t scan[8];
};
static_assert(sizeof(Control) <= 2048, "control block");

// Where every CTA's range begins, from a scan of the sequences' lengths.
template <int R, int THREADS>
__device__ __forceinline__ void find_start(const Params& p, Control& ctl, int64_t least) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int each = (p.num_seqs + THREADS - 1) / THREADS;
    const int s0 = min(static_cast<int>(threadIdx.x) * each, p.num_seqs);
    const int s1 = min(s0 + each, p.num_seqs);
    auto length = [&](const SeqInfo& x) -> int64_t {
        const int n = row_tiles<R>(p, x);
        int64_t sum = 0;
        for (int rt = 0; rt < n; ++rt) sum += view_of<R>(p, x, rt).cost();
        return sum * p.nkv;
    };
    int64_t mine = 0;
    SeqInfo x;  // (with one sequence a thread, still there for the second look)
    for (int s = s0; s < s1; ++s) {
        x = load_seq(p, s);
        mine += length(x);
        if (blockIdx.x == 0) {
            if (__ldg(p.q_offsets + s + 1) - x.q0 > p.max_q)
                raise_error(p.dev_status, p.lib_error, HSS_ERR_INVALID_ARGUMENT);
            if (x.cut && x.rows > 0) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
        }
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
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, least);
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
            int64_t cost = view_of<R>(p, x, 0).cost();
            while (o >= cost * p.nkv) {
                o -= cost * p.nkv;
                cost = view_of<R>(p, x, ++rt).cost();
            }
            ctl.start.s = s;
            ctl.start.rt = rt;
            ctl.start.h = static_cast<int>(o / cost);
            ctl.start.t = o % cost;
            ctl.start.cost = cost;
        }
        before += n;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.starts[blockIdx.x] = ctl.start;
}

// A finished row: out and lse.
template <int HD>
__device__ __forceinline__ void write_row(const Params& p, const SeqInfo& x, int r, int h, float m,
                                          float l, const float2 (&acc)[HD / 64]) {
    const int lane = threadIdx.x & 31;
    const int64_t at = (static_cast<int64_t>(x.q0) + r / p.g) * p.nq + h * p.g + r % p.g;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t* to = reinterpret_cast<uint32_t*>(p.out + at * HD);
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
        to[lane + 32 * i] = l == 0.0f ? 0u : pack_bf16x2(acc[i].x * inv, acc[i].y * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

template <int HD, int NT>
__global__ void __launch_bounds__(Shape<HD, NT>::kThreads, 1) attend_kernel(const Params p) {
    using S = Shape<HD, NT>;
    using T = Tile<HD>;
    constexpr int R = S::kRows, W = S::kWarps, NG = T::kGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    Control& ctl = *reinterpret_cast<Control*>(smem);
    float* sh_o = reinterpret_cast<float*>(smem + 2048);  // [W][R][kOStride]
    float2* sh_ml = reinterpret_cast<float2*>(smem + 2048 + S::kOBytes);  // [W][R]
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + 2048 + S::kOBytes + S::kMlBytes + warp * S::kSlots * S::kTileBytes;
    uint64_t* full = ctl.full + warp * 16;
    int* bad = ctl.bad + warp * 16;

    if (threadIdx.x == 0) {
        for (int i = 0; i < W; ++i)
            for (int k = 0; k < S::kSlots; ++k) mbar_init(&ctl.full[i * 16 + k], 1);
        mbar_init(&ctl.arrived, W);
        mbar_init(&ctl.merged, W);
        ctl.abort = 0;
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    find_start<R, S::kThreads>(p, ctl, W);
    volatile int* abort_flag = &ctl.abort;

    // ---- the copies, a ring ahead of the products
    Walk<R> ahead;
    ahead.begin(p, ctl.start);
    bool more = ahead.next(p);
    int ahead_j = 0;        // the warp's tiles of the piece: warp, warp + W, ...
    uint32_t issued = 0;
    int ids = 0;            // lane i: the block of tile 32 b + i of them
    auto issue = [&]() {
        while (more && warp + ahead_j * W >= ahead.n) {
            more = ahead.next(p);
            ahead_j = 0;
        }
        if (!more) return;
        if (ahead_j % 32 == 0) {
            const int k = warp + (ahead_j + lane) * W;
            if (k < ahead.n)
                ids = __ldg(p.table + ahead.x.e0 + ahead.v.tile(ahead.k + k) * 16 / p.bs);
        }
        const int id = __shfl_sync(0xffffffffu, ids, ahead_j % 32);
        if (lane == 0) {
            const int slot = static_cast<int>(issued % S::kSlots);
            const bool good = id >= 0 && id < p.max_blocks;
            bad[slot] = !good;
            if (good) {
                const int pos = ahead.v.tile(ahead.k + warp + ahead_j * W) * 16;
                const int64_t at = (static_cast<int64_t>(id) * p.nkv + ahead.h) * (p.bs / 16) +
                                   pos % p.bs / 16;
                mbar_arrive_expect_tx(&full[slot], T::kBytes);
                bulk_copy_g2s(ring + slot * T::kBytes, p.cache + at * T::kBytes, T::kBytes,
                              &full[slot]);
            } else {
                raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
                mbar_arrive(&full[slot]);
            }
        }
        ++issued;
        ++ahead_j;
    };
    for (int i = 0; i < S::kSlots; ++i) issue();

    // ---- the products
    Walk<R> walk;
    walk.begin(p, ctl.start);
    uint32_t used = 0, pieces = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
        const View& v = walk.v;
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
        int at[NT][2];  // positions of rows 8 i + 2 c and the next
        float m[NT][2], l[NT][2], o[NT][HD / 16][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c + e;
                at[i][e] = r < v.live ? walk.x.ctx + (v.r0 + r) / p.g : -1;
                m[i][e] = -INFINITY;
                l[i][e] = 0.0f;
            }
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][d][e] = 0.0f;
        }
        for (int j = warp; j < walk.n; j += W) {
            const int slot = static_cast<int>(used % S::kSlots);
            ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], (used / S::kSlots) & 1)) != 0;
            if (!ok) break;
            ++used;
            const uint8_t* tile = ring + slot * T::kBytes;
            const int p0 = v.tile(walk.k + j) * 16;
            if (*(volatile int*)&bad[slot] == 0) {
                uint32_t k0[NG], k1[NG], ks0[NG / 2], ks1[NG / 2];
                load_words(k0, tile + g * (HD / 2) + c * 4 * NG);
                load_words(k1, tile + (g + 8) * (HD / 2) + c * 4 * NG);
                load_words(ks0, tile + key_scale<HD>(0, 0) + g * 2 * NG);
                load_words(ks1, tile + key_scale<HD>(8, 0) + g * 2 * NG);
                // Scores: token g and rows 2 c, 2 c + 1; token g + 8 and the same.
                float s[NT][4];
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    const uint32_t a0[4] = {two_codes(k0[G], 0), two_codes(k1[G], 0),
                                            two_codes(k0[G], 1), two_codes(k1[G], 1)};
                    const uint32_t a1[4] = {two_codes(k0[G], 2), two_codes(k1[G], 2),
                                            two_codes(k0[G], 3), two_codes(k1[G], 3)};
                    const float x0 = scale_at(ks0, G) * p.c, x1 = scale_at(ks1, G) * p.c;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma(d, a0, q[i][G][0], q[i][G][1]);
                        mma(d, a1, q[i][G][2], q[i][G][3]);
                        s[i][0] = G == 0 ? d[0] * x0 : fmaf(d[0], x0, s[i][0]);
                        s[i][1] = G == 0 ? d[1] * x0 : fmaf(d[1], x0, s[i][1]);
                        s[i][2] = G == 0 ? d[2] * x1 : fmaf(d[2], x1, s[i][2]);
                        s[i][3] = G == 0 ? d[3] * x1 : fmaf(d[3], x1, s[i][3]);
                    }
                }
                // What a row does not see goes to -inf, and its weight below to a plain 0.
                const bool open = p0 + 15 <= v.at0 && p0 + 15 < walk.x.tokens &&
                                  (p0 + 15 < p.sinks || p0 > v.at1 - p.window);
                uint32_t hidden = 0;  // bit 4 i + e: s[i][e]
                if (!open) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int pos = p0 + g + 8 * (e >> 1), own = at[i][e & 1];
                            const bool see = pos <= own && pos < walk.x.tokens &&
                                             (pos < p.sinks || pos > own - p.window);
                            if (!see) {
                                s[i][e] = -INFINITY;
                                hidden |= 1u << (4 * i + e);
                            }
                        }
                }
                bool grow = false;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        grow |= fmaxf(s[i][e], s[i][e + 2]) > m[i][e] + kLazy;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(s[i][e], s[i][e + 2]);
#pragma unroll
                            for (int k = 4; k < 32; k <<= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                            if (top > m[i][e]) {  // (the same for all lanes of the row)
                                const float shrink = ex2(m[i][e] - top);
                                l[i][e] *= shrink;
#pragma unroll
                                for (int d = 0; d < HD / 16; ++d) {
                                    o[i][d][e] *= shrink;
                                    o[i][d][e + 2] *= shrink;
                                }
                                m[i][e] = top;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float base = m[i][e & 1] == -INFINITY ? 0.0f : m[i][e & 1];
                        s[i][e] = ex2(s[i][e] - base);
                        l[i][e & 1] += s[i][e];
                    }
                uint32_t vs0[NG / 2], vs1[NG / 2];
                load_words(vs0, tile + value_scale<HD>(0, 0) + g * 2 * NG);
                load_words(vs1, tile + value_scale<HD>(8, 0) + g * 2 * NG);
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    // A group's weights: the token's weight by its scale, rounded to bf16 because
                    // both operands of a product have one type (an output is off by up to
                    // 2^-9 sum p |v| for it), rows over tokens turned to tokens over rows.
                    const float x0 = scale_at(vs0, G), x1 = scale_at(vs1, G);
                    uint32_t b[NT][2];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float y[4] = {s[i][0] * x0, s[i][1] * x0, s[i][2] * x1, s[i][3] * x1};
                        if (!open) {  // (a hidden token's scale may be anything)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((hidden >> (4 * i + e)) & 1) y[e] = 0.0f;
                        }
                        b[i][0] = transpose8x8(pack_bf16x2(y[0], y[1]));
                        b[i][1] = transpose8x8(pack_bf16x2(y[2], y[3]));
                    }
                    // elements 32 G .. + 31: two products' rows, two words of the lane's four
                    const uint2 w = *reinterpret_cast<const uint2*>(
                        tile + T::kCodes + (G / 2 * 32 + lane) * 16 + G % 2 * 8);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t word = h ? w.y : w.x;
                        const uint32_t a[4] = {two_codes(word, 0), two_codes(word, 1),
                                               two_codes(word, 2), two_codes(word, 3)};
#pragma unroll
                        for (int i = 0; i < NT; ++i) mma(o[i][2 * G + h], a, b[i][0], b[i][1]);
                    }
                }
            }
            __syncwarp();  // the slot has been read
            issue();
        }
        if (!ok) break;

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
        const bool some = walk.n > warp;  // else O is not looked at
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c + e;
                if (g == 0) sh_ml[warp * R + r] = make_float2(m[i][e], l[i][e]);
                if (some && r < v.live) {
#pragma unroll
                    for (int d = 0; d < HD / 16; ++d) {
                        mine[r * S::kOStride + 16 * d + g] = o[i][d][e];
                        mine[r * S::kOStride + 16 * d + g + 8] = o[i][d][e + 2];
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
            const float base = top == -INFINITY ? 0.0f : top;
            float2 acc[HD / 64];
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
            for (int w = 0; w < W; ++w) {
                const float2 ml = sh_ml[w * R + r];
                if (ml.y == 0.0f) continue;
                const float wt = ex2(ml.x - base);
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
                write_row<HD>(p, walk.x, v.r0 + r, walk.h, base, sum, acc);
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
    // Nobody leaves before its copies have landed.
    for (; used < issued; ++used)
        (void)mbar_wait_for(&full[used % S::kSlots], (used / S::kSlots) & 1, 1000000);
    __syncthreads();
}

// Joins the pieces of the units that were cut: CTA x looks at the cut before range x + 1, and takes
// the unit there if this is its first cut.  A warp takes a row.
template <int HD, int NT>
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
    constexpr int R = 8 * NT;
    grid_dependency_wait();
    grid_launch_dependents();
    const int range = blockIdx.x + 1;
    const Start st = p.starts[range];
    if (st.t == 0) return;
    const int64_t f = range * st.per - st.t;  // the unit's first tile
    if (f / st.per != range - 1) return;
    const int last = static_cast<int>((f + st.cost - 1) / st.per);
    const int count = last - range + 2;
    const SeqInfo x = load_seq(p, st.s);
    const View v = view_of<R>(p, x, st.rt);
    const int lane = threadIdx.x & 31;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (r >= v.live) return;
    // piece 0 is the end of range - 1, piece k the beginning of range + k - 1
    auto part = [&](int k) -> int64_t {
        return (k == 0 ? 2 * (range - 1) + 1 : 2 * (range + k - 1)) * static_cast<int64_t>(R) + r;
    };
    float top = -INFINITY;
    for (int k = lane; k < count; k += 32) {
        const float2 ml = p.part_ml[part(k)];
        if (ml.y != 0.0f) top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    float2 acc[HD / 64];
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
        const float2 ml = p.part_ml[part(k)];
        const float wt = ml.y != 0.0f ? ex2(ml.x - base) : 0.0f;
        const float* from = p.part_o + part(k) * HD;
        float2 y[HD / 64];
#pragma unroll
        for (int i = 0; i < HD / 64; ++i)
            y[i] = *reinterpret_cast<const float2*>(from + 2 * lane + 64 * i);
        if (ml.y == 0.0f) continue;
        sum = fmaf(wt, ml.y, sum);
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            acc[i].x = fmaf(wt, y[i].x, acc[i].x);
            acc[i].y = fmaf(wt, y[i].y, acc[i].y);
        }
    }
    write_row<HD>(p, x, v.r0 + r, st.h, base, sum, acc);
}

template <int HD, int NT>
hss_status launch_rows(const Params& p, cudaStream_t stream) {
    using S = Shape<HD, NT>;
    auto kern = attend_kernel<HD, NT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes) !=
        cudaSuccess)
        return HSS_ERR_CUDA;
    if (launch_pdl(kern, dim3(kGrid), dim3(S::kThreads), S::kSmemBytes, stream, p) != cudaSuccess)
        return HSS_ERR_CUDA;
    if (launch_pdl(join_kernel<HD, NT>, dim3(kGrid - 1, NT), dim3(256), 0, stream, p) !=
        cudaSuccess)
        return HSS_ERR_CUDA;
    return HSS_OK;
}

// Of each head_dim's unit.
template <int HD>
hss_status launch_head_dim(const Params& p, int n_tiles, cudaStream_t stream);

}  // namespace packed
}  // namespace hss
