// attend_packed_tc.cuh -- attention of many rows over the packed cache, on tcgen05.
//
// Row tiles of 128 rows (one or two to a CTA) against jobs of 64 tokens:
//   S = Q K^T,  P = exp2(c S - m),  O = P V,  l = sum P
// with S and O in tensor memory, a row to a lane, P written back over S as the first operand of the
// second product.  Eight warps decode a job's packed tiles, once for both row tiles, into shared
// memory as the tensor cores read them:
//   - in fp16, where a bf16 scale (8 bits) times a code (3 bits) has a place for every bit, so that
//     K and V enter the products exactly.  Scales outside [2^-17, 2^6] (but for 0), or not finite,
//     do not fit: the call's flags then ask the kernel for few rows to do all of it (Params::guard),
//     as they do for queries whose scores may pass fp32;
//   - a 16-byte piece of K is one word's eight elements in the order 0 4 1 5 2 6 3 7, as they come
//     out of the nibbles' places, and Q is laid out the same;
//   - tokens lie in the order 2c, 2c + 1, 2c + 8, 2c + 9 (c = 0 .. 3) of a tile's 16, in which a
//     word of V holds them; the columns of S and P follow K's rows.  V is stored by element, tokens
//     side by side, so both operands are K-major.
// Q is scaled by a power of two for every row, weights by 2^7 (with the maximum's lag of 2^8 they
// reach 2^15), so that fp16's range serves both.  A weight is off by 2^-11 of itself in the product with
// V or, below 2^-21 of the largest, where fp16 has no full place for it, by 2^-32 of the largest; in l
// it is as it was.
//
// Roles (20 warps): 10 copies; 0-7 decode; 8, 9 issue the products of a row tile each; 12-19
// softmax, four to a row tile, with registers that the others hand over.  One row tile's exponentials
// run under the other's products.
//
// Split: as for few rows (attend_packed.cuh), the list counted in jobs.
//
// What bounds it, and what it reaches: shared memory.  A job of two row tiles reads Q (64 KB), K and V
// (64 KB for both) from it and writes 32 KB of decoded operands, 1300 cycles at 128 bytes a cycle,
// where the products alone take 1000 to 1250 and the exponentials 1000; it takes 2000.  512 rows of 64
// heads over 32768 tokens 511 us in a graph, 1.08 PFLOP/s, 56 % of what a large bf16 product reaches (over a bf16
// cache hss_attend_tree takes 209 us for half the context).  Steps there: four warps that copied and
// decoded 1310 us; eight that hand scales on by shuffles 825; a warp of its own for the copies 537
// (their issue, 64-bit addresses and divisions in it, had taken 1500 of a job's 3400 cycles); a join of
// 16 rows at a time 511.  Tried and not kept: waiting for a job's operands before its weights (554).
#pragma once

#include <cuda_fp16.h>

#include "attend_packed.cuh"

namespace hss {
namespace packed {

template <int HD>
struct Many {
    static constexpr int kThreads = 640;
    static constexpr int kGroups = HD <= 128 ? 2 : 1;  // row tiles: O takes HD columns for each
    static constexpr int kRows = 128 * kGroups;
    static constexpr int kStages = HD <= 128 ? 4 : (HD == 192 ? 3 : 2);  // jobs decoded ahead
    static constexpr int kRawSlots = HD == 256 ? 1 : (HD == 192 ? 2 : 3);
    static constexpr int kOperand = 64 * HD * 2;  // bytes of a job's K, and of its V
    static constexpr int kQBytes = kRows * HD * 2;
    static constexpr int kRawBytes = 4 * Tile<HD>::kBytes;
    static constexpr int kControl = 5120;
    static constexpr int kSmemBytes =
        1024 + kQBytes + 2 * kStages * kOperand + kRawSlots * kRawBytes + kControl;
    static constexpr int kOCols = kGroups * 128;  // where O begins in tensor memory
    static_assert(kOCols + kGroups * HD <= 512, "tensor memory");
    static_assert(kSmemBytes <= 232448, "shared memory");
};

struct ManyBarriers {
    uint64_t full[4], empty[4];
    uint64_t raw_full[3], raw_empty[3];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2];
    uint32_t have[3];    // [raw slot] tiles that are there
    uint32_t hidden[4];  // [stage] tiles that nobody sees: missing, or with a bad id
    uint32_t tmem;
    int abort, unfit;
};
static_assert(sizeof(ManyBarriers) <= 512, "barrier block");

__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ bool wait_bounded(uint64_t* b, uint32_t parity,
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

// Registers of a warpgroup: 256 threads at 72, 128 at 48 and 256 at 144 come to 61,440, what 640
// threads of 96 were launched with.
template <int N>
__device__ __forceinline__ void shrink_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void grow_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t half_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The codes of a word (nibbles j and j + 4 in y[j]) times scales that are given times 2^9, for j = 0
// and 2, and 2^5: low bits of an fp16 count in steps of 2^-24, so a nibble in the lowest eight needs
// no shift; times 2^15, less 8, it is a code times 2^-9 or 2^-5, and both operations are exact.
__device__ __forceinline__ void decode_word(uint32_t (&y)[4], uint32_t w, uint32_t lo9,
                                            uint32_t lo5, uint32_t hi9, uint32_t hi5) {
    const uint32_t t = w >> 8;
    y[0] = half_mul(half_fma(w & 0x000F000Fu, 0x78007800u, 0xA400A400u), lo9);
    y[1] = half_mul(half_fma(w & 0x00F000F0u, 0x78007800u, 0xB400B400u), lo5);
    y[2] = half_mul(half_fma(t & 0x000F000Fu, 0x78007800u, 0xA400A400u), hi9);
    y[3] = half_mul(half_fma(t & 0x00F000F0u, 0x78007800u, 0xB400B400u), hi5);
}

// 32 columns of this thread's TMEM lane and their maximum (usable after the wait).
__device__ __forceinline__ float load_scores(uint32_t taddr, uint32_t* v) {
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
__device__ __forceinline__ void hold(uint32_t* v) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i])::"memory");
}

template <int HD>
__global__ void __launch_bounds__(Many<HD>::kThreads, 1)
    many_kernel(const Params p, int32_t* flags) {
    using M = Many<HD>;
    using T = Tile<HD>;
    constexpr int R = M::kRows, NG = T::kGroups, NS = M::kStages, RD = M::kRawSlots;
    constexpr int kChunks = HD / 64;  // 128-byte columns of a row of Q or K
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;
    uint8_t* sKV = sQ + M::kQBytes;  // [stage] K, V
    uint8_t* raw = sKV + 2 * NS * M::kOperand;
    uint8_t* rest = raw + RD * M::kRawBytes;
    Control& ctl = *reinterpret_cast<Control*>(rest);
    ManyBarriers& bar = *reinterpret_cast<ManyBarriers*>(rest + 512);
    using MyWalk = Walk<R, 4>;
    static_assert(28 * sizeof(MyWalk) <= M::kControl - 1024, "walks");
    MyWalk* walks = reinterpret_cast<MyWalk*>(rest + 1024);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;

    if (warp == 8) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bar.full[i], 8);
            mbar_init(&bar.empty[i], M::kGroups);
        }
        for (int i = 0; i < RD; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], 8);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&bar.q_full[w], 4);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&bar.s_full[w][b], 1);
                mbar_init(&bar.p_full[w][b], 4);
                mbar_init(&bar.o_done[w][b], 1);
            }
        }
        bar.abort = 0;
        bar.unfit = 0;
        fence_mbarrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bar.tmem;
    grid_dependency_wait();
    grid_launch_dependents();
    if (p.row_tiles == 0) find_start<R, 4, M::kThreads>(p, ctl, 2);
    volatile int* abort_flag = &bar.abort;

    auto advance = [&](MyWalk& w) {
        __syncwarp();
        bool got = false;
        if (lane == 0) got = w.next(p);
        __syncwarp();
        return __shfl_sync(0xffffffffu, static_cast<int>(got), 0) != 0;
    };
    auto wait = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(b, parity, abort_flag)) != 0;
    };
    auto give_up = [&]() {
        if (lane == 0 && *abort_flag == 0)
            raise_error(p.dev_status, p.lib_error, HSS_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    };
    MyWalk& walk = walks[warp];
    if (lane == 0) {
        if (p.row_tiles == 0) {
            walk.begin(p, ctl.start, ctl.seq, ctl.view);
        } else {
            walk.begin_unit(p, blockIdx.x);
            if (warp == 0 && walk.h == 0 && walk.rt == 0) report(p, walk.s, walk.x);
        }
    }
    bool ok = true;

    if (warp < 8) {
        shrink_registers<72>();
        // ---------------------------------------------------------------- codes
        const int tid = threadIdx.x;
        bool unfit = false;
        int slot = 0;
        uint32_t raw_parity = 0, job = 0;
        // A bf16 scale times 2^9 in fp16, or 0 where nobody sees the token or it does not fit.
        auto fit = [&](uint16_t bits, bool seen) -> uint32_t {
            const float s = __uint_as_float(static_cast<uint32_t>(bits) << 16);
            const bool fits = s == 0.0f || (s >= 7.62939453125e-6f && s <= 64.0f);
            unfit |= seen && !fits;
            return half2_bits(seen && fits ? s * 512.0f : 0.0f, 0.0f);
        };
        // Where the thread's parts of a job go.  K: tile, token and quarter of its words; 16-byte
        // pieces of even and odd groups, two groups to a 128-byte column.
        const int ku = tid >> 6, kt = (tid >> 2) & 15, kc = tid & 3;
        const int k_row = 16 * ku + kt % 8 / 2 * 4 + kt % 2 + kt / 8 * 2;
        const uint32_t k_even = swizzled_offset(k_row, 16 * kc, 128);
        const uint32_t k_odd = swizzled_offset(k_row, 16 * (4 + kc), 128);
        const int vg = lane >> 2, vc = lane & 3;
        while (ok && advance(walk)) {
            const View& v = walk.v;
            const int n = walk.n, tokens = walk.x.tokens, at1 = v.at1;
            const int window_end = v.at0 - p.window;
            const int k_first = walk.k, sinks = v.sinks, w0 = v.w0 - v.sinks;
            auto seen = [&](int pos) {
                return pos <= at1 && pos < tokens && (pos < p.sinks || pos > window_end);
            };
            for (int k = 0; k < n; k += 4, ++job) {
                const int stage = static_cast<int>(job % NS);
                auto position = [&](int u) {
                    const int i = k_first + k + u;
                    return (i < sinks ? i : w0 + i) * 16;
                };
                if (!(ok = wait(&bar.raw_full[slot], raw_parity))) break;
                if (!(ok = wait(&bar.empty[stage], (job / NS + 1) & 1))) break;
                const uint32_t have = *(volatile uint32_t*)&bar.have[slot];
                const uint8_t* from = raw + slot * M::kRawBytes;
                uint8_t* sK = sKV + 2 * stage * M::kOperand;
                uint8_t* sV = sK + M::kOperand;
                {
                    const uint8_t* tile = from + ku * T::kBytes;
                    uint32_t w[NG], s9[(NG + 3) / 4];
                    load_words(w, tile + kt * (HD / 2) + kc * 4 * NG);
                    // (a token's scales by its four lanes, handed on by shuffles)
                    const bool there = ((have >> ku) & 1) && seen(position(ku) + kt);
#pragma unroll
                    for (int i = 0; i < (NG + 3) / 4; ++i) {
                        const int G = 4 * i + kc < NG ? 4 * i + kc : 0;
                        s9[i] = fit(*reinterpret_cast<const uint16_t*>(
                                        tile + key_scale<HD>(0, 0) + (kt * NG + G) * 2),
                                    there);
                    }
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        const uint32_t s = __byte_perm(
                            __shfl_sync(0xffffffffu, s9[G / 4], (lane & ~3) | (G % 4)), 0, 0x1010);
                        const uint32_t s5 = half_mul(s, 0x2C002C00u);  // 2^-4
                        uint32_t y[4];
                        decode_word(y, w[G], s, s5, s, s5);
                        *reinterpret_cast<uint4*>(sK + (G & 1 ? k_odd : k_even) + G / 2 * 8192) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                // V: a warp takes 64 elements of a tile, a lane four words of them.
#pragma unroll
                for (int i0 = 0; i0 < 2 * HD; i0 += 256) {
                    const int i = i0 / 32 + warp, u = i / kChunks, q = i % kChunks;
                    if (i >= HD / 16) break;
                    const uint8_t* tile = from + u * T::kBytes;
                    uint32_t w[4];
                    load_words(w, tile + T::kCodes + (q * 32 + lane) * 16);
                    const int t = lane & 15;
                    const bool there = ((have >> u) & 1) && seen(position(u) + t);
                    uint32_t s9 = fit(*reinterpret_cast<const uint16_t*>(
                                          tile + value_scale<HD>(0, 0) +
                                          (t * NG + 2 * q + (lane >> 4)) * 2),
                                      there);
                    // (even lanes: their token's scale and the next one's)
                    s9 = __byte_perm(s9, __shfl_down_sync(0xffffffffu, s9, 1), 0x5410);
                    uint8_t* to = sV + swizzled_offset(64 * q + vg, 32 * u + 8 * vc, 128);
#pragma unroll
                    for (int G = 0; G < 2; ++G) {
                        const uint32_t lo = __shfl_sync(0xffffffffu, s9, 16 * G + 2 * vc);
                        const uint32_t hi = __shfl_sync(0xffffffffu, s9, 16 * G + 2 * vc + 8);
                        const uint32_t lo5 = half_mul(lo, 0x2C002C00u);
                        const uint32_t hi5 = half_mul(hi, 0x2C002C00u);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t y[4];
                            decode_word(y, w[2 * G + e], lo, lo5, hi, hi5);
                            uint8_t* at = to + (2 * G + e) * 2048;  // 16 rows on
                            *reinterpret_cast<uint2*>(at) = make_uint2(y[0], y[2]);
                            *reinterpret_cast<uint2*>(at + 1024) = make_uint2(y[1], y[3]);
                        }
                    }
                }
                if (tid == 0) bar.hidden[stage] = ~have & 15u;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.full[stage]);
                if (lane == 0) mbar_arrive(&bar.raw_empty[slot]);
                if (++slot == RD) {
                    slot = 0;
                    raw_parity ^= 1;
                }
            }
        }
        if (unfit) *(volatile int*)&bar.unfit = 1;
        if (!ok) give_up();
    } else if (warp < 12) {
        shrink_registers<48>();
        // ---------------------------------------------------------------- products of row tile w
        const int w = warp - 8;
        if (w < M::kGroups) {
            constexpr uint32_t idesc_s = idesc_f16_f32(128, 64);
            constexpr uint32_t idesc_o = idesc_f16_f32(128, HD);
            const uint32_t leader = elect_one();
            const uint64_t dq = smem_desc_kmajor(smem_u32(sQ + w * 128 * HD * 2), 128);
            const uint64_t dk = smem_desc_kmajor(smem_u32(sKV), 128);
            const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
            const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
            const uint32_t d_s = tmem + w * 128, d_o = tmem + M::kOCols + w * HD;
            uint32_t job = 0, pieces = 0, taken = 0;
            while (ok && advance(walk)) {
                const int jobs = (walk.n + 3) / 4;
                if (jobs == 0) continue;
                if (walk.v.live <= 128 * w) {  // no rows: only the stages go on
                    for (int j = 0; j < jobs && ok; ++j, ++job) {
                        if (!(ok = wait(&bar.full[job % NS], (job / NS) & 1))) break;
                        if (leader) mbar_arrive(&bar.empty[job % NS]);
                        __syncwarp();
                    }
                    continue;
                }
                if (!(ok = wait(&bar.q_full[w], pieces & 1))) break;
                ++pieces;
                auto score = [&](int j) {
                    const uint32_t at = job + j;
                    if (!(ok = wait(&bar.full[at % NS], (at / NS) & 1))) return;
                    tc_fence_after_sync();
                    const uint32_t k = k_lo + (at % NS) * (2 * M::kOperand >> 4);
#pragma unroll
                    for (int s = 0; s < HD / 16; ++s)
                        umma_bf16_warp(leader, d_s + 64 * (j & 1),
                                       q_lo + (s >> 2) * (16384 >> 4) + 2 * (s & 3), q_hi,
                                       k + (s >> 2) * (8192 >> 4) + 2 * (s & 3), k_hi, idesc_s,
                                       s > 0);
                    umma_commit_warp(leader, &bar.s_full[w][j & 1]);
                };
                score(0);
                if (ok && jobs > 1) score(1);
                for (int j = 0; j < jobs && ok; ++j) {
                    const int b = j & 1;
                    if (!(ok = wait(&bar.p_full[w][b], (taken >> b) & 1))) break;
                    taken ^= 1u << b;
                    tc_fence_after_sync();
                    const uint32_t at = job + j;
                    const uint32_t v =
                        k_lo + ((2 * (at % NS) + 1) * (M::kOperand >> 4));
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_bf16_ts_warp(leader, d_o, d_s + 64 * b + 8 * s, v + 2 * s, k_hi,
                                          idesc_o, j > 0 || s > 0);
                    umma_commit_warp(leader, &bar.empty[at % NS]);
                    if (j + 2 < jobs)
                        score(j + 2);
                    else
                        umma_commit_warp(leader, &bar.o_done[w][b]);
                }
                job += jobs;
            }
            if (!ok) give_up();
        } else if (w == 2) {
            // ------------------------------------------------------------ copies
            // A bulk copy for each of a job's tiles, a lane each; the block ids of a job are asked
            // for when the one before it is copied.
            bool more = advance(walk);
            int n = walk.n, k = 0, slot = 0, id = -1, sub = 0, head = 0;
            uint32_t parity = 1, job = 0;
            bool mine = false;
            auto prepare = [&]() {
                while (more && k >= n) {
                    more = advance(walk);
                    n = walk.n;
                    k = 0;
                }
                mine = more && lane < 4 && k + lane < n;
                if (mine) {
                    const int pos = walk.v.tile(walk.k + k + lane) * 16;
                    const int entry = pos / p.bs;
                    sub = (pos - entry * p.bs) / 16;
                    id = __ldg(p.table + walk.x.e0 + entry);
                }
                if (more) head = walk.h;
            };
            prepare();
            for (; more; ++job) {
                const bool good = mine && id >= 0 && id < p.max_blocks;
                if (mine && !good) raise_error(p.dev_status, p.lib_error, HSS_ERR_OUT_OF_RANGE);
                const int64_t place =
                    ((static_cast<int64_t>(id) * p.nkv + head) * (p.bs / 16) + sub) * T::kBytes;
                const uint32_t have = __ballot_sync(0xffffffffu, good);
                if (!(ok = wait(&bar.raw_empty[slot], parity))) break;
                if (lane == 0) {
                    bar.have[slot] = have;
                    if (have != 0)
                        mbar_arrive_expect_tx(&bar.raw_full[slot], __popc(have) * T::kBytes);
                    else
                        mbar_arrive(&bar.raw_full[slot]);
                }
                __syncwarp();
                if (good)
                    bulk_copy_g2s(raw + slot * M::kRawBytes + lane * T::kBytes, p.cache + place,
                                  T::kBytes, &bar.raw_full[slot]);
                __syncwarp();
                if (++slot == RD) {
                    slot = 0;
                    parity ^= 1;
                }
                k += 4;
                prepare();
            }
            if (!ok) give_up();
            // Nobody leaves before the copies have landed: the last use of every slot.
            for (uint32_t i = 0; i < RD && i < job; ++i) {
                const uint32_t use = job - 1 - i;
                (void)mbar_wait_for(&bar.raw_full[use % RD], (use / RD) & 1,
                                    ok ? kWaitLimitNs : 1000000);
            }
        }
    } else {
        grow_registers<144>();
        // ---------------------------------------------------------------- softmax
        const int w = (warp - 12) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        if (w < M::kGroups) {
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t s_cols = lanes + w * 128, o_cols = lanes + M::kOCols + w * HD;
            uint8_t* q_rows = sQ + w * 128 * HD * 2;
            uint32_t next = 0, ends = 0;  // bit b: parity of buffer b's next scores, next end
            uint32_t job = 0;
            while (ok && advance(walk)) {
                const View& v = walk.v;
                const int n = walk.n, jobs = (n + 3) / 4;
                const int live = min(max(v.live - 128 * w, 0), 128);
                if (live == 0) {
                    job += jobs;
                    continue;
                }
                const int r = v.r0 + 128 * w + row, tokens = walk.x.tokens;
                const bool here = row < live;
                const int64_t to = (static_cast<int64_t>(walk.x.q0) + r / p.g) * p.nq +
                                   walk.h * p.g + r % p.g;
                const int own = here ? walk.x.ctx + r / p.g : -1;
                float c = 0.0f;
                if (jobs > 0) {
                    // The row of Q times 2^n, its largest element between 2^10 and 2^11.
                    const uint4* from = reinterpret_cast<const uint4*>(p.Q + to * HD);
                    uint32_t most = 0;
                    if (here) {
#pragma unroll 4
                        for (int i = 0; i < HD / 8; ++i) {
                            const uint4 u = __ldg(from + i);
                            most = __vmaxu2(
                                __vmaxu2(most, __vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu)),
                                __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
                        }
                    }
                    most = max(most & 0xFFFFu, most >> 16);
                    const int e = min(137 - static_cast<int>(most >> 7), 126);
                    // (c is never 0: times what is hidden, -inf, it has to be -inf)
                    const float up = p.c < 0.0f ? -pow2(e) : (p.c > 0.0f ? pow2(e) : 0.0f);
                    c = p.c == 0.0f ? 1.0f : fmaxf(fabsf(p.c) * pow2(-e), 1.2e-38f);
                    // Scores here are below 2^28, so that times c they may be past fp32: then the
                    // kernel for few rows, which does not shift rows so, says what they come to.
                    if (here && c > 0x1p98f && most < 0x7F80u) *(volatile int*)&bar.unfit = 1;
#pragma unroll 2
                    for (int i = 0; i < HD / 8; ++i) {
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (here) u = __ldg(from + i);
                        auto lo = [&](uint32_t x) { return __uint_as_float(x << 16) * up; };
                        auto hi = [&](uint32_t x) {
                            return __uint_as_float(x & 0xFFFF0000u) * up;
                        };
                        *reinterpret_cast<uint4*>(q_rows + (i >> 3) * 16384 +
                                                  swizzled_offset(row, 16 * (i & 7), 128)) =
                            make_uint4(half2_bits(lo(u.x), lo(u.z)), half2_bits(hi(u.x), hi(u.z)),
                                       half2_bits(lo(u.y), lo(u.w)), half2_bits(hi(u.y), hi(u.w)));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full[w]);
                }
                // Jobs [open0, open1) are seen whole by every row of the tile.
                const int at0 = walk.x.ctx + (v.r0 + 128 * w) / p.g;
                const int at1 = walk.x.ctx + (v.r0 + 128 * w + live - 1) / p.g;
                const int w0 = v.w0 - v.sinks, k_first = walk.k, sinks = v.sinks;
                const int window_end = at1 - p.window, open_end = min(at0, tokens - 1) - 15;
                const int t0 = max(sinks, window_end < 0 ? 0 : window_end / 16 + 1 - w0) - k_first;
                const int t1 =
                    min((open_end < 0 ? 0 : open_end / 16 + 1) - w0 - k_first, n);
                const int open0 = (max(t0, 0) + 3) / 4, open1 = t1 < 4 ? 0 : t1 / 4;
                // The maximum that weights go by, less 7; and what a score has to pass to move it.
                float base = 0.0f, limit = -INFINITY, l = 0.0f;
                for (int j = 0; j < jobs; ++j, ++job) {
                    const int b = j & 1;
                    if (!(ok = wait(&bar.s_full[w][b], (next >> b) & 1))) break;
                    next ^= 1u << b;
                    tc_fence_after_sync();
                    const uint32_t hidden = *(volatile uint32_t*)&bar.hidden[job % NS];
                    uint32_t x[64];
                    float m0 = load_scores(s_cols + 64 * b, x);
                    float m1 = load_scores(s_cols + 64 * b + 32, x + 32);
                    tmem_ld_wait();
                    hold(x);
                    hold(x + 32);
                    order_after_wait(m0);
                    order_after_wait(m1);
                    float top = fmaxf(m0, m1);
                    if (j < open0 || j >= open1 || hidden != 0) {
                        // What the row does not see goes to -inf.
                        top = -INFINITY;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int k = k_first + 4 * j + u;
                            const int p0 = (k < sinks ? k : w0 + k) * 16;
                            const bool there = !((hidden >> u) & 1) && 4 * j + u < n;
                            const int last = there ? min(own, tokens - 1) - p0 : -1;
                            const int sink = p.sinks - p0, from = max(own - p0, -16) - p.window;
#pragma unroll
                            for (int d = 0; d < 16; ++d) {
                                const int t = 8 * ((d >> 1) & 1) + d / 4 * 2 + (d & 1);
                                const bool see = t <= last && (t < sink || t > from);
                                const float s = see ? __uint_as_float(x[16 * u + d]) : -INFINITY;
                                x[16 * u + d] = __float_as_uint(s);
                                top = fmaxf(top, s);
                            }
                        }
                    }
                    top = top == -INFINITY ? top : top * c;
                    const bool grow = top > limit;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to_base = grow ? top - 7.0f : base;
                        if (j > 0) {
                            // The product before has to be done with O; what was issued after it
                            // tells: the next scores, or at the end of the piece its own commit.
                            const int o = b ^ 1;
                            ok = j + 1 < jobs ? wait(&bar.s_full[w][o], (next >> o) & 1)
                                              : wait(&bar.o_done[w][o], (ends >> o) & 1);
                            if (!ok) break;
                            tc_fence_after_sync();
                            const float shrink =
                                !grow ? 1.0f : (limit == -INFINITY ? 0.0f : ex2(base - to_base));
                            l *= shrink;
#pragma unroll 1
                            for (int k = 0; k < HD; k += 32) {
                                uint32_t o32[32];
                                tmem_ld_32x32b_x32(o_cols + k, o32);
                                tmem_ld_wait();
                                hold(o32);
#pragma unroll
                                for (int d = 0; d < 32; ++d)
                                    o32[d] =
                                        __float_as_uint(__uint_as_float(o32[d]) * shrink);
                                tmem_st_32x32b_x32(o_cols + k, o32);
                            }
                        }
                        base = to_base;
                        if (grow) limit = top + kLazy;
                    }
                    uint32_t packed[32];
                    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                    for (int d = 0; d < 32; ++d) {
                        const float a = ex2(fmaf(__uint_as_float(x[2 * d]), c, -base));
                        const float e = ex2(fmaf(__uint_as_float(x[2 * d + 1]), c, -base));
                        sum0 += a;
                        sum1 += e;
                        // (fp16, as V: a weight is off by up to 2^-11 of itself)
                        packed[d] = half2_bits(a, e);
                    }
                    l += sum0 + sum1;
                    tmem_st_32x32b_x32(s_cols + 64 * b, packed);
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[w][b]);
                }
                if (!ok) break;
                // What this piece came to.
                if (jobs > 0) {
                    const int b = (jobs - 1) & 1;
                    if (!(ok = wait(&bar.o_done[w][b], (ends >> b) & 1))) break;
                    ends ^= jobs > 1 ? 3u : 1u;
                    tc_fence_after_sync();
                }
                const int64_t part =
                    (2 * static_cast<int64_t>(blockIdx.x) + (k_first > 0 ? 0 : 1)) * R + 128 * w +
                    row;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if (jobs > 0) {
#pragma unroll 1
                    for (int k = 0; k < HD; k += 32) {
                        uint32_t o[32];
                        __syncwarp();
                        tmem_ld_32x32b_x32(o_cols + k, o);
                        tmem_ld_wait();
                        hold(o);
                        if (here && walk.whole) {
                            uint4* at = reinterpret_cast<uint4*>(p.out + to * HD + k);
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                uint32_t u[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    u[e] = l == 0.0f
                                               ? 0u
                                               : pack_bf16x2(
                                                     __uint_as_float(o[8 * d + 2 * e]) * inv,
                                                     __uint_as_float(o[8 * d + 2 * e + 1]) * inv);
                                at[d] = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        } else if (here) {
                            uint4* at = reinterpret_cast<uint4*>(p.part_o + part * HD + k);
#pragma unroll
                            for (int d = 0; d < 8; ++d)
                                at[d] = make_uint4(o[4 * d], o[4 * d + 1], o[4 * d + 2],
                                                   o[4 * d + 3]);
                        }
                    }
                    tc_fence_before_sync();
                } else if (here && walk.whole) {
                    uint4* at = reinterpret_cast<uint4*>(p.out + to * HD);
                    for (int d = 0; d < HD / 8; ++d) at[d] = make_uint4(0, 0, 0, 0);
                }
                if (here && walk.whole && p.lse != nullptr)
                    p.lse[to] =
                        l == 0.0f ? -INFINITY : (base + log2f(l)) * 0.693147180559945309f;
                if (here && !walk.whole) p.part_ml[part] = make_float2(base, l);
            }
            if (!ok) give_up();
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0) flags[blockIdx.x] = bar.unfit;
    if (warp == 8) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// What is left of a row in several pieces, of the kernel that did the work.
template <int HD>
__global__ void __launch_bounds__(kJoinThreads, 1)
    join_either_kernel(const Params many, const Params few, bool many_joined, bool few_joined) {
    grid_dependency_wait();
    grid_launch_dependents();
    if (wanted(few)) {
        if (few_joined && blockIdx.y < 2) join_pieces<HD, 16, 1>(few);
    } else if (many_joined && blockIdx.x < kSms - 1) {
        join_pieces<HD, Many<HD>::kRows, 4>(many);
    }
}

template <int HD>
hss_status launch_many(const Params& args, const Params& few, int32_t* flags,
                       cudaStream_t stream) {
    using M = Many<HD>;
    auto kern = many_kernel<HD>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kSmemBytes) !=
        cudaSuccess)
        return HSS_ERR_CUDA;
    Params many = args, guarded = few;
    const int64_t row_tiles = row_tiles_bound(many, M::kRows);
    const int64_t units = many.num_seqs * row_tiles * many.nkv;
    const bool many_joined = !many_by_units(tiles_bound(many), units);
    many.row_tiles = many_joined ? 0 : static_cast<int32_t>(row_tiles);
    guarded.guards = many_joined ? kSms : static_cast<int32_t>(units);
    if (launch_pdl(kern, dim3(guarded.guards), dim3(M::kThreads), M::kSmemBytes, stream, many,
                   flags) != cudaSuccess)
        return HSS_ERR_CUDA;
    // (does nothing unless a scale did not fit)
    bool few_joined;
    const hss_status st = launch_few<HD, 2>(guarded, &few_joined, stream);
    if (st != HSS_OK || (!many_joined && !few_joined)) return st;
    return launch_pdl(join_either_kernel<HD>, dim3(Shape<HD, 2>::kRanges - 1, 8),
                      dim3(kJoinThreads), 0, stream, many, guarded, many_joined,
                      few_joined) == cudaSuccess
               ? HSS_OK
               : HSS_ERR_CUDA;
}

}  // namespace packed
}  // namespace hss
