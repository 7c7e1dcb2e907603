// attention_prefix.cu -- tensor-core (tcgen05) HCA attention for a batch whose
// elements share their first N_p compressed entries.
//
// For query row (b, q) at position t, head h (one softmax over the union):
//   keys = logical entries s < min(floor((t+1)/m), n_entries[b])   (kv_p, then kv_c[b])
//          and the raw window rows at [max(0, t-W+1), t]
//   o = sum softmax(scale * q.key) key                  (key = value: shared-KV MQA)
// The shared entries are the same keys for every row of the batch, so they are
// one GEMM over all (row, head) pairs.  What bounds it: per (row, head, key)
// the two products take 512 flops and the weight one exponential, and on an SM
// both take about the same time (1024 cycles for 128 pairs x 128 keys), so the
// tensor pipe and the MUFU have to run at once; HBM traffic is small (the
// prefix is read from L2, 32 KB a tile and CTA).
//
// Unit of work: 128 consecutive (row, head) pairs, an MMA's M = G = 128 / H query
// rows.  Its list of key tiles (128 keys):
//   - shared tiles: prefix entries that every row of the unit sees, by TMA;
//   - own tiles: each of the G rows gets H columns, filled with that row's further
//     keys (its window, the rest of the prefix it sees, its own entries); P V
//     updates each row's lanes from its own columns only (the other row's keys may
//     be infinite or NaN, which a weight of zero would not take out).  Runs of 64
//     rows in one place come by TMA, the rest by 16-byte cp.async, rows past a
//     list's end as zero rows, so nothing that a row may not see enters its output.
// The units' lists are dealt over the CTAs of one wave: CTA c of n takes the
// part [c U / n, (c+1) U / n) of the U units laid end to end, each unit's tiles
// cut in that proportion.  A unit that stays whole is written out by its CTA;
// the parts of a cut one leave their unnormalised O (fp32), running maximum
// and sums in the workspace, and a second kernel joins them in a fixed order.
// Only a CTA's first and last unit can be cut, so the workspace goes with the
// CTAs, not with the units: slot c for the first unit of CTA c, n + c for its last.
//
// Roles (20 warps, one CTA per SM): warps 0-1 load key tiles; warp 2 loads Q and
// issues S = Q.K; warp 3 issues O += P.V; warps 4-11 and 12-19 turn S into P,
// every other tile each, two threads a row.  TMEM: three buffers S / P (P, in
// bf16, overwrites S) and O, 128 columns each, so Q.K runs up to three tiles
// ahead of P.V and neither the tensor pipe nor the MUFU waits for the other.
// (Two M tiles a CTA, each with one S, shared the key tiles but ran S -> P -> S
// as a chain: 1.4 times the time a tile, and twice the O to join.)
//
// The offset.  The weights are exp2(z - m) with m the row's score of one key of
// the part's first tile, not a maximum: the true maximum is not below it, so
// nothing that counts underflows, and fp32 sums and bf16 weights lose nothing
// while z - m stays below 64.  Where a sum of weights reaches 2^64, or that one
// score is not finite, the part is run again: once for the rows' maxima alone, once
// with those as m.
// P has bf16's 8 significant bits (A and B of an MMA share their type, and the
// keys are bf16): its rounding moves an output by at most 2^-8 of the spread of
// the averaged values, like the rounding of the output itself.  The output
// divides by the sum of the rounded weights, the LSE uses the exact sum.
#include <cudaTypedefs.h>

#include <math.h>

#include <algorithm>

#include "attn_rows.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tc;

constexpr int kD = 128;
constexpr int kRows = 128;                  // rows of a unit
constexpr int kBN = 128;                    // keys per tile
constexpr int kStages = 5;
constexpr int kBufs = 3;                    // S / P buffers
constexpr int kHalf = 16384;                // one 64-column half of a 128-row tile
constexpr int kBox = 8192;                  // 64 rows of it: what a TMA copy brings
constexpr int kTileBytes = 2 * kHalf;
constexpr int kLoadWarps = 2;
constexpr int kLoadThreads = kLoadWarps * 32;
constexpr int kQkWarp = 2, kPvWarp = 3, kSoftWarp0 = 4;
constexpr int kSoftWarps = 16;              // two groups of 8
constexpr int kThreads = (kSoftWarp0 + kSoftWarps) * 32;
constexpr int kSms = 148;
constexpr uint32_t kOCol = kBufs * 128;     // O's first TMEM column
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRange = 0x1p64f;
constexpr int kPartFloats = kRows * kD + 3 * kRows;    // O, then m, l_r, l_e of a part
constexpr int kMaxUnits = 32;               // units a CTA meets, at most

struct __align__(8) Ctrl {
    uint64_t bar_q, q_free;
    uint64_t full[kStages], freeb[kStages];
    uint64_t s_full[kBufs], p_ready[kBufs][2], s_free[kBufs];   // p_ready: by 64-key half
    uint64_t o_full, o_free;
    uint64_t m_ready;        // the rows' offsets are there
    uint64_t done;           // every warp is through with the attempt
    uint64_t fin[2], stall_bar;
    uint32_t tmem_base;
    int abort;
    int q_ahead;             // the first unit's Q was requested in the prologue
    int over[3];             // (attempt mod 3) some sum of weights left the range
    // offsets in use (base 2), by the parity of the CTA's units: the next unit's first tile
    // may give its offsets while this unit's are still read for the LSE and the workspace
    float m[2][kRows];
    float xm[4][kRows];      // per thread of a row: its maximum
    float xl[2][4][2][kRows];   // (by attempt parity) its sums of rounded / exact weights
};

struct PrefixParams {
    const __nv_bfloat16* kv_p;
    const __nv_bfloat16* kv_c;
    const __nv_bfloat16* kv_raw;
    AttnArgs a;              // sizes and per-element arrays
    int hshift;              // log2(H)
    int R;                   // query rows
    int U;                   // units
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    float* ws;
    uint32_t* err;
    uint64_t wait_ns;
    int stall;
};

// What one query row sees (in smem, filled once by the CTA's threads).
struct RowRec {
    int on;                  // it exists and has a position
    int b;
    int vis;                 // visible logical entries
    int win_lo, n_win;       // raw rows
    int n_pre, n_own;        // prefix entries beyond the shared tiles, own entries
    int pad;
};
// A unit's tile list (P shared tiles, then T own tiles) and the CTA's part of it.
struct Geo {
    int P, T;
    int lo, hi;              // tiles [lo, hi)
    int whole;               // all of the unit?
};
constexpr size_t kSmem = 1024 + kTileBytes + kStages * kTileBytes + sizeof(Ctrl) +
                         kMaxUnits * (sizeof(Geo) + 2 * sizeof(RowRec));

// x / n for x >= 0 (64-bit division only where it is needed).
__device__ __forceinline__ int div_of(long x, int n) {
    return x < (1L << 31) ? (int)((unsigned)x / (unsigned)n) : (int)(x / n);
}
__device__ __forceinline__ int first_unit(const PrefixParams& p, int c, int n) { return div_of((long)c * p.U, n); }
__device__ __forceinline__ int end_unit(const PrefixParams& p, int c, int n) {
    return div_of((long)(c + 1) * p.U + n - 1, n);
}

// The CTA's units u0 .. u0 + n - 1: a thread per query row, then one per unit.
template <int G>
__device__ __forceinline__ void fill_geometry(const PrefixParams& p, int c, int n_cta, int u0, int n, Geo* geo,
                                              RowRec* rows) {
    constexpr int H = kRows / G;
    // (by warps that have nothing else to set up; a row's arrays are read at once)
    constexpr int kFirst = kSoftWarp0 * 32, kStep = kThreads - kFirst;
    for (int i = (int)threadIdx.x - kFirst; i >= 0 && i < n * G; i += kStep) {
        const int row = u0 * G + i;
        RowRec r{};
        if (row < p.R) {
            r.b = row / p.a.n_q;
            const int t = p.a.q_pos ? __ldg(p.a.q_pos + row) : row - r.b * p.a.n_q;
            const RowKeys k = row_keys(p.a, r.b, t);
            if (t >= 0) {
                r.on = 1;
                r.vis = k.n_comp;
                r.win_lo = k.win_lo;
                r.n_win = k.n_win;
            }
        }
        rows[i] = r;
    }
    __syncthreads();
    for (int k = (int)threadIdx.x - kFirst; k >= 0 && k < n; k += kStep) {
        Geo g{};
        int lo = p.a.N_p, on = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const RowRec& r = rows[k * G + i];
            if (r.on) lo = min(lo, r.vis);
            on |= r.on;
        }
        g.P = on ? lo / kBN : 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            RowRec& r = rows[k * G + i];
            if (!r.on) continue;
            r.n_pre = max(min(r.vis, p.a.N_p) - g.P * kBN, 0);
            r.n_own = max(r.vis - p.a.N_p, 0);
            g.T = max(g.T, (r.n_pre + r.n_own + r.n_win + H - 1) / H);
        }
        // CTA c takes [c U, (c+1) U) of the line on which unit u is [u n_cta, (u+1) n_cta)
        const long a = (long)c * p.U, b = a + p.U, x = (long)(u0 + k) * n_cta, y = x + n_cta;
        g.lo = div_of((max(a, x) - x) * (g.P + g.T), n_cta);
        g.hi = div_of((min(b, y) - x) * (g.P + g.T), n_cta);
        g.whole = a <= x && b >= y;
        geo[k] = g;
    }
}
// A bounded wait: one try in line, the rest out of line.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                       uint64_t limit_ns) {
    return mbar_wait(bar, parity, abort, err, limit_ns);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                         uint64_t limit_ns) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, err, limit_ns);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float f2lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Adds bytes that the barrier's current phase waits for, without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// True in one lane of a warp that is together (always the same one).
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}
// 16-byte copy global -> shared, or 16 zero bytes (nothing is read) when !on.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// One fp32 column of this thread's TMEM lane.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
                 "tcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(taddr) : "memory");
    return __uint_as_float(v);
}
// Largest of the first n (1 .. 64) S values at s_addr of this thread's row.
__device__ __noinline__ float row_max(uint32_t s_addr, int n) {
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < n; c += 32) {
        float sv[32];
        tmem_ld32(s_addr + c, sv);
        if (n < c + 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (c + e >= n) sv[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            mx0 = max3(mx0, sv[e], sv[e + 1]);
            mx1 = max3(mx1, sv[e + 2], sv[e + 3]);
        }
    }
    return fmaxf(mx0, mx1);
}

// A unit's Q, 128 rows.
__device__ __forceinline__ void load_q(uint8_t* sQ, const CUtensorMap* tm, int u, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, kTileBytes);
    for (int q = 0; q < 4; ++q)
        tma_load_2d(sQ + (q & 1) * kHalf + (q >> 1) * kBox, tm, (q & 1) * 64, u * kRows + (q >> 1) * 64, bar);
}

// An attempt at a part, as every role walks it: kFast, and where that left the
// range, kMax (the rows' maxima) and kExact (with them).
enum Mode { kFast = 0, kMax = 1, kExact = 2 };

template <int G, bool LSE>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_p,
                   const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ PrefixParams p) {
    constexpr int H = kRows / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = base;                                  // [32 KB]
    uint8_t* sK = sQ + kTileBytes;                       // [kStages][32 KB]
    Ctrl* ctl = reinterpret_cast<Ctrl*>(sK + kStages * kTileBytes);
    Geo* geo = reinterpret_cast<Geo*>(ctl + 1);          // [kMaxUnits]
    RowRec* rows = reinterpret_cast<RowRec*>(geo + kMaxUnits);   // [kMaxUnits][G]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort = &ctl->abort;
    const int c = blockIdx.x, n_cta = gridDim.x;
    const int u0 = first_unit(p, c, n_cta), u1 = end_unit(p, c, n_cta);

    grid_wait();
    if (threadIdx.x == 0) {
        // a CTA started after another one timed out does no work
        const bool dead = *reinterpret_cast<volatile uint32_t*>(p.err) != 0u;
        mbar_init(&ctl->bar_q, 1);
        mbar_init(&ctl->q_free, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl->full[i], kLoadThreads);
            mbar_init(&ctl->freeb[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_ready[i][0], kSoftWarps / 2);
            mbar_init(&ctl->p_ready[i][1], kSoftWarps / 2);
            mbar_init(&ctl->s_free[i], 1);
        }
        mbar_init(&ctl->o_full, 1);
        mbar_init(&ctl->o_free, kSoftWarps);
        mbar_init(&ctl->m_ready, 4);
        mbar_init(&ctl->done, kThreads / 32);
        for (int i = 0; i < 2; ++i) mbar_init(&ctl->fin[i], 1);
        mbar_init(&ctl->stall_bar, 1);
        ctl->over[0] = ctl->over[1] = ctl->over[2] = 0;
        fence_barrier_init();
        ctl->abort = dead;
        ctl->q_ahead = !dead;
    }
    if (warp == 0) {
        __syncwarp();
        // (by an elected lane: TMA copies issued under a lane number took 200 cycles each)
        if (__all_sync(0xffffffffu, *(volatile int*)&ctl->q_ahead != 0) && elect_one()) load_q(sQ, &tm_q, u0, &ctl->bar_q);
        __syncwarp();
    }
    if (warp == kQkWarp) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    fill_geometry<G>(p, c, n_cta, u0, u1 - u0, geo, rows);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {       // by a whole warp
        return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, p.err, p.wait_ns));
    };
    // What follows an attempt: the same answer for every role.  Its flag is read
    // once every warp has arrived, and goes back after the next meeting.
    int k = 0;                       // attempts so far
    auto next_mode = [&](Mode mode, bool* ok) -> Mode {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->done);
        *ok = wait(&ctl->done, k & 1);
        const bool over = *(volatile int*)&ctl->over[k % 3] != 0;
        if (threadIdx.x == kThreads - 1) *(volatile int*)&ctl->over[(k + 2) % 3] = 0;
        ++k;
        return mode == kFast ? (over ? kMax : kFast) : (mode == kMax ? kExact : kFast);
    };

    if (warp < kLoadWarps) {
        // ------------------------------------------------------------ key tiles
        const int lt = threadIdx.x, c16 = lt & 15;
        const uint32_t col = (uint32_t)(c16 >> 3) * kHalf;   // this thread's 16 bytes of a row
        int L = 0;                    // tiles handed out
        int pend = -1;                // stage of a copied tile that has not arrived yet
        uint32_t tma_stage = 0;       // stages whose latest tile came (in part) by TMA
        // the copied tile before the latest commit group has landed: hand it over
        auto settle = [&](bool all) {
            if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
            else asm volatile("cp.async.wait_group 1;" ::: "memory");
            if (pend >= 0) {
                fence_proxy_async_smem();
                mbar_arrive(&ctl->full[pend]);
                pend = -1;
            }
        };
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const Geo g = geo[u - u0];
            const RowRec* rec = rows + (u - u0) * G;
            Mode mode = kFast;
            if (g.lo < g.hi) do {
                for (int i = g.lo; i < g.hi; ++i, ++L) {
                    const int slot = L % kStages, use = L / kStages;
                    if (use > 0) ok = wait(&ctl->freeb[slot], (use - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok && *abort == 0);
                    if (!ok) break;
                    uint8_t* dst = sK + slot * kTileBytes;
                    uint64_t* bar = &ctl->full[slot];
                    bool copies = false, boxes = i < g.P;
                    if (i < g.P) {
                        if (warp == 0 && elect_one()) {
                            mbar_expect_tx(bar, kTileBytes);
                            for (int q = 0; q < 4; ++q)
                                tma_load_2d(dst + (q & 1) * kHalf + (q >> 1) * kBox, &tm_p, (q & 1) * 64, i * kBN + (q >> 1) * 64, bar);
                        }
                    } else {
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {                 // 64 rows of the tile
                            const RowRec rw = rec[G == 2 ? q : 0];
                            const int j = (i - g.P) * H + (G == 2 ? 0 : 64 * q);
                            const int e1 = rw.n_win, e2 = e1 + rw.n_pre, e3 = e2 + rw.n_own;
                            // one segment holds all 64 rows: window, rest of the prefix, own entries
                            const bool w = j + 64 <= e1, pre = j >= e1 && j + 64 <= e2, own = j >= e2 && j + 64 <= e3;
                            if (w || pre || own) {
                                boxes = true;
                                if (warp == 0 && elect_one()) {
                                    const CUtensorMap* m = w ? &tm_w : (pre ? &tm_p : &tm_c);
                                    const int y = w ? rw.b * p.a.L_raw + rw.win_lo + j
                                                    : (pre ? g.P * kBN + (j - e1) : rw.b * p.a.N_cap + (j - e2));
                                    mbar_expect_tx(bar, 2 * kBox);
                                    tma_load_2d(dst + q * kBox, m, 0, y, bar);
                                    tma_load_2d(dst + kHalf + q * kBox, m, 64, y, bar);
                                }
                                continue;
                            }
                            // row by row, zero rows past the list's end (nothing is read there)
                            copies = true;
                            const __nv_bfloat16* pw = p.kv_raw + ((long)rw.b * p.a.L_raw + rw.win_lo + j) * kD + c16 * 8;
                            const __nv_bfloat16* pp = p.kv_p + ((long)g.P * kBN + j - e1) * kD + c16 * 8;
                            const __nv_bfloat16* po = p.kv_c + ((long)rw.b * p.a.N_cap + j - e2) * kD + c16 * 8;
#pragma unroll 4
                            for (int it = 0; it < 64 / (kLoadThreads / 16); ++it) {
                                const int rr = (lt >> 4) + it * (kLoadThreads / 16), jj = j + rr;
                                const __nv_bfloat16* src = jj < e1 ? pw : (jj < e2 ? pp : po);
                                src = jj < e3 ? src + rr * kD : p.out;
                                cp_async16_or_zero(dst + col + (64 * q + rr) * 128 + (((c16 & 7) ^ (rr & 7)) << 4), src, jj < e3);
                            }
                        }
                    }
                    if (boxes) tma_stage |= 1u << slot;
                    else tma_stage &= ~(1u << slot);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    settle(false);
                    if (copies) pend = slot;
                    else mbar_arrive(bar);
                }
                settle(true);
                if (ok) mode = next_mode(mode, &ok);
            } while (ok && mode != kFast);
        }
        settle(true);
        // TMA tiles in flight land before the CTA's shared memory is given up
        if (lt == 0) {
            volatile int never = 0;
            for (int q = 0; q < kStages; ++q)
                if (((tma_stage >> q) & 1u) && L > q)
                    mbar_wait(&ctl->full[q], ((L - 1 - q) / kStages) & 1, &never, p.err);
        }
    } else if (warp == kQkWarp) {
        // ------------------------------------------------------------ Q, S = Q.K
        // The whole warp runs this (and the next role), kept together by votes, and
        // elect.sync picks the issuing lane: for a branch on the lane number the
        // compiler cannot know that one thread issues, and an MMA took 90 - 120
        // cycles to issue.  Issuing still takes about as long as an MMA's 64 cycles,
        // so Q.K and P.V have a warp each.
        constexpr uint32_t id_qk = idesc_bf16(kRows, kBN, false, false);
        const uint64_t qd = sw128_desc(smem_u32(sQ), 16, 1024), kd0 = sw128_desc(smem_u32(sK), 16, 1024);
        const int ahead = __shfl_sync(0xffffffffu, ctl->q_ahead, 0);
        int L = 0, nq = ahead, nf = 0;            // tiles, Q loads, Q's used up
        bool ok = ahead != 0;
        if (p.stall && ok) ok = wait(&ctl->stall_bar, 0);
        for (int u = u0; u < u1 && ok; ++u) {
            const int n = __shfl_sync(0xffffffffu, geo[u - u0].hi - geo[u - u0].lo, 0);
            if (n == 0) continue;
            if (u != u0) {
                // the Q before has been used (or, its part empty, at least landed)
                ok = nf > 0 ? wait(&ctl->q_free, (nf - 1) & 1) : wait(&ctl->bar_q, (nq - 1) & 1);
                ok = __all_sync(0xffffffffu, ok && *abort == 0);
                if (!ok) break;
                if (elect_one()) load_q(sQ, &tm_q, u, &ctl->bar_q);
                __syncwarp();
                ++nq;
            }
            ok = wait(&ctl->bar_q, (nq - 1) & 1);
            Mode mode = kFast;
            do {
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ++L) {
                    const int slot = L % kStages, buf = L % kBufs, use = L / kBufs;
                    const uint64_t kd = kd0 + (uint64_t)(slot * (kTileBytes >> 4));
                    const uint32_t d = tmem + buf * 128;
                    ok = (use == 0 || wait(&ctl->s_free[buf], (use - 1) & 1)) && wait(&ctl->full[slot], (L / kStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kq = 0; kq < kD / 16; ++kq) {
                            const uint32_t off16 = ((kq >> 2) * kHalf + (kq & 3) * 32) >> 4;
                            mma_bf16_ss(d, qd + off16, kd + off16, id_qk, kq > 0);
                        }
                        mma_commit(&ctl->s_full[buf]);
                    }
                    __syncwarp();
                }
                if (ok) mode = next_mode(mode, &ok);
            } while (ok && mode != kFast);
            if (ok) {
                if (elect_one()) mma_commit(&ctl->q_free);
                __syncwarp();
                ++nf;
            }
        }
        // every MMA must finish before TMEM is released, a Q load in flight
        // must land before shared memory is given up
        if (elect_one()) mma_commit(&ctl->fin[0]);
        __syncwarp();
        volatile int never = 0;
        mbar_wait(&ctl->fin[0], 0, &never, p.err);
        if (nq > 0) mbar_wait(&ctl->bar_q, (nq - 1) & 1, &never, p.err);
        __syncwarp();
    } else if (warp == kPvWarp) {
        // ------------------------------------------------------------ O += P.V
        constexpr uint32_t id_pv = idesc_bf16(kRows, kD, false, true);
        const uint64_t vd0 = sw128_desc(smem_u32(sK), kHalf, 1024);
        int L = 0, no = 0;            // tiles; parts with tiles so far
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const int n = __shfl_sync(0xffffffffu, geo[u - u0].hi - geo[u - u0].lo, 0);
            const int shared = __shfl_sync(0xffffffffu, geo[u - u0].P - geo[u - u0].lo, 0);   // (may be below 0)
            if (n == 0) continue;
            if (no > 0) ok = wait(&ctl->o_free, (no - 1) & 1);      // the previous part's O has been read
            ++no;
            Mode mode = kFast;
            do {
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i, ++L) {
                    const int slot = L % kStages, buf = L % kBufs;
                    const uint64_t vd = vd0 + (uint64_t)(slot * (kTileBytes >> 4));
                    const uint32_t a = tmem + buf * 128;
                    const uint32_t acc = i > 0;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        ok = ok && wait(&ctl->p_ready[buf][q], (L / kBufs) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            if (mode != kMax) {
// (an own tile of two rows: each row's lanes with its own 64 keys)
                                const bool own = G == 2 && i >= shared;
                                const uint32_t pa = a + 64 * q;
                                const uint64_t v = vd + (uint64_t)(4 * q * (2048 >> 4));
                                if (own) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        mma_bf16_ts_half(tmem + kOCol, pa + (kk >> 1) * 32 + (kk & 1) * 8,
                                                         v + (uint64_t)(kk * (2048 >> 4)), id_pv, kk > 0 ? 1u : acc, q);
                                } else {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        mma_bf16_ts(tmem + kOCol, pa + (kk >> 1) * 32 + (kk & 1) * 8,
                                                    v + (uint64_t)(kk * (2048 >> 4)), id_pv, kk + q > 0 ? 1u : acc);
                                }
                                if (q == 1) {
                                    mma_commit(&ctl->freeb[slot]);
                                    mma_commit(&ctl->s_free[buf]);
                                    if (i + 1 == n) mma_commit(&ctl->o_full);
                                }
                            } else if (q == 1) {          // no weights yet: the tile and S are done with
                                mbar_arrive(&ctl->freeb[slot]);
                                mbar_arrive(&ctl->s_free[buf]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                if (ok) mode = next_mode(mode, &ok);
            } while (ok && mode != kFast);
        }
        if (elect_one()) mma_commit(&ctl->fin[1]);
        __syncwarp();
        volatile int never = 0;
        mbar_wait(&ctl->fin[1], 0, &never, p.err);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and output
        // Group gr takes every other tile, thread h of a row 32 columns of each
        // 64-key half (id: which of the row's four threads).  P V of a half
        // starts when its P is there, which frees the buffer sooner: 1490 -> 1420
        // cycles a tile.
        const int gr = (warp - kSoftWarp0) >> 3, h = ((warp - kSoftWarp0) >> 2) & 1, id = 2 * gr + h;
        const int r = (warp & 3) * 32 + lane;                // row of the unit
        const uint32_t my = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int grp = r / H;                               // its query row in the unit
        int L = 0, L_grp = gr;                               // tiles so far; this group's next
        int no = 0, nm = 0;                                  // O's made; first tiles met
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const Geo g = geo[u - u0];
            const RowRec row = rows[(u - u0) * G + grp];
            const int own_len = row.n_pre + row.n_own + row.n_win;
            const int n = g.hi - g.lo;
            float l_r = 0.0f, l_e = 0.0f, m = -INFINITY;
            float* offset = ctl->m[nm & 1];                      // (a unit adds one to nm)
            Mode mode = kFast;
            if (n > 0) do {
                l_r = l_e = 0.0f;
                m = mode == kExact ? offset[r] : -INFINITY;
                const bool leads = L_grp == L;               // this group has the attempt's first tile
                bool have_m = mode != kFast;                 // kFast: m comes with the first tile
                float top = -INFINITY;                       // kMax: largest score seen
                bool large = false;
#pragma unroll 1
                for (; L_grp < L + n; L_grp += 2) {
                    const int buf = L_grp % kBufs, i = g.lo + (L_grp - L);
                    const uint32_t s_addr = my + buf * 128 + 32 * h;
                    // the columns of each half that are keys of the row (the same in all lanes)
                    int nvs = 32 | 32 << 8;
                    if (i >= g.P) {
                        const int left = own_len - (i - g.P) * H - 32 * h;
                        nvs = max(min(left, 32), 0);
                        if (G == 2) nvs <<= 8 * grp;
                        else nvs |= max(min(left - 64, 32), 0) << 8;
                    }
                    // every wait is warp-collective: the TMEM accesses below are .sync.aligned
                    ok = wait(&ctl->s_full[buf], (L_grp / kBufs) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (mode == kMax) {
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            if (nvs & 255) top = fmaxf(top, row_max(s_addr + 64 * q, nvs & 255));
                            nvs >>= 8;
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ctl->p_ready[buf][q]);
                        }
                    } else {
                        if (!have_m) {
                            // the row's first score in the first tile, from the group that has
                            // it.  (A row without keys there has none in the part: the lists
                            // are filled from the front.)
                            if (leads && h == 0) {
                                const int c0 = i < g.P ? 0 : grp * H;
                                float z = tmem_ld1(my + buf * 128 + c0) * p.scale_log2;
                                const bool some = i < g.P || own_len > (i - g.P) * H;
                                // (a score below fp32's range says nothing about the others)
                                large |= row.on && some && !(fabsf(z) < INFINITY);
                                if (!(fabsf(z) < INFINITY)) z = 0.0f;
                                if (!some) z = -INFINITY;
                                offset[r] = z;
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&ctl->m_ready);
                            }
                            ok = wait(&ctl->m_ready, nm & 1);
                            if (!ok) break;
                            m = offset[r];
                            have_m = true;
                        }
                        // P over the S it is made from
                        const float mm = (m == -INFINITY) ? 0.0f : m;
                        const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2), negm = f2_pack(-mm, -mm);
                        uint64_t accr = 0, acce = 0;
                        // (rolled: this much straight-line code would wait for its instructions)
#pragma unroll 1
                        for (int q = 0; q < 2; ++q) {
                            const int nv = nvs & 255;
                            nvs >>= 8;
                            if (nv > 0) {
                                uint32_t pk[16];
                                float sv[32];
                                tmem_ld32(s_addr + 64 * q, sv);
                                if (nv < 32) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (e >= nv) sv[e] = -INFINITY;
                                }
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const uint64_t z = f2_fma(f2_pack(sv[e], sv[e + 1]), sl2, negm);
                                    const float p0 = ex2(f2lo(z)), p1 = ex2(f2hi(z));
                                    uint32_t d;
                                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(p1), "f"(p0));
                                    pk[e >> 1] = d;
                                    accr = f2_add(accr, f2_pack(__uint_as_float(d << 16), __uint_as_float(d & 0xffff0000u)));
                                    if (LSE) acce = f2_add(acce, f2_pack(p0, p1));
                                }
                                tmem_st16(s_addr + 64 * q, pk);
                            } else {
                                uint32_t zero[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) zero[e] = 0u;
                                tmem_st16(s_addr + 64 * q, zero);
                            }
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ctl->p_ready[buf][q]);
                        }
                        const float sum = f2lo(accr) + f2hi(accr);
                        large |= row.on && !(sum < kRange);
                        l_r += sum;
                        l_e += f2lo(acce) + f2hi(acce);
                    }
                }
                if (!ok) break;
                L += n;
                // the attempt's end: what this thread has, for the row's others
                if (mode == kMax) ctl->xm[id][r] = top * p.scale_log2;
                ctl->xl[k & 1][id][0][r] = l_r;
                ctl->xl[k & 1][id][1][r] = l_e;
                if (mode == kFast && __any_sync(0xffffffffu, large) && lane == 0) *(volatile int*)&ctl->over[k % 3] = 1;
                nm += mode == kFast;
                no += mode != kMax;
                const Mode was = mode;
                mode = next_mode(mode, &ok);
                // (waited for in every attempt: a phase must not be skipped)
                if (ok && was != kMax) ok = wait(&ctl->o_full, (no - 1) & 1);
                if (ok && was == kMax) {
                    // (each of the row's four threads writes the same value)
                    offset[r] = max3(fmaxf(ctl->xm[0][r], ctl->xm[1][r]), ctl->xm[2][r], ctl->xm[3][r]);
                    __syncwarp();
                }
            } while (ok && mode != kFast);
            if (!ok) break;
            // ---------------------------------------------------------- the part's end
            // each thread a quarter of its row's O
            if (n > 0) {
                tc_fence_after();
                l_r = l_e = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    l_r += ctl->xl[(k - 1) & 1][q][0][r];
                    l_e += ctl->xl[(k - 1) & 1][q][1][r];
                }
                m = offset[r];
                // keys whose scores are all NaN have no maximum, but are not no keys
                if (m == -INFINITY && l_r != 0.0f) m = 0.0f;
            }
            if (!row.on) {               // no position: no key, whatever the shared tiles held
                m = -INFINITY;
                l_r = l_e = 0.0f;
            }
            const long orow = (long)u * kRows + r;           // flattened (row, head)
            const bool row_ok = u * G + grp < p.R;
            float ov[32];
            tmem_ld32(my + kOCol + 32 * id, ov);             // (nothing of it is used without keys)
            if (g.whole) {
                const bool some = n > 0 && l_r != 0.0f;
                const float inv = some ? 1.0f / l_r : 0.0f;
                __nv_bfloat16* dst = p.out + orow * kD + 32 * id;
                if (row_ok) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[q])
                                : "f"(ov[e + 2 * q + 1] * inv), "f"(ov[e + 2 * q] * inv));
                        *reinterpret_cast<uint4*>(dst + e) = some ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (LSE && id == 0) p.lse[orow] = (n == 0 || l_e == 0.0f) ? -INFINITY : (m + log2f(l_e)) / kLog2e;
                }
            } else {
                // O as [column quad][row] of float4: lanes (rows) are consecutive
                float* ws = p.ws + (size_t)(u == u0 ? c : n_cta + c) * kPartFloats;
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(ws + ((id * 8 + (e >> 2)) * kRows + r) * 4) =
                        make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                if (id == 0) {
                    ws[kRows * kD + r] = n > 0 ? m : -INFINITY;
                    ws[kRows * kD + kRows + r] = l_r;
                    ws[kRows * kD + 2 * kRows + r] = l_e;
                }
            }
            if (n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->o_free);
            }
        }
    }
    // (the issuing warps waited for their final commits: no MMA is in flight)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kQkWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- join
// A CTA per unit (with more units than CTAs, per border between two CTAs: each
// lies in another unit) and 8 of its columns; a thread per row and share of the
// parts.  What bounds it is the latency of the loads (a few parts of
// L2-resident data): a thread's parts are fetched kBatch at a time, and where a
// unit has many parts (few units, so few CTAs), kGroups threads share a row and
// meet in shared memory.  The order of the sums is fixed.
constexpr int kJoinCols = 8;

struct JoinState {
    float m, lr, le;
    float o[kJoinCols];
    // brings this state's scale to maximum M (its own is not above it)
    __device__ __forceinline__ void rescale(float M) {
        const float w = (m == -INFINITY) ? 0.0f : exp2f(m - M);
        m = M;
        lr *= w;
        le *= w;
#pragma unroll
        for (int i = 0; i < kJoinCols; ++i) o[i] *= w;
    }
};

template <bool LSE, int kGroups, int kBatch>
__global__ void __launch_bounds__(kGroups * kRows)
prefix_join_kernel(const __grid_constant__ PrefixParams p, int n_cta) {
    constexpr int kPer = kD / kJoinCols;
    __shared__ float sh[kGroups > 1 ? kGroups - 1 : 1][3 + kJoinCols][kRows];
    const int at = blockIdx.x / kPer, q0 = (blockIdx.x % kPer) * (kJoinCols / 4);
    const int u = p.U > n_cta ? (int)((long)(at + 1) * p.U / n_cta) : at;
    const int r = threadIdx.x & (kRows - 1), grp = threadIdx.x / kRows;
    const long x = (long)u * n_cta, y = x + n_cta;
    const int c0 = (int)(x / p.U), n = (int)((y + p.U - 1) / p.U) - c0;      // the unit's parts
    grid_wait();                                                            // the parts are there
    if (n <= 1) return;                                                     // written whole
    const long orow = (long)u * kRows + r;
    // the parts but the first are of their CTA's first unit
    const int slot0 = (long)c0 * p.U == x ? c0 : n_cta + c0;
    JoinState t;
    t.m = -INFINITY;
    t.lr = t.le = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) t.o[i] = 0.0f;
    for (int k0 = grp; k0 < n; k0 += kGroups * kBatch) {
        float m[kBatch], lr[kBatch], le[kBatch];
        float4 v0[kBatch], v1[kBatch];
        float M = t.m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int k = k0 + j * kGroups;
            m[j] = -INFINITY;
            if (k >= n) continue;
            const float* part = p.ws + (size_t)(k == 0 ? slot0 : c0 + k) * kPartFloats;
            m[j] = part[kRows * kD + r];
            lr[j] = part[kRows * kD + kRows + r];
            le[j] = part[kRows * kD + 2 * kRows + r];
            v0[j] = *reinterpret_cast<const float4*>(part + (q0 * kRows + r) * 4);
            v1[j] = *reinterpret_cast<const float4*>(part + ((q0 + 1) * kRows + r) * 4);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            M = fmaxf(M, m[j]);
        t.rescale(M);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            // a part without keys of the row (m = -inf) left nothing to read in O
            if (m[j] == -INFINITY) continue;
            const float w = exp2f(m[j] - M);
            t.lr += w * lr[j];
            t.le += w * le[j];
            t.o[0] = fmaf(w, v0[j].x, t.o[0]);
            t.o[1] = fmaf(w, v0[j].y, t.o[1]);
            t.o[2] = fmaf(w, v0[j].z, t.o[2]);
            t.o[3] = fmaf(w, v0[j].w, t.o[3]);
            t.o[4] = fmaf(w, v1[j].x, t.o[4]);
            t.o[5] = fmaf(w, v1[j].y, t.o[5]);
            t.o[6] = fmaf(w, v1[j].z, t.o[6]);
            t.o[7] = fmaf(w, v1[j].w, t.o[7]);
        }
    }
    if (grp > 0) {
        float(*d)[kRows] = sh[grp - 1];
        d[0][r] = t.m;
        d[1][r] = t.lr;
        d[2][r] = t.le;
#pragma unroll
        for (int i = 0; i < kJoinCols; ++i) d[3 + i][r] = t.o[i];
    }
    if (kGroups > 1) __syncthreads();
    if (grp > 0 || orow >= (long)p.R << p.hshift) return;
    float M = t.m;
#pragma unroll
    for (int j = 0; j < kGroups - 1; ++j) M = fmaxf(M, sh[j][0][r]);
    t.rescale(M);
#pragma unroll
    for (int j = 0; j < kGroups - 1; ++j) {
        const float mk = sh[j][0][r];
        if (mk == -INFINITY) continue;
        const float w = exp2f(mk - M);
        t.lr += w * sh[j][1][r];
        t.le += w * sh[j][2][r];
#pragma unroll
        for (int i = 0; i < kJoinCols; ++i) t.o[i] = fmaf(w, sh[j][3 + i][r], t.o[i]);
    }
    const float inv = (t.lr == 0.0f) ? 0.0f : 1.0f / t.lr;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(t.o[2 * i + 1] * inv), "f"(t.o[2 * i] * inv));
    *reinterpret_cast<uint4*>(p.out + orow * kD + q0 * 4) = make_uint4(w[0], w[1], w[2], w[3]);
    if (LSE && q0 == 0) p.lse[orow] = (t.le == 0.0f) ? -INFINITY : (M + log2f(t.le)) / kLog2e;
}

// ---------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn_prefix() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

// 2D bf16 tensor [rows, 128] with a 128-byte-swizzled box of {64, 64}.
bool make_map_prefix(CUtensorMap* m, const void* ptr, uint64_t rows) {
    auto fn = encode_fn_prefix();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
    cuuint32_t box[2] = {64, 64};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Units and CTAs of a call, from its sizes alone.
struct Plan {
    int R, U, n_cta, parts;              // parts of a unit, at most
};
Plan plan_of(const AttnArgs& a) {
    Plan p;
    p.R = a.B * a.n_q;
    const int per = kRows / a.H;                         // query rows of a unit
    p.U = (p.R + per - 1) / per;
    // a unit's tiles, at most: shared and own
    const long own = (std::min<long>(kBN, a.N_p) + a.N_cap + a.window + a.H - 1) / a.H;
    const long T = std::max<long>(a.N_p / kBN + own, 1);
    if (p.U > kSms * (kMaxUnits - 2)) {
        // several waves: whole units for every CTA (those behind the last row are empty), so
        // no parts to join, and no workspace that grows with the rows
        p.n_cta = (p.U + kSms * (kMaxUnits - 2) - 1) / (kSms * (kMaxUnits - 2)) * kSms;
        p.U = (p.U + p.n_cta - 1) / p.n_cta * p.n_cta;
    } else if (p.U >= kSms) {
        p.n_cta = kSms;
    } else {
        // as many whole cuts of every unit as fit one wave, no cut below one
        // tile; or an uneven cut over all SMs, whose CTAs meet two units and
        // flush O twice (about 3 tiles' time), where that is still shorter
        const long S = std::min<long>(kSms / p.U, T);
        p.n_cta = (int)(p.U * S);
        const double even = (double)((T + S - 1) / S), uneven = (double)T * p.U / kSms + 4.0;
        if (uneven < even) p.n_cta = kSms;
    }
    p.parts = (p.n_cta + p.U - 1) / p.U + 1;
    return p;
}

}  // namespace

// Served by the tensor-core kernel: bf16, 64 or 128 heads of 128.
bool attention_prefix_tc_supported(const AttnArgs& a) {
    return a.dt == DT_BF16 && a.D == kD && (a.H == 64 || a.H == 128) && (long)a.B * a.n_q * a.H < (1L << 31);
}

unsigned long long attention_prefix_tc_workspace(const AttnArgs& a) {
    const Plan pl = plan_of(a);
    if (pl.n_cta <= pl.U && pl.U % pl.n_cta == 0) return 0;          // no unit is cut
    // (every unit cut alike: no CTA has two)
    return (unsigned long long)pl.n_cta * (pl.n_cta % pl.U ? 2 : 1) * kPartFloats * sizeof(float);
}

cudaError_t launch_attention_prefix_tc(const AttnArgs& a, void* workspace, uint32_t* err, cudaStream_t s) {
    const Plan pl = plan_of(a);
    CUtensorMap tm_q, tm_p, tm_c, tm_w;
    // (a tensor without rows is never loaded: any valid address)
    const auto map = [&](CUtensorMap* m, const void* ptr, long n) {
        return make_map_prefix(m, n > 0 ? ptr : a.q, n > 0 ? (uint64_t)n : 1);
    };
    if (!map(&tm_q, a.q, (long)pl.R * a.H) || !map(&tm_p, a.kv_p, a.N_p) || !map(&tm_c, a.kv_c, (long)a.B * a.N_cap) ||
        !map(&tm_w, a.kv_raw, (long)a.B * a.L_raw))
        return cudaErrorInvalidValue;
    PrefixParams p;
    p.kv_p = static_cast<const __nv_bfloat16*>(a.kv_p);
    p.kv_c = static_cast<const __nv_bfloat16*>(a.kv_c);
    p.kv_raw = static_cast<const __nv_bfloat16*>(a.kv_raw);
    p.a = a;
    p.hshift = a.H == 64 ? 6 : 7;
    p.R = pl.R;
    p.U = pl.U;
    p.scale_log2 = a.scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse_out;
    p.ws = static_cast<float*>(workspace);
    p.err = err;
    p.wait_ns = wait_limit_ns();
    p.stall = take_stall();
    const bool cut = attention_prefix_tc_workspace(a) > 0;
    const bool lse = a.lse_out != nullptr;
    auto kern = a.H == 64 ? (lse ? attn_prefix_kernel<2, true> : attn_prefix_kernel<2, false>)
                          : (lse ? attn_prefix_kernel<1, true> : attn_prefix_kernel<1, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, (unsigned)pl.n_cta, kThreads, kSmem, s, tm_q, tm_p, tm_c, tm_w, p);
    count_launch();
    if (e != cudaSuccess || !cut) return e;
    // (A dependent launch whose start nothing triggers before the parts are written: it
    // only spares the gap between the two, 41.1 -> 39.9 us a call for 101 units issued one
    // after the other.  Triggered early, its waiting CTAs cost the call 6 us.  With four
    // threads a row throughout, one CTA fills an SM, and 101 units of 2 to 3 parts took
    // 20 us.)
    const unsigned grid = (unsigned)((pl.U > pl.n_cta ? pl.n_cta - 1 : pl.U) * (kD / kJoinCols));
    const unsigned threads = pl.parts > 5 ? 4 * kRows : kRows;
    const auto join = pl.parts > 5 ? (lse ? prefix_join_kernel<true, 4, 5> : prefix_join_kernel<false, 4, 5>)
                                   : (lse ? prefix_join_kernel<true, 1, 3> : prefix_join_kernel<false, 1, 3>);
    e = launch_dependent(join, grid, threads, 0, s, p, pl.n_cta);
    if (e != cudaSuccess) return e;
    count_launch();
    return cudaGetLastError();
}

}  // namespace csa
