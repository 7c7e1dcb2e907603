// attention_prefix.cu -- tensor-core (tcgen05) HCA attention for a batch whose
// elements share their first N_p compressed entries.
//
// For query row (b, q) at position t, head h (one softmax over the union):
//   keys = logical entries s < min(floor((t+1)/m), n_entries[b])   (kv_p, then kv_c[b])
//          and the raw window rows at [max(0, t-W+1), t]
//   o = sum softmax(scale * q.key) key                  (key = value: shared-KV MQA)
// The shared entries are the same keys for every row of the batch, so they are
// a GEMM over all (row, head) pairs at once: 128 of them are the M of an MMA
// whose B operand, a tile of 128 entries, is loaded once per CTA for two such
// M tiles.  What bounds it: per (row, head, key) the two products take 512
// flops and the weight one exponential, and on an SM both take about the same
// time (1024 cycles for 128 x 128), so tensor pipe and MUFU have to run at
// once; HBM traffic is small (the prefix is read from L2).
//
// Unit of work: 256 consecutive (row, head) pairs = two M tiles ("slots") of
// G = 128 / H query rows each.  Its list of key tiles:
//   - shared tiles: 128 prefix entries that every row of the unit sees, used by
//     both slots, brought by TMA;
//   - own tiles, of one slot: each of its G rows gets H columns, filled with
//     that row's further keys (the rest of the prefix it sees, its own entries,
//     its window) by 16-byte cp.async; the other rows' weights there are zero.
//     Rows past a list's end are zero rows, so nothing a row may not see is
//     ever multiplied, whatever it holds.
// The units' lists are dealt over the CTAs of one wave: CTA c of G takes the
// part [c U / G, (c+1) U / G) of the U units laid end to end, each unit's tiles
// cut in that proportion.  A unit that stays whole is written out by its CTA;
// the parts of a cut one leave their unnormalised O (fp32), running maximum
// and sums in the workspace, and a second kernel joins them in a fixed order.
//
// Roles (12 warps, one CTA per SM): warps 0-2 load key tiles; warp 3 allocates
// TMEM and one lane loads Q (TMA) and issues every MMA; warps 4-7 / 8-11 run the
// softmax of slot 0 / 1, a thread per row.  TMEM: S0 S1 O0 O1, 128 columns each;
// P (bf16) overwrites S.  The two slots alternate: while one's weights are
// computed the tensor pipe runs the other's P.V and next Q.K.
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
constexpr int kRows = 128;                  // rows of an M tile
constexpr int kBN = 128;                    // keys per tile
constexpr int kStages = 4;
constexpr int kHalf = 16384;                // one 64-column half of a 128-row tile
constexpr int kTileBytes = 2 * kHalf;
constexpr int kLoadWarps = 3;
constexpr int kLoadThreads = kLoadWarps * 32;
constexpr int kMmaWarp = kLoadWarps;
constexpr int kSoftWarp0 = 4;                // 8 softmax warps a slot
constexpr int kThreads = (kSoftWarp0 + 16) * 32;
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kRange = 0x1p40f;
constexpr int kPartFloats = kRows * kD + 3 * kRows;    // O, then m, l_r, l_e of a slot's part

struct __align__(8) Ctrl {
    uint64_t bar_q, q_free;
    uint64_t full[kStages], freeb[kStages];
    uint64_t s_full[2], p_ready[2], o_full[2], o_free[2];
    uint64_t pair[2][4];                     // the two warps of a slot's 32 rows meet
    uint64_t fin, stall_bar;
    uint32_t tmem_base;
    int abort;
    int redo[2];             // the slot's last P has a weight out of range: S is made again
    // between the two threads of a row: maximum, sums of rounded / exact weights
    float xm[2][2][kRows];
    float xl[2][2][2][2][kRows];             // (by unit parity)
};

struct PrefixParams {
    const __nv_bfloat16* kv_p;
    const __nv_bfloat16* kv_c;
    const __nv_bfloat16* kv_raw;
    AttnArgs a;              // sizes and per-element arrays
    int hshift;              // log2(H)
    int R;                   // query rows
    int U;                   // units
    int parts;               // workspace slots per unit
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    float* ws;
    uint32_t* err;
    uint64_t wait_ns;
    int stall;
};

// What one query row sees beyond the unit's shared tiles (all in smem, filled
// once by the CTA's threads).
struct RowRec {
    int on;                  // it exists and has a position
    int b;
    int vis;                 // visible logical entries
    int win_lo, n_win;       // raw rows
    int n_pre, n_own;        // further prefix entries, own entries
    int pad;
};
// A unit's tile list: P shared tiles, then the slots' own tiles (T0, T1),
// alternating while both have some.
struct Geo {
    int P, T0, T1;
    int on;                  // bit s: slot s has a row with a position
    // the CTA's part of the list: tiles [lo, hi); the unit's part number; all of it?
    int lo, hi, ord, whole;
    __device__ __forceinline__ int total() const { return P + T0 + T1; }
    __device__ __forceinline__ int own_slot(int i) const {
        const int j = i - P, both = 2 * min(T0, T1);
        return j < both ? (j & 1) : (T0 > T1 ? 0 : 1);
    }
    __device__ __forceinline__ int own_step(int i) const {
        const int j = i - P, lo = min(T0, T1);
        return j < 2 * lo ? (j >> 1) : j - lo;
    }
    // bit s: slot s uses tile i
    __device__ __forceinline__ int mask(int i) const { return i < P ? on : 1 << own_slot(i); }
    // the part's first tile of slot s at or after i (hi: none)
    __device__ __forceinline__ int next_of(int s, int i) const {
        if (i < P) {
            if ((on >> s) & 1) return min(i, hi);
            i = P;
        }
        const int lo = min(T0, T1), both = P + 2 * lo;
        if (i < both) {
            if (((i - P) & 1) != s) ++i;
            if (i < both) return min(i, hi);
        }
        return (s ? T1 : T0) > lo ? min(i, hi) : hi;
    }
};
constexpr int kMaxUnits = 32;            // units a CTA meets, at most

// The CTA's units u0 .. u0 + n - 1: a thread per query row, then one per unit.
template <int G>
__device__ __forceinline__ void fill_geometry(const PrefixParams& p, int c, int n_cta, int u0, int n, Geo* geo,
                                              RowRec* rows) {
    for (int i = threadIdx.x; i < n * 2 * G; i += kThreads) {
        const int row = u0 * 2 * G + i;
        RowRec r{};
        if (row < p.R) {
            r.b = row / p.a.n_q;
            const int t = p.a.q_pos ? __ldg(p.a.q_pos + row) : row - r.b * p.a.n_q;
            if (t >= 0) {
                const RowKeys k = row_keys(p.a, r.b, t);
                r.on = 1;
                r.vis = k.n_comp;
                r.win_lo = k.win_lo;
                r.n_win = k.n_win;
            }
        }
        rows[i] = r;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += kThreads) {
        Geo g{};
        int lo = p.a.N_p;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
            const RowRec& r = rows[k * 2 * G + i];
            if (r.on) {
                lo = min(lo, r.vis);
                g.on |= 1 << (i / G);
            }
        }
        g.P = g.on ? lo / kBN : 0;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
            RowRec& r = rows[k * 2 * G + i];
            if (!r.on) continue;
            r.n_pre = max(min(r.vis, p.a.N_p) - g.P * kBN, 0);
            r.n_own = max(r.vis - p.a.N_p, 0);
            const int T = (r.n_pre + r.n_own + r.n_win + kRows / G - 1) / (kRows / G);
            if (i < G) g.T0 = max(g.T0, T);
            else g.T1 = max(g.T1, T);
        }
        // CTA c takes [c U, (c+1) U) of the line on which unit u is [u n_cta, (u+1) n_cta)
        const long a = (long)c * p.U, b = a + p.U, x = (long)(u0 + k) * n_cta, y = x + n_cta;
        g.lo = (int)((max(a, x) - x) * g.total() / n_cta);
        g.hi = (int)((min(b, y) - x) * g.total() / n_cta);
        g.ord = c - (int)(x / p.U);
        g.whole = a <= x && b >= y;
        geo[k] = g;
    }
}

__device__ __forceinline__ int first_unit(const PrefixParams& p, int c, int n) { return (int)((long)c * p.U / n); }
__device__ __forceinline__ int end_unit(const PrefixParams& p, int c, int n) {
    return (int)(((long)(c + 1) * p.U + n - 1) / n);
}

constexpr size_t kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + sizeof(Ctrl) +
                         kMaxUnits * (sizeof(Geo) + 4 * sizeof(RowRec));

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

// The row maximum grew by more than 2^8: rescale this thread's half of the row's O.
__device__ __noinline__ void rescale_o(uint32_t o_addr, float alpha) {
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
        float ov[32];
        tmem_ld32(o_addr + q * 32, ov);
#pragma unroll
        for (int i = 0; i < 32; ++i) ov[i] *= alpha;
        tmem_st32(o_addr + q * 32, ov);
    }
    tmem_st_wait();
}

template <int G, bool LSE>
__global__ void __maxnreg__(96)
attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_p,
                   const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ PrefixParams p) {
    constexpr int H = kRows / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = base;                                  // [2][32 KB]
    uint8_t* sK = sQ + 2 * kTileBytes;                   // [kStages][32 KB]
    Ctrl* ctl = reinterpret_cast<Ctrl*>(sK + kStages * kTileBytes);
    Geo* geo = reinterpret_cast<Geo*>(ctl + 1);          // [kMaxUnits]
    RowRec* rows = reinterpret_cast<RowRec*>(geo + kMaxUnits);   // [kMaxUnits][2 G]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort = &ctl->abort;
    const int c = blockIdx.x, n_cta = gridDim.x;
    const int u0 = first_unit(p, c, n_cta), u1 = end_unit(p, c, n_cta);

    if (threadIdx.x == 0) {
        mbar_init(&ctl->bar_q, 1);
        mbar_init(&ctl->q_free, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ctl->full[s], kLoadThreads);
            mbar_init(&ctl->freeb[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_ready[i], 8);
            mbar_init(&ctl->o_full[i], 1);
            mbar_init(&ctl->o_free[i], 8);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&ctl->pair[i >> 2][i & 3], 2);
        ctl->redo[0] = ctl->redo[1] = 0;
        mbar_init(&ctl->fin, 1);
        mbar_init(&ctl->stall_bar, 1);
        // a CTA started after another one timed out does no work
        ctl->abort = (*reinterpret_cast<volatile uint32_t*>(p.err) != 0u) ? 1 : 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    fill_geometry<G>(p, c, n_cta, u0, u1 - u0, geo, rows);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;

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
            for (int i = g.lo; i < g.hi; ++i, ++L) {
                const int slot = L % kStages, use = L / kStages;
                if (use > 0 && !wait_bar(&ctl->freeb[slot], (use - 1) & 1, abort, p.err, p.wait_ns)) { ok = false; break; }
                if (*abort) { ok = false; break; }
                uint8_t* dst = sK + slot * kTileBytes;
                uint64_t* bar = &ctl->full[slot];
                // the tile as 128 / N runs of N rows: contiguous rows come by TMA boxes of 64
                const bool shared = i < g.P;
                const int ms = shared ? 0 : g.own_slot(i), j0 = shared ? 0 : g.own_step(i) * H;
                const RowRec* rec = rows + ((u - u0) * 2 + ms) * G;
                bool copies = false;
                uint32_t boxes = 0;
                if (shared) {
                    boxes = 4;
                    if (lt == 0) {
                        mbar_expect_tx(bar, kTileBytes);
                        for (int k = 0; k < 4; ++k)
                            tma_load_2d(dst + (k & 1) * kHalf + (k >> 1) * 8192, &tm_p, (k & 1) * 64, i * kBN + (k >> 1) * 64, bar);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kBN / 64; ++k) {          // 64 rows of the tile
                        const RowRec rw = rec[G == 2 ? k : 0];
                        const int j = j0 + (G == 2 ? 0 : 64 * k);
                        const int e1 = rw.n_win, e2 = e1 + rw.n_pre, e3 = e2 + rw.n_own;
                        // one segment holds all 64 rows: window, rest of the prefix, own entries
                        const bool w = j + 64 <= e1, pre = j >= e1 && j + 64 <= e2, own = j >= e2 && j + 64 <= e3;
                        if (w || pre || own) {
                            boxes += 2;
                            if (lt == 0) {
                                const CUtensorMap* m = w ? &tm_w : (pre ? &tm_p : &tm_c);
                                const int y = w ? rw.b * p.a.L_raw + rw.win_lo + j
                                                : (pre ? g.P * kBN + (j - e1) : rw.b * p.a.N_cap + (j - e2));
                                mbar_expect_tx(bar, 2 * 8192);
                                tma_load_2d(dst + k * 8192, m, 0, y, bar);
                                tma_load_2d(dst + kHalf + k * 8192, m, 64, y, bar);
                            }
                            continue;
                        }
                        // row by row, zero rows past the list's end
                        copies = true;
#pragma unroll 1
                        for (int rr = lt >> 4; rr < 64; rr += kLoadThreads / 16) {
                            const int jj = j + rr;
                            const __nv_bfloat16* src = p.out;      // any address: nothing is read past the end
                            if (jj < e1) src = p.kv_raw + ((size_t)rw.b * p.a.L_raw + rw.win_lo + jj) * kD;
                            else if (jj < e2) src = p.kv_p + (size_t)(g.P * kBN + (jj - e1)) * kD;
                            else if (jj < e3) src = p.kv_c + ((size_t)rw.b * p.a.N_cap + (jj - e2)) * kD;
                            cp_async16_or_zero(dst + col + (64 * k + rr) * 128 + (((c16 & 7) ^ (rr & 7)) << 4), src + c16 * 8,
                                               jj < e3);
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
        }
        settle(true);
        // TMA tiles in flight land before the CTA's shared memory is given up
        if (lt == 0) {
            volatile int never = 0;
            for (int k = 0; k < kStages; ++k)
                if (((tma_stage >> k) & 1u) && L > k)
                    mbar_wait(&ctl->full[k], ((L - 1 - k) / kStages) & 1, &never, p.err);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ Q and every MMA
        // The whole warp runs this, kept together by votes, and elect.sync picks the
        // issuing lane: for a branch on the lane number the compiler cannot know
        // that one thread issues, and an MMA took 90 - 120 cycles to issue.
        constexpr uint32_t id_qk = idesc_bf16(kRows, kBN, false, false);
        constexpr uint32_t id_pv = idesc_bf16(kRows, kD, false, true);
        const uint64_t qd0 = sw128_desc(smem_u32(sQ), 16, 1024), kd0 = sw128_desc(smem_u32(sK), 16, 1024);
        const uint64_t vd0 = sw128_desc(smem_u32(sK), kHalf, 1024);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, p.err, p.wait_ns));
        };
        int ld0 = 0;                  // tiles of earlier units
        uint32_t pp = 0;              // bit s: parity of slot s's next P
        uint32_t po = 0;              // bit s: parity of slot s's next o_free (once it had a part)
        uint32_t had = 0;             // bit s: slot s had tiles in an earlier part
        int nq = 0, nfree = 0;        // Q loads; parts whose Q was used up
        bool ok = true;
        if (p.stall) ok = wait(&ctl->stall_bar, 0);
        for (int u = u0; u < u1 && ok; ++u) {
            Geo g = geo[u - u0];
            g.P = __shfl_sync(0xffffffffu, g.P, 0);
            g.T0 = __shfl_sync(0xffffffffu, g.T0, 0);
            g.T1 = __shfl_sync(0xffffffffu, g.T1, 0);
            g.on = __shfl_sync(0xffffffffu, g.on, 0);
            g.lo = __shfl_sync(0xffffffffu, g.lo, 0);
            g.hi = __shfl_sync(0xffffffffu, g.hi, 0);
            if (g.lo >= g.hi) continue;
            if (nfree > 0) ok = wait(&ctl->q_free, (nfree - 1) & 1);
            ok = __all_sync(0xffffffffu, ok && *abort == 0);
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&ctl->bar_q, 2 * kTileBytes);
                for (int k = 0; k < 8; ++k)
                    tma_load_2d(sQ + (k >> 1) * 8192 + (k & 1) * kHalf + (k >> 2) * kHalf, &tm_q, (k & 1) * 64,
                                2 * u * kRows + (k >> 1) * 64, &ctl->bar_q);
            }
            __syncwarp();
            ++nq;
            ok = wait(&ctl->bar_q, (nq - 1) & 1);
            // S of slot s = Q . tile `ld` of the CTA
            auto issue_qk = [&](int s, int ld) -> bool {
                const int slot = ld % kStages;
                if (!wait(&ctl->full[slot], (ld / kStages) & 1)) return false;
                tc_fence_after();
                const uint64_t qd = qd0 + (uint64_t)(s * (kTileBytes >> 4)), kd = kd0 + (uint64_t)(slot * (kTileBytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kq = 0; kq < kD / 16; ++kq) {
                        const uint32_t off16 = ((kq >> 2) * kHalf + (kq & 3) * 32) >> 4;
                        mma_bf16_ss(tm + s * 128, qd + off16, kd + off16, id_qk, kq > 0);
                    }
                    mma_commit(&ctl->s_full[s]);
                }
                __syncwarp();
                return true;
            };
            const int ldx = ld0 - g.lo;               // tile i of the list is the CTA's tile ldx + i
            for (int s = 0; s < 2 && ok; ++s) {
                const int i = g.next_of(s, g.lo);
                if (i < g.hi) ok = issue_qk(s, ldx + i);
            }
            const int dual_end = g.on == 3 ? min(g.P, g.hi) : 0;    // tiles below it serve both slots
            uint32_t first = 3u;
            uint32_t again = 0u;          // bit s: slot s makes its P again
#pragma unroll 1
            for (int i = g.lo, s = 0; i < g.hi && ok;) {
                // slot s's P of tile i: O += P . V, then its next Q . K
                const int m = i < dual_end ? 3 : g.mask(i);
                const bool last = s == 1 || m == 1;   // the tile's last use
                if ((m >> s) & 1) {
                    const int slot = (ldx + i) % kStages;
                    const int nx = i + 1 < dual_end ? i + 1 : g.next_of(s, i + 1);
                    ok = wait(&ctl->p_ready[s], (pp >> s) & 1);
                    pp ^= 1u << s;
                    if (ok && ((first & had) >> s & 1)) {          // the slot's previous O has been read
                        ok = wait(&ctl->o_free[s], (po >> s) & 1);
                        po ^= 1u << s;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    // a weight outgrew the range: S of this tile once more (the warps then
                    // raise the maximum first); answered, the flag goes back
                    if (__shfl_sync(0xffffffffu, *(volatile int*)&ctl->redo[s], 0)) {
                        if (!((again >> s) & 1)) {
                            again |= 1u << s;
                            ok = issue_qk(s, ldx + i);
                            continue;
                        }
                        again &= ~(1u << s);
                        if (lane == 0) *(volatile int*)&ctl->redo[s] = 0;
                        __syncwarp();
                    }
                    const uint64_t vd = vd0 + (uint64_t)(slot * (kTileBytes >> 4));
                    const uint32_t acc = ((first >> s) & 1) ^ 1u;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            mma_bf16_ts(tm + 256 + s * 128, tm + s * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                                        vd + (uint64_t)(kk * (2048 >> 4)), id_pv, kk > 0 ? 1u : acc);
                        if (last) mma_commit(&ctl->freeb[slot]);
                        if (nx >= g.hi) mma_commit(&ctl->o_full[s]);
                    }
                    __syncwarp();
                    first &= ~(1u << s);
                    if (nx < g.hi) {
                        ok = issue_qk(s, ldx + nx);
                    } else {
                        had |= 1u << s;
                    }
                }
                i += last;
                s = last ? 0 : 1;
            }
            if (ok) {
                if (elect_one()) mma_commit(&ctl->q_free);
                __syncwarp();
                ++nfree;
            }
            ld0 += g.hi - g.lo;
        }
        // every MMA must finish before TMEM is released, a Q load in flight
        // must land before shared memory is given up
        if (elect_one()) mma_commit(&ctl->fin);
        __syncwarp();
        volatile int never = 0;
        mbar_wait(&ctl->fin, 0, &never, p.err);
        if (nq > 0) mbar_wait(&ctl->bar_q, (nq - 1) & 1, &never, p.err);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and output
        // A row belongs to two threads, one per 64-column half of S (and of O).
        const int s = (warp - kSoftWarp0) >> 3, h = ((warp - kSoftWarp0) >> 2) & 1;
        const int r = (warp & 3) * 32 + lane;                // row of the M tile
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + s * 128;
        const uint32_t o_addr = tmem + lane_addr + 256 + s * 128 + 64 * h;
        const int grp = r / H;                               // the row's query row in the slot
        // The row's two warps meet (a bounded wait).
        uint32_t px = 0;
        auto pair_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->pair[s][warp & 3]);
            const bool o = __all_sync(0xffffffffu, wait_bar(&ctl->pair[s][warp & 3], px, abort, p.err, p.wait_ns));
            px ^= 1;
            return o;
        };
        volatile int* redo = &ctl->redo[s];
        uint32_t ps = 0, po = 0;                             // parities of s_full, o_full
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const Geo g = geo[u - u0];
            const int qrow = (2 * u + s) * G + grp;
            const RowRec row = rows[((u - u0) * 2 + s) * G + grp];
            const int own_len = row.n_pre + row.n_own + row.n_win;
            // m_used: the maximum in use (base 2); l_r, l_e: this half's sums of the
            // rounded / exact weights, l_r0, l_e0 those before the last tile
            float m_used = -INFINITY, l_r = 0.0f, l_e = 0.0f, l_r0 = 0.0f, l_e0 = 0.0f;
            int n = 0;                                       // tiles of this part
            int nv = 0;
#pragma unroll 1
            for (int i = g.next_of(s, g.lo); i < g.hi;) {
                // (what the tile needs is worked out before the wait for it)
                // this half's columns that are keys of the row (the same in all lanes)
                int nvi = 64;
                if (i >= g.P) {
                    nvi = own_len - g.own_step(i) * H - (G == 1 ? 64 * h : 0);
                    nvi = (G == 2 && h != grp) ? 0 : max(min(nvi, 64), 0);
                }
                int nx = g.next_of(s, i + 1);
                // every wait is warp-collective: the TMEM accesses below are .sync.aligned
                ok = __all_sync(0xffffffffu, wait_bar(&ctl->s_full[s], ps, abort, p.err, p.wait_ns));
                if (!ok) break;
                ps ^= 1;
                tc_fence_after();
                const bool back = *redo != 0;                // the tile before, again
                if (back) {
                    nx = i;
                    l_r = l_r0;
                    l_e = l_e0;
                } else {
                    nv = nvi;
                    l_r0 = l_r;
                    l_e0 = l_e;
                }
                // The maximum of the part's first tile serves the later ones: bf16 and
                // fp32 hold weights up to kRange times it without loss.  A tile with
                // larger ones is made again with the maximum raised first; the last
                // tile, after which S is not made any more, looks for it beforehand.
                const bool seek = back || n == 0 || nx >= g.hi;
                if (seek) {
                    float mx = -INFINITY;
                    if (nv > 0) mx = row_max(s_addr + 64 * h, nv) * p.scale_log2;
                    ctl->xm[s][h][r] = mx;
                    ok = pair_sync();
                    if (!ok) break;
                    // (xm is written again only after the next s_full, which both warps'
                    // p_ready precede)
                    mx = fmaxf(mx, ctl->xm[s][h ^ 1][r]);
                    float alpha = 1.0f;
                    const bool raise = mx > m_used + kRescaleLog2;       // true for a row's first keys
                    if (raise) {
                        alpha = (m_used == -INFINITY) ? 0.0f : ex2(m_used - mx);
                        m_used = mx;
                        l_r *= alpha;
                        l_e *= alpha;
                    }
                    // (s_full of this tile was committed after the P.V of the one
                    // before was issued, so that P.V has completed: O is stable)
                    if (n > 0 && __any_sync(0xffffffffu, raise)) rescale_o(o_addr, alpha);
                }
                // P of this half's 64 keys, over the S it was made from
                bool large = false;
                if (nv > 0) {
                    const float mm = (m_used == -INFINITY) ? 0.0f : m_used;
                    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2), negm = f2_pack(-mm, -mm);
                    uint64_t accr = 0, acce = 0;
                    // (rolled: this much straight-line code would wait for its instructions)
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float sv[32];
                        tmem_ld32(s_addr + 64 * h + 32 * q, sv);
                        if (nv < 64) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * q + e >= nv) sv[e] = -INFINITY;
                        }
                        uint32_t pk[16];
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
                        tmem_st16(s_addr + 64 * h + 16 * q, pk);
                    }
                    const float sum = f2lo(accr) + f2hi(accr);
                    large = !(sum < kRange) || m_used == -INFINITY;      // (no maximum yet: the row's first keys)
                    l_r += sum;
                    l_e += f2lo(acce) + f2hi(acce);
                } else {
                    uint32_t zero[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) zero[e] = 0u;
                    tmem_st16(s_addr + 64 * h, zero);
                    tmem_st16(s_addr + 64 * h + 16, zero);
                }
                if (!seek && __any_sync(0xffffffffu, large)) {
                    if (lane == 0) *redo = 1;
                    __threadfence_block();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_ready[s]);
                n += !back;
                i = nx;
            }
            if (!ok) break;
            // ---------------------------------------------------------- the part's end
            if (n > 0) {
                ok = __all_sync(0xffffffffu, wait_bar(&ctl->o_full[s], po, abort, p.err, p.wait_ns));
                po ^= 1;
                tc_fence_after();
            }
            ctl->xl[u & 1][s][h][0][r] = l_r;
            ctl->xl[u & 1][s][h][1][r] = l_e;
            ok = ok && pair_sync();
            if (!ok) break;
            l_r += ctl->xl[u & 1][s][h ^ 1][0][r];
            l_e += ctl->xl[u & 1][s][h ^ 1][1][r];
            const long orow = (long)(2 * u + s) * kRows + r;         // flattened (row, head)
            const bool row_ok = qrow < p.R;
            if (!row.on) {               // no position: no key, whatever the shared tiles held
                m_used = -INFINITY;
                l_r = l_e = 0.0f;
            }
            if (g.whole) {
                __nv_bfloat16* dst = p.out + orow * kD + 64 * h;
                const float inv = (l_r == 0.0f) ? 0.0f : 1.0f / l_r;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    float ov[32];
                    tmem_ld32(o_addr + q * 32, ov);          // (nothing of it is used without keys)
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (n > 0 && l_r != 0.0f) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k])
                                        : "f"(ov[e + 2 * k + 1] * inv), "f"(ov[e + 2 * k] * inv));
                                v = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            *reinterpret_cast<uint4*>(dst + q * 32 + e) = v;
                        }
                    }
                }
                if (LSE && row_ok && h == 0) p.lse[orow] = (l_e == 0.0f) ? -INFINITY : (m_used + log2f(l_e)) / kLog2e;
            } else {
                // O as [column quad][row] of float4: lanes (rows) are consecutive
                float* ws = p.ws + ((size_t)(u * p.parts + g.ord) * 2 + s) * kPartFloats;
                {
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float ov[32];
                        tmem_ld32(o_addr + q * 32, ov);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(ws + ((h * 16 + q * 8 + (e >> 2)) * kRows + r) * 4) =
                                make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                    }
                }
                if (h == 0) {
                    ws[kRows * kD + r] = n > 0 ? m_used : -INFINITY;
                    ws[kRows * kD + kRows + r] = l_r;
                    ws[kRows * kD + 2 * kRows + r] = l_e;
                }
            }
            if (n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->o_free[s]);
            }
        }
    }
    // (the MMA issuer waited for its final commit: no MMA is in flight)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- join
// A CTA per slot of a cut unit and 8 of its columns; a thread per row and
// quarter of the parts.  What bounds it is the latency of the loads (a few
// parts of L2-resident data), so a thread's parts are fetched at once, 5 at a
// time (a unit is cut into about 10 parts or, alone on the GPU, 20), and the
// four partial results meet in shared memory.  The order of the sums is fixed.
constexpr int kJoinCols = 8;
constexpr int kJoinGroups = 4;
constexpr int kJoinBatch = 5;

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

template <bool LSE>
__global__ void __launch_bounds__(kJoinGroups * kRows)
prefix_join_kernel(const __grid_constant__ PrefixParams p, int n_cta) {
    constexpr int kPer = kD / kJoinCols;
    __shared__ float sh[kJoinGroups - 1][3 + kJoinCols][kRows];
    const int slot = blockIdx.x / kPer, q0 = (blockIdx.x % kPer) * (kJoinCols / 4);
    const int u = slot >> 1, r = threadIdx.x & (kRows - 1), grp = threadIdx.x / kRows;
    const long x = (long)u * n_cta, y = x + n_cta;
    const int c0 = (int)(x / p.U), n = (int)((y + p.U - 1) / p.U) - c0;      // the unit's parts
    if (n <= 1) return;                                                     // written whole
    const long orow = (long)slot * kRows + r;
    const float* ws = p.ws + ((size_t)u * p.parts * 2 + (slot & 1)) * kPartFloats;
    const size_t stride = 2 * (size_t)kPartFloats;
    JoinState t;
    t.m = -INFINITY;
    t.lr = t.le = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) t.o[i] = 0.0f;
    for (int k0 = grp; k0 < n; k0 += kJoinGroups * kJoinBatch) {
        float m[kJoinBatch], lr[kJoinBatch], le[kJoinBatch];
        float4 v0[kJoinBatch], v1[kJoinBatch];
        float M = t.m;
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
            const int k = min(k0 + j * kJoinGroups, n - 1);
            const float* part = ws + k * stride;
            m[j] = part[kRows * kD + r];
            lr[j] = part[kRows * kD + kRows + r];
            le[j] = part[kRows * kD + 2 * kRows + r];
            v0[j] = *reinterpret_cast<const float4*>(part + (q0 * kRows + r) * 4);
            v1[j] = *reinterpret_cast<const float4*>(part + ((q0 + 1) * kRows + r) * 4);
        }
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j)
            if (k0 + j * kJoinGroups < n) M = fmaxf(M, m[j]);
        t.rescale(M);
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
            // a part without keys of the row (m = -inf) left nothing to read in O
            if (k0 + j * kJoinGroups >= n || m[j] == -INFINITY) continue;
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
    __syncthreads();
    if (grp > 0 || orow >= (long)p.R << p.hshift) return;
    float M = t.m;
#pragma unroll
    for (int j = 0; j < kJoinGroups - 1; ++j) M = fmaxf(M, sh[j][0][r]);
    t.rescale(M);
#pragma unroll
    for (int j = 0; j < kJoinGroups - 1; ++j) {
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
    int R, U, n_cta, parts;
};
Plan plan_of(const AttnArgs& a) {
    Plan p;
    p.R = a.B * a.n_q;
    const int per = 2 * kRows / a.H;                     // query rows of a unit
    p.U = (p.R + per - 1) / per;
    // a unit's tiles, at most: shared ones, and each slot's own
    const long own = (std::min<long>(kBN, a.N_p) + a.N_cap + a.window + a.H - 1) / a.H;
    const long T = std::max<long>(a.N_p / kBN + (p.R > per / 2 ? 2 : 1) * own, 1);
    if (p.U >= kSms) {
        p.n_cta = std::max(kSms, (p.U + kMaxUnits - 3) / (kMaxUnits - 2));
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
    return (unsigned long long)pl.U * pl.parts * 2 * kPartFloats * sizeof(float);
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
    p.parts = pl.parts;
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
    kern<<<(unsigned)pl.n_cta, kThreads, kSmem, s>>>(tm_q, tm_p, tm_c, tm_w, p);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess || !cut) return e;
    auto join = lse ? prefix_join_kernel<true> : prefix_join_kernel<false>;
    // (launched in stream order: started early, its waiting CTAs cost the call 6 us)
    join<<<(unsigned)(pl.U * 2 * (kD / kJoinCols)), kJoinGroups * kRows, 0, s>>>(p, pl.n_cta);
    count_launch();
    return cudaGetLastError();
}

}  // namespace csa
