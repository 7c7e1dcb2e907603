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
// and sums in the workspace, and a second kernel, launched overlapped, joins
// them in a fixed order.
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
constexpr int kSoftWarp0 = 4;
constexpr int kThreads = 12 * 32;
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kPartFloats = kRows * kD + 3 * kRows;    // O, then m, l_r, l_e of a slot's part

struct __align__(8) Ctrl {
    uint64_t bar_q, q_free;
    uint64_t full[kStages], freeb[kStages];
    uint64_t s_full[2], p_ready[2], o_full[2], o_free[2];
    uint64_t fin, stall_bar;
    uint32_t tmem_base;
    int abort;
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
    int cut;                 // some unit is cut: a join follows
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
    // the first tile of slot s at or after i (hi: none below it)
    __device__ __forceinline__ int next_of(int s, int i, int hi) const {
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
__device__ __forceinline__ void fill_geometry(const PrefixParams& p, int u0, int n, Geo* geo, RowRec* rows) {
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
        Geo g{0, 0, 0, 0};
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
        geo[k] = g;
    }
}

// The part of unit u that CTA c of n takes, as a range of its tile list.
struct Part {
    int lo, hi, ord;         // ord: which of the unit's parts
    bool whole;
};
__device__ __forceinline__ Part part_of(const PrefixParams& p, int c, int n, int u, int T) {
    const long a = (long)c * p.U, b = a + p.U, x = (long)u * n, y = x + n;
    Part r;
    r.lo = (int)((max(a, x) - x) * T / n);
    r.hi = (int)((min(b, y) - x) * T / n);
    r.ord = c - (int)(x / p.U);
    r.whole = a <= x && b >= y;
    return r;
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

// 16-byte copy global -> shared, or 16 zero bytes (nothing is read) when !on.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// Largest S of the row's columns [c_lo, c_hi) (c_lo a multiple of 32; uniform in a warp).
__device__ __noinline__ float row_max(uint32_t s_addr, int c_lo, int c_hi) {
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
    for (int c = c_lo; c < c_hi; c += 32) {
        float sv[32];
        tmem_ld32(s_addr + c, sv);
        if (c_hi < c + 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (c + e >= c_hi) sv[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            mx0 = max3(mx0, sv[e], sv[e + 1]);
            mx1 = max3(mx1, sv[e + 2], sv[e + 3]);
        }
    }
    return fmaxf(mx0, mx1);
}

// The row maximum grew by more than 2^8: rescale the row's O in TMEM.
__device__ __noinline__ void rescale_o(uint32_t o_addr, float alpha) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        float ov[32];
        tmem_ld32(o_addr + q * 32, ov);
#pragma unroll
        for (int i = 0; i < 32; ++i) ov[i] *= alpha;
        tmem_st32(o_addr + q * 32, ov);
    }
    tmem_st_wait();
}

template <int G, bool LSE>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_p,
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
            mbar_init(&ctl->p_ready[i], 4);
            mbar_init(&ctl->o_full[i], 1);
            mbar_init(&ctl->o_free[i], 4);
        }
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
    fill_geometry<G>(p, u0, u1 - u0, geo, rows);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;

    if (warp < kLoadWarps) {
        // ------------------------------------------------------------ key tiles
        const int lt = threadIdx.x, c16 = lt & 15, half = c16 >> 3, cc = c16 & 7;
        int L = 0;                    // tiles handed out
        int pend = -1;                // stage of a copied tile that has not arrived yet
        uint32_t tma_stage = 0;       // stages whose latest tile came by TMA (thread 0's)
        bool ok = true;
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
        for (int u = u0; u < u1 && ok; ++u) {
            const Geo g = geo[u - u0];
            const Part pt = part_of(p, c, n_cta, u, g.total());
            for (int i = pt.lo; i < pt.hi; ++i, ++L) {
                const int slot = L % kStages, use = L / kStages;
                if (use > 0 && !wait_bar(&ctl->freeb[slot], (use - 1) & 1, abort, p.err, p.wait_ns)) { ok = false; break; }
                if (*abort) { ok = false; break; }
                uint8_t* dst = sK + slot * kTileBytes;
                if (i < g.P) {
                    if (lt == 0) {
                        mbar_arrive_expect_tx(&ctl->full[slot], kTileBytes);
                        tma_load_2d(dst, &tm_p, 0, i * kBN, &ctl->full[slot]);
                        tma_load_2d(dst + kHalf, &tm_p, 64, i * kBN, &ctl->full[slot]);
                        tma_stage |= 1u << slot;
                    } else {
                        mbar_arrive(&ctl->full[slot]);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    settle(false);
                } else {
                    if (lt == 0) tma_stage &= ~(1u << slot);
                    const int ms = g.own_slot(i), j0 = g.own_step(i) * H;
                    const RowRec* rec = rows + ((u - u0) * 2 + ms) * G;
#pragma unroll 2
                    for (int rr = lt >> 4; rr < kBN; rr += kLoadThreads / 16) {
                        const int k = rr / H, j = j0 + rr % H;
                        const RowRec rw = rec[k];
                        const __nv_bfloat16* src = p.out;          // any address: nothing is read past the list
                        const int e1 = rw.n_pre, e2 = e1 + rw.n_own, e3 = e2 + rw.n_win;
                        if (j < e1) src = p.kv_p + (size_t)(g.P * kBN + j) * kD;
                        else if (j < e2) src = p.kv_c + ((size_t)rw.b * p.a.N_cap + (j - e1)) * kD;
                        else if (j < e3) src = p.kv_raw + ((size_t)rw.b * p.a.L_raw + rw.win_lo + (j - e2)) * kD;
                        cp_async16_or_zero(dst + half * kHalf + rr * 128 + ((cc ^ (rr & 7)) << 4), src + c16 * 8,
                                           j < e3);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    settle(false);
                    pend = slot;
                }
            }
        }
        settle(true);
        // TMA tiles in flight land before the CTA's shared memory is given up
        if (lt == 0) {
            volatile int never = 0;
            for (int s = 0; s < kStages; ++s)
                if (((tma_stage >> s) & 1u) && L > s)
                    mbar_wait(&ctl->full[s], ((L - 1 - s) / kStages) & 1, &never, p.err);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ Q and every MMA
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            constexpr uint32_t id_qk = idesc_bf16(kRows, kBN, false, false);
            constexpr uint32_t id_pv = idesc_bf16(kRows, kD, false, true);
            int ld0 = 0;                  // tiles of earlier units
            uint32_t pp = 0;              // bit s: parity of slot s's next P
            uint32_t po = 0;              // bit s: parity of slot s's next o_free (once it had a part)
            uint32_t had = 0;             // bit s: slot s had tiles in an earlier part
            int nq = 0;                   // Q loads
            bool ok = true;
            if (p.stall) mbar_wait(&ctl->stall_bar, 0, abort, p.err, p.wait_ns);
            for (int u = u0; u < u1 && ok; ++u) {
                const Geo g = geo[u - u0];
                const Part pt = part_of(p, c, n_cta, u, g.total());
                if (pt.lo >= pt.hi) continue;
                if (*abort || (nq > 0 && !wait_bar(&ctl->q_free, (nq - 1) & 1, abort, p.err, p.wait_ns))) break;
                mbar_arrive_expect_tx(&ctl->bar_q, 2 * kTileBytes);
                for (int s = 0; s < 2; ++s)
                    for (int h = 0; h < 2; ++h)
                        tma_load_2d(sQ + s * kTileBytes + h * kHalf, &tm_q, h * 64, (2 * u + s) * kRows, &ctl->bar_q);
                ++nq;
                ok = wait_bar(&ctl->bar_q, (nq - 1) & 1, abort, p.err, p.wait_ns);
                auto issue_qk = [&](int s, int i) -> bool {
                    const int ld = ld0 + i - pt.lo, slot = ld % kStages;
                    if (!wait_bar(&ctl->full[slot], (ld / kStages) & 1, abort, p.err, p.wait_ns)) return false;
                    tc_fence_after();
                    const uint64_t qd = sw128_desc(smem_u32(sQ + s * kTileBytes), 16, 1024);
                    const uint64_t kd = sw128_desc(smem_u32(sK + slot * kTileBytes), 16, 1024);
#pragma unroll
                    for (int kq = 0; kq < kD / 16; ++kq) {
                        const uint32_t off16 = ((kq >> 2) * kHalf + (kq & 3) * 32) >> 4;
                        mma_bf16_ss(tmem + s * 128, qd + off16, kd + off16, id_qk, kq > 0);
                    }
                    mma_commit(&ctl->s_full[s]);
                    return true;
                };
                // nx0, nx1: the slots' next tiles to multiply with Q
                int nx0 = g.next_of(0, pt.lo, pt.hi), nx1 = g.next_of(1, pt.lo, pt.hi);
                uint32_t first = 3u;
                for (int s = 0; s < 2 && ok; ++s) {
                    const int i = s ? nx1 : nx0;
                    if (i >= pt.hi) continue;
                    ok = issue_qk(s, i);
                    const int nx = g.next_of(s, i + 1, pt.hi);
                    if (s) nx1 = nx;
                    else nx0 = nx;
                }
                if (ok && nx0 >= pt.hi && nx1 >= pt.hi) mma_commit(&ctl->q_free);
                for (int i = pt.lo; i < pt.hi && ok; ++i) {
                    const int m = g.mask(i), slot = (ld0 + i - pt.lo) % kStages;
#pragma unroll 1
                    for (int s = 0; s < 2; ++s) {
                        if (!((m >> s) & 1)) continue;
                        ok = wait_bar(&ctl->p_ready[s], (pp >> s) & 1, abort, p.err, p.wait_ns);
                        pp ^= 1u << s;
                        // the slot's previous O has been read
                        if (ok && ((first & had) >> s & 1)) {
                            ok = wait_bar(&ctl->o_free[s], (po >> s) & 1, abort, p.err, p.wait_ns);
                            po ^= 1u << s;
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = sw128_desc(smem_u32(sK + slot * kTileBytes), kHalf, 1024);
                        const uint32_t fresh = (first >> s) & 1;
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            mma_bf16_ts(tmem + 256 + s * 128, tmem + s * 128 + kk * 8, vd + (uint64_t)(kk * (2048 >> 4)),
                                        id_pv, kk > 0 ? 1u : fresh ^ 1u);
                        first &= ~(1u << s);
                        if ((m >> (s + 1)) == 0) mma_commit(&ctl->freeb[slot]);
                        const int nx = s ? nx1 : nx0;
                        if (nx < pt.hi) {
                            ok = issue_qk(s, nx);
                            if (!ok) break;
                            const int after = g.next_of(s, nx + 1, pt.hi);
                            if (s) nx1 = after;
                            else nx0 = after;
                            if (nx0 >= pt.hi && nx1 >= pt.hi) mma_commit(&ctl->q_free);
                        } else {
                            mma_commit(&ctl->o_full[s]);
                            had |= 1u << s;
                        }
                    }
                }
                ld0 += pt.hi - pt.lo;
            }
            // every MMA must finish before TMEM is released, a Q load in
            // flight must land before shared memory is given up
            mma_commit(&ctl->fin);
            volatile int never = 0;
            mbar_wait(&ctl->fin, 0, &never, p.err);
            if (nq > 0) mbar_wait(&ctl->bar_q, (nq - 1) & 1, &never, p.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and output
        const int s = (warp - kSoftWarp0) >> 2;
        const int r = (warp & 3) * 32 + lane;                // row of the M tile
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + s * 128;
        const uint32_t o_addr = tmem + lane_addr + 256 + s * 128;
        const int grp = r / H;                               // the row's query row in the slot
        int J = 0, kO = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const Geo g = geo[u - u0];
            const Part pt = part_of(p, c, n_cta, u, g.total());
            const int qrow = (2 * u + s) * G + grp;
            const RowRec row = rows[((u - u0) * 2 + s) * G + grp];
            const int own_len = row.n_pre + row.n_own + row.n_win;
            float m_used = -INFINITY, l_r = 0.0f, l_e = 0.0f;
            int n = 0;                                       // tiles of this part
            for (int i = pt.lo; i < pt.hi; ++i) {
                if (!((g.mask(i) >> s) & 1)) continue;
                // columns of this row: all, or [c_lo, c_hi) of its H columns (uniform in a warp)
                int c_lo = 0, c_hi = kBN;
                if (i >= g.P) {
                    c_lo = grp * H;
                    c_hi = c_lo + max(min(own_len - g.own_step(i) * H, H), 0);
                }
                // every wait is warp-collective: the TMEM accesses below are .sync.aligned
                if (!__all_sync(0xffffffffu, wait_bar(&ctl->s_full[s], J & 1, abort, p.err, p.wait_ns))) { ok = false; break; }
                ++J;
                tc_fence_after();
                // One pass with the maximum in use; where a score outgrows it by more
                // than 2^8 (and for a part's first tile) the maximum is raised and the
                // pass repeated -- P is stored only at the end, so S is still there.
                uint32_t pk[64];
                bool seek = n == 0;                          // uniform in the warp
                while (true) {
                    if (seek) {
                        const float mx = row_max(s_addr, c_lo, c_hi) * p.scale_log2;
                        const bool raise = mx > m_used + kRescaleLog2;      // true for a row's first keys
                        float alpha = 1.0f;
                        if (raise) {
                            alpha = (m_used == -INFINITY) ? 0.0f : ex2(m_used - mx);
                            m_used = mx;
                            l_r *= alpha;
                            l_e *= alpha;
                        }
                        // (s_full of this tile was committed after the P.V of the one
                        // before was issued, so that P.V has completed: O is stable)
                        if (n > 0) rescale_o(o_addr, alpha);
                    }
                    const float mm = (m_used == -INFINITY) ? 0.0f : m_used;
                    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2), negm = f2_pack(-mm, -mm);
                    uint64_t accr = 0, acce = 0;
                    float zmax = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (c_lo >= 32 * q + 32 || c_hi <= 32 * q) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[16 * q + e] = 0u;
                            continue;
                        }
                        float sv[32];
                        tmem_ld32(s_addr + 32 * q, sv);
                        if (c_hi < 32 * q + 32) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * q + e >= c_hi) sv[e] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint64_t z = f2_fma(f2_pack(sv[e], sv[e + 1]), sl2, negm);
                            zmax = max3(zmax, f2lo(z), f2hi(z));
                            const float p0 = ex2(f2lo(z)), p1 = ex2(f2hi(z));
                            uint32_t d;
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(p1), "f"(p0));
                            pk[16 * q + (e >> 1)] = d;
                            accr = f2_add(accr, f2_pack(__uint_as_float(d << 16), __uint_as_float(d & 0xffff0000u)));
                            if (LSE) acce = f2_add(acce, f2_pack(p0, p1));
                        }
                    }
                    if (!seek && __any_sync(0xffffffffu, zmax > kRescaleLog2 || (m_used == -INFINITY && zmax > -INFINITY))) {
                        seek = true;
                        continue;
                    }
                    l_r += f2lo(accr) + f2hi(accr);
                    l_e += f2lo(acce) + f2hi(acce);
                    break;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_st16(s_addr + 16 * q, pk + 16 * q);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_ready[s]);
                ++n;
            }
            if (!ok) break;
            // ---------------------------------------------------------- the part's end
            if (n > 0) {
                if (!__all_sync(0xffffffffu, wait_bar(&ctl->o_full[s], kO & 1, abort, p.err, p.wait_ns))) break;
                ++kO;
                tc_fence_after();
            }
            const long orow = (long)(2 * u + s) * kRows + r;         // flattened (row, head)
            const bool row_ok = qrow < p.R;
            if (!row.on) {               // no position: no key, whatever the shared tiles held
                m_used = -INFINITY;
                l_r = l_e = 0.0f;
            }
            if (pt.whole) {
                __nv_bfloat16* dst = p.out + orow * kD;
                const float inv = (l_r == 0.0f) ? 0.0f : 1.0f / l_r;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float ov[32];
                    if (n > 0) tmem_ld32(o_addr + q * 32, ov);
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
                if (LSE && row_ok) p.lse[orow] = (l_e == 0.0f) ? -INFINITY : (m_used + log2f(l_e)) / kLog2e;
            } else {
                // O as [column quad][row] of float4: lanes (rows) are consecutive
                float* ws = p.ws + ((size_t)(u * p.parts + pt.ord) * 2 + s) * kPartFloats;
                if (n > 0) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float ov[32];
                        tmem_ld32(o_addr + q * 32, ov);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(ws + ((q * 8 + (e >> 2)) * kRows + r) * 4) =
                                make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                    }
                }
                ws[kRows * kD + r] = n > 0 ? m_used : -INFINITY;
                ws[kRows * kD + kRows + r] = l_r;
                ws[kRows * kD + 2 * kRows + r] = l_e;
            }
            if (n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->o_free[s]);
            }
        }
    }
    // the join may start its launch; it waits for this grid's end before it reads
    if (p.cut) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (the MMA issuer waited for its final commit: no MMA is in flight)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- join
// One CTA per slot of a cut unit and quarter of its columns: the parts' O and
// sums, brought to the largest maximum, are added in the parts' order.
constexpr int kJoinThreads = 256;
constexpr int kMaxParts = kSms + 1;

template <bool LSE>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ PrefixParams p, int n_cta) {
    extern __shared__ float wgt[];                       // [parts][128] weights
    const int slot = blockIdx.x >> 2, quarter = blockIdx.x & 3;
    const int u = slot >> 1;
    const long x = (long)u * n_cta, y = x + n_cta;
    const int c0 = (int)(x / p.U), n = (int)((y + p.U - 1) / p.U) - c0;      // the unit's parts
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n <= 1) return;                                                     // written whole
    const float* ws = p.ws + ((size_t)u * p.parts * 2 + (slot & 1)) * kPartFloats;
    const size_t stride = 2 * (size_t)kPartFloats;
    const int r = threadIdx.x & 127, hi = threadIdx.x >> 7;
    const long orow = (long)slot * kRows + r;
    float M = -INFINITY, lr = 0.0f, le = 0.0f;
    for (int k = 0; k < n; ++k) M = fmaxf(M, ws[k * stride + kRows * kD + r]);
    for (int k = 0; k < n; ++k) {
        const float* st = ws + k * stride + kRows * kD;
        const float mk = st[r];
        const float w = (mk == -INFINITY) ? 0.0f : exp2f(mk - M);
        if (w != 0.0f) {
            lr += w * st[kRows + r];
            le += w * st[2 * kRows + r];
        }
        if (hi == 0) wgt[k * kRows + r] = w;
    }
    __syncthreads();
    if (orow >= (long)p.R << p.hshift) return;
    const float inv = (lr == 0.0f) ? 0.0f : 1.0f / lr;
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int q0 = quarter * 8 + hi * 4;                 // column quads q0 .. q0 + 3
    for (int k = 0; k < n; ++k) {
        const float w = wgt[k * kRows + r];
        if (w == 0.0f) continue;                         // an empty part's O was not written
        const float4* o = reinterpret_cast<const float4*>(ws + k * stride);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = o[(q0 + i) * kRows + r];
            acc[i].x = fmaf(w, v.x, acc[i].x);
            acc[i].y = fmaf(w, v.y, acc[i].y);
            acc[i].z = fmaf(w, v.z, acc[i].z);
            acc[i].w = fmaf(w, v.w, acc[i].w);
        }
    }
    __nv_bfloat16* dst = p.out + orow * kD + q0 * 4;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        uint32_t w[4];
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(acc[i].y * inv), "f"(acc[i].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[1]) : "f"(acc[i].w * inv), "f"(acc[i].z * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[2]) : "f"(acc[i + 1].y * inv), "f"(acc[i + 1].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[3]) : "f"(acc[i + 1].w * inv), "f"(acc[i + 1].z * inv));
        *reinterpret_cast<uint4*>(dst + i * 4) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (LSE && quarter == 0 && hi == 0) p.lse[orow] = (le == 0.0f) ? -INFINITY : (M + log2f(le)) / kLog2e;
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

// 2D bf16 tensor [rows, 128] with a 128-byte-swizzled box of {64, 128}.
bool make_map_prefix(CUtensorMap* m, const void* ptr, uint64_t rows) {
    auto fn = encode_fn_prefix();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)kBN};
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
    CUtensorMap tm_q, tm_p;
    if (!make_map_prefix(&tm_q, a.q, (uint64_t)pl.R * a.H)) return cudaErrorInvalidValue;
    // (without prefix rows no shared tile is loaded: any valid address)
    if (!make_map_prefix(&tm_p, a.N_p > 0 ? a.kv_p : a.q, a.N_p > 0 ? (uint64_t)a.N_p : 1)) return cudaErrorInvalidValue;
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
    p.cut = cut;
    const bool lse = a.lse_out != nullptr;
    auto kern = a.H == 64 ? (lse ? attn_prefix_kernel<2, true> : attn_prefix_kernel<2, false>)
                          : (lse ? attn_prefix_kernel<1, true> : attn_prefix_kernel<1, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)pl.n_cta, kThreads, kSmem, s>>>(tm_q, tm_p, p);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess || !cut) return e;
    auto join = lse ? prefix_join_kernel<true> : prefix_join_kernel<false>;
    const size_t smem = (size_t)pl.parts * kRows * sizeof(float);
    e = cudaFuncSetAttribute(join, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMaxParts * kRows * sizeof(float)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pl.U * 2 * 4), 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join, p, pl.n_cta);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
