// entry_weights_tc.cu -- the attention weight each compressed entry received, on
// tcgen05 (see entry_weights.cu for the definition).
//
// The keys are the MMA's M: z^T = K.Q^T puts one key's scores against 128
// (query row, head) columns into one TMEM lane, so a thread adds the weights of
// one key over its columns in registers: no cross-lane sums, no atomics, and a
// key that no row sees can hold anything, since it touches its own lane only.
// Work item: 128 entries (or list slots) of one element, all columns in steps of
// 128 (where a cluster shares an item, a run of the steps a CTA).  Persistent, one CTA
// per SM; item i is tile i / B of element i mod B, so the
// tiles past the elements' ends come last and cost nothing.
// Roles (24 warps): warp 0 loads Q and the entries' tiles (TMA); warps 1-2 stage
// the columns' lse and reach; warps 3-6 gather listed entries row by row
// (cp.async); warp 7 issues the MMAs; warps 8-23 add the weights, four threads a
// key.  (One group of warps for all loads took 1800 cycles a step, most
// of it waiting for its own instructions and lse, and 8 warps for the sums left
// tensor-memory loads and exponentials one after the other: 47 us for 64 query
// rows over 16384 entries.)
// What bounds it: decode (one step an item) reads every key once, HBM; with many
// query rows the exponentials, 1024 MUFU cycles a step against 512 of the tensor
// pipe.  mma.sync ran at 150 TFLOP/s here, three times both bounds.
#include <cudaTypedefs.h>

#include <math.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tc;

constexpr int kD = 128;
constexpr int kKeys = 128;                  // entries of an item
constexpr int kCols = 128;                  // columns of a step
constexpr int kKBufs = 3, kStages = 3, kBufs = 4;
constexpr int kHalf = 16384;                // 64 channels of 128 rows
constexpr int kTileBytes = 2 * kHalf;
constexpr int kTmaWarp = 0, kColWarp0 = 1, kColWarps = 2, kGatherWarp0 = 3, kGatherWarps = 4;
constexpr int kMmaWarp = 7, kSumWarp0 = 8;
constexpr int kGatherThreads = kGatherWarps * 32;
constexpr int kQuarters = 4, kSumWarps = 4 * kQuarters;
constexpr int kThreads = (kSumWarp0 + kSumWarps) * 32;
constexpr int kNe = 1024;                   // elements whose entry count is kept in shared memory
constexpr int kSms = 148;
constexpr int kXs = 8;                      // items whose other quarters' sums may wait
constexpr int kCx = 24, kRounds = 8;         // a cluster's sums that may wait; its items, at most
constexpr float kLog2e = 1.4426950408889634f;

struct __align__(16) Ctrl {
    float nlse[kBufs][kCols];               // -lse * log2(e) of the step's columns
    int vis[kBufs][kCols];                  // entries the column's row sees (0: no column, empty row)
    int low[kBufs][kCols / 32];             // all of them, by 32 columns; -1: they differ
    int ne[kNe];                            // the elements' entries
    float xs[kXs][kQuarters - 1][kKeys];    // the other quarters' sums
    uint64_t full[kStages], freeb[kStages];        // Q
    uint64_t kfull[kKBufs], kfree[kKBufs];
    uint64_t s_full[kBufs], s_free[kBufs];         // scores, and the columns' lse and reach
    float cx[kCx][kKeys];                   // the other CTAs' sums (in the cluster's first)
    uint64_t x_full[kXs], c_full[kRounds];
    uint64_t fin, stall_bar;     // (stall_bar: a barrier that nothing completes, for tests)
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kSmem = 1024 + (kKBufs + kStages) * kTileBytes + sizeof(Ctrl);

struct TcWeights {
    WeightsArgs a;
    int items, steps, cols;
    int cshift;                  // log2 of a cluster's CTAs
    int hshift, mshift;          // log2 of H and m where they are powers of two, else -1
    int qbox;                    // Q rows a TMA copy brings: 64 where no step has more columns, else 128
    float sl2;
    uint32_t* err;
    uint64_t wait_ns;
    int stall;                   // test hook: the MMA warp waits on stall_bar first
};

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                       uint64_t limit_ns) {
    return mbar_wait(bar, parity, abort, err, limit_ns);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// The rows of a map's box from row y on, both 64-column halves.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* m, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(y), "r"(0), "r"(smem_u32(bar))
        : "memory");
}
// (within 2^-22 of itself, below 2^-126 as 0: less than the scores' own rounding)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// Sum of exp2(z * sl2 + nlse) over N columns of this thread's TMEM lane.
template <int N>
__device__ __forceinline__ float sum_columns(uint32_t taddr, const float* nlse, uint64_t sl2) {
    float z[N];
    if constexpr (N == 32) tmem_ld32(taddr, z);
    else tmem_ld16(taddr, z);
    uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(nlse + e);
        const uint64_t x0 = f2_fma(f2_pack(z[e], z[e + 1]), sl2, f2_pack(l.x, l.y));
        const uint64_t x1 = f2_fma(f2_pack(z[e + 2], z[e + 3]), sl2, f2_pack(l.z, l.w));
        acc0 = f2_add(acc0, f2_pack(ex2(f2lo(x0)), ex2(f2hi(x0))));
        acc1 = f2_add(acc1, f2_pack(ex2(f2lo(x1)), ex2(f2hi(x1))));
    }
    acc0 = f2_add(acc0, acc1);
    return f2lo(acc0) + f2hi(acc0);
}

__device__ __forceinline__ int entries_of(const WeightsArgs& a, int b) {
    return clampi(a.n_entries ? __ldg(a.n_entries + b) : a.N_cap, 0, a.N_cap);
}
// A CTA's items, `width` apart (dchunk tiles and db elements): tile i / B of element i mod B.
struct Walk {
    int first, width, dchunk, db;
};
__device__ __forceinline__ Walk walk_of(const TcWeights& p, int shared) {
    Walk w;
    w.first = (int)blockIdx.x >> shared;
    w.width = (int)gridDim.x >> shared;
    w.dchunk = w.width / p.a.B;
    w.db = w.width - w.dchunk * p.a.B;
    return w;
}
struct Item {
    int i, b, chunk, ne;
    bool live;               // some key of it can be seen
};
__device__ __forceinline__ void look(const TcWeights& p, const int* ne, Item& t) {
    t.ne = 0;
    if (t.i < p.items) t.ne = t.b < kNe ? ne[t.b] : entries_of(p.a, t.b);
    t.live = p.a.idx ? t.ne > 0 : t.chunk * kKeys < t.ne;
}
__device__ __forceinline__ Item first_item(const TcWeights& p, const Walk& w, const int* ne) {
    Item t;
    t.i = w.first;
    t.chunk = t.i / p.a.B;
    t.b = t.i - t.chunk * p.a.B;
    look(p, ne, t);
    return t;
}
__device__ __forceinline__ void next_item(const TcWeights& p, const Walk& w, const int* ne, Item& t) {
    t.i += w.width;
    t.chunk += w.dchunk;
    t.b += w.db;
    if (t.b >= p.a.B) {
        t.b -= p.a.B;
        ++t.chunk;
    }
    look(p, ne, t);
}

// This address in another CTA of the cluster; a store and an arrival there.
__device__ __forceinline__ uint32_t peer_addr(const void* local, int rank) {
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(local)), "r"(rank));
    return d;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// By every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// kOne: items of one step.  kCluster: the 2^cshift CTAs of a cluster share an item, a run
// of its steps each; their sums meet in the first CTA's shared memory, in the CTAs' order.
template <bool kOne, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1)
weights_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ TcWeights p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = base;                                  // [kKBufs][32 KB]
    uint8_t* sQ = sK + kKBufs * kTileBytes;              // [kStages][32 KB]
    Ctrl* ctl = reinterpret_cast<Ctrl*>(sQ + kStages * kTileBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort = &ctl->abort;
    const WeightsArgs& a = p.a;
    auto try_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, p.err, p.wait_ns);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {       // by a whole warp
        return __all_sync(0xffffffffu, try_wait(bar, parity));
    };

    grid_wait();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->freeb[i], 1);
        }
        for (int i = 0; i < kKBufs; ++i) {
            mbar_init(&ctl->kfull[i], a.idx ? kGatherThreads : 1);
            mbar_init(&ctl->kfree[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&ctl->s_full[i], 1 + kColWarps);
            mbar_init(&ctl->s_free[i], kOne ? kSumWarps / 2 : kSumWarps);
        }
        for (int i = 0; i < kXs; ++i) mbar_init(&ctl->x_full[i], kOne ? 4 : kSumWarps - 4);
        for (int i = 0; i < kRounds; ++i) mbar_init(&ctl->c_full[i], kCluster ? 4 * ((1 << p.cshift) - 1) : 1);
        mbar_init(&ctl->fin, 1);
        mbar_init(&ctl->stall_bar, 1);
        // a CTA started after another one timed out does no work
        ctl->abort = (*reinterpret_cast<volatile uint32_t*>(p.err) != 0u) ? 1 : 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem_base, kBufs * kCols);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < min(a.B, kNe); i += kThreads) ctl->ne[i] = entries_of(a, i);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
    if (kCluster) cluster_meet();                        // (the peers' barriers are there, too)
    const int shared = kCluster ? p.cshift : 0;
    const int rank = (int)blockIdx.x & ((1 << shared) - 1);
    const int s_lo = rank * p.steps >> shared, s_hi = (rank + 1) * p.steps >> shared;        // the CTA's steps
    const Walk walk = walk_of(p, shared);

    // the CTA's live items
    const auto first_live = [&]() -> Item {
        Item t = first_item(p, walk, ctl->ne);
        while (t.i < p.items && !t.live) next_item(p, walk, ctl->ne, t);
        return t;
    };
    const auto next_live = [&](Item& t) {
        do next_item(p, walk, ctl->ne, t);
        while (t.i < p.items && !t.live);
    };
    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA: tiles and Q
        int k = 0, L = 0;                    // live items, steps
        bool ok = true;
        for (Item t = first_live(); t.i < p.items && ok; next_live(t), ++k) {
            if (!a.idx) {
                const int kb = k % kKBufs;
                if (k >= kKBufs) ok = wait(&ctl->kfree[kb], (k / kKBufs - 1) & 1);
                ok = __all_sync(0xffffffffu, ok && !*abort);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctl->kfull[kb], kTileBytes);
                    const int y = t.b * a.N_cap + t.chunk * kKeys;
                    tma_load_rows(sK + kb * kTileBytes, &tm_k, y, &ctl->kfull[kb]);
                }
                __syncwarp();
            }
            for (int st = s_lo; st < s_hi; ++st, ++L) {
                const int sl = L % kStages;
                if (L >= kStages) ok = wait(&ctl->freeb[sl], (L / kStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok && !*abort);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&ctl->full[sl], 2 * 128 * p.qbox);
                    tma_load_rows(sQ + sl * kTileBytes, &tm_q, t.b * p.cols + st * kCols, &ctl->full[sl]);
                }
                __syncwarp();
            }
        }
        // loads in flight land before the CTA's shared memory is given up
        volatile int never = 0;
        for (int q = 0; q < kStages; ++q)
            if (L > q) mbar_wait(&ctl->full[q], ((L - 1 - q) / kStages) & 1, &never, p.err);
        for (int q = 0; q < kKBufs; ++q)
            if (!a.idx && k > q) mbar_wait(&ctl->kfull[q], ((k - 1 - q) / kKBufs) & 1, &never, p.err);
        __syncwarp();
    } else if (warp < kColWarp0 + kColWarps) {
        // ------------------------------------------------------------ the columns
        // Two columns a thread.  What a step needs is asked for one step ahead, into
        // registers that the next step uses in place (two sets, taken in turn).
        const int cw = warp - kColWarp0;
        struct Col {
            float lse[2];
            int pos[2];
            int ne;
        };
        const auto fetch = [&](const Item& t, int st) -> Col {
            Col c;
            c.ne = t.ne;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = st * kCols + 64 * cw + 32 * e + lane;
                c.lse[e] = 0.0f;
                c.pos[e] = -1;
                if (at < p.cols) {
                    const int qi = p.hshift >= 0 ? at >> p.hshift : at / a.H;
                    c.pos[e] = a.q_pos ? __ldg(a.q_pos + (size_t)t.b * a.n_q + qi) : qi;
                    c.lse[e] = __ldg(a.lse + (size_t)t.b * p.cols + at);
                }
            }
            return c;
        };
        int L = 0;
        bool ok = true;
        const auto put = [&](const Col& col) -> bool {
            const int sl = L % kBufs;
            if (L >= kBufs) ok = wait(&ctl->s_free[sl], (L / kBufs - 1) & 1);
            if (!ok) return false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float l = -col.lse[e] * kLog2e;
                const unsigned n = (unsigned)col.pos[e] + 1u;
                const int vis = (col.pos[e] < 0 || l == INFINITY) ? 0 : (int)min(p.mshift >= 0 ? n >> p.mshift : n / (unsigned)a.m, (unsigned)col.ne);
                ctl->nlse[sl][64 * cw + 32 * e + lane] = l;
                ctl->vis[sl][64 * cw + 32 * e + lane] = vis;
                const int low = __reduce_min_sync(0xffffffffu, vis), high = __reduce_max_sync(0xffffffffu, vis);
                if (lane == 0) ctl->low[sl][2 * cw + e] = low == high ? low : -1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->s_full[sl]);
            ++L;
            return true;
        };
        Item t = first_live();
        int st = s_lo;
        const auto advance = [&]() {
            if (++st == s_hi) {
                st = s_lo;
                next_live(t);
            }
        };
        Col c0, c1;
        if (t.i < p.items) c0 = fetch(t, st);
        while (t.i < p.items) {
            advance();
            const bool more = t.i < p.items;
            if (more) c1 = fetch(t, st);
            if (!put(c0) || !more) break;
            advance();
            if (t.i < p.items) c0 = fetch(t, st);
            if (!put(c1)) break;
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ listed entries
        // 16 lanes a row (an entry that is not in the cache: its first row, which the sums
        // leave out).  An item's copies are handed over once the next item's are under way.
        const int lt = threadIdx.x - kGatherWarp0 * 32, c16 = lt & 15;
        int pend = -1;
        const auto settle = [&](bool all) {
            if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
            else asm volatile("cp.async.wait_group 1;" ::: "memory");
            if (pend >= 0) {
                fence_proxy_async_smem();
                mbar_arrive(&ctl->kfull[pend]);
                pend = -1;
            }
        };
        int k = 0;
        bool ok = true;
        Item t = first_live();
        for (; a.idx && t.i < p.items && ok; ++k) {
            const int kb = k % kKBufs;
            constexpr int kPasses = kKeys * 16 / kGatherThreads;
            int ent[kPasses];
#pragma unroll
            for (int it = 0; it < kPasses; ++it) {
                const int j = t.chunk * kKeys + it * (kGatherThreads / 16) + (lt >> 4);
                ent[it] = j < a.topk ? __ldg(a.idx + (size_t)t.b * a.topk + j) : 0;
            }
            const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv_c) + (size_t)t.b * a.N_cap * kD + c16 * 8;
            next_live(t);
            if (k >= kKBufs) ok = wait(&ctl->kfree[kb], (k / kKBufs - 1) & 1);
            ok = __all_sync(0xffffffffu, ok && !*abort);
            if (!ok) break;
            uint8_t* dk = sK + kb * kTileBytes + (c16 >> 3) * kHalf;
#pragma unroll
            for (int it = 0; it < kPasses; ++it) {
                const int r = it * (kGatherThreads / 16) + (lt >> 4), s = (ent[it] >= 0 && ent[it] < a.N_cap) ? ent[it] : 0;
                cp_async16(dk + r * 128 + (((c16 & 7) ^ (r & 7)) << 4), kv + (size_t)s * kD);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            settle(false);
            pend = kb;
        }
        settle(true);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ z^T = K.Q^T
        const uint64_t kd0 = sw128_desc(smem_u32(sK), 16, 1024), qd0 = sw128_desc(smem_u32(sQ), 16, 1024);
        int k = 0, L = 0;
        bool ok = !p.stall || wait(&ctl->stall_bar, 0);
        for (Item t = first_live(); t.i < p.items && ok; next_live(t)) {
            const int kb = k % kKBufs;
            ok = wait(&ctl->kfull[kb], (k / kKBufs) & 1);
            for (int st = s_lo; st < s_hi && ok; ++st, ++L) {
                const int sl = L % kStages, buf = L % kBufs;
                ok = (L < kBufs || wait(&ctl->s_free[buf], (L / kBufs - 1) & 1)) && wait(&ctl->full[sl], (L / kStages) & 1);
                if (!ok) break;
                tc_fence_after();
                const int n = min(kCols, (p.cols - st * kCols + 15) & ~15);
                const uint32_t id = idesc_bf16(kKeys, kCols, false, false) - ((uint32_t)((kCols - n) >> 3) << 17);
                const uint64_t kd = kd0 + (uint64_t)(kb * (kTileBytes >> 4)), qd = qd0 + (uint64_t)(sl * (kTileBytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint32_t off = (kk & 3) * 32;
                        mma_bf16_ss(tmem + buf * kCols, kd + (((kk >> 2) * kHalf + off) >> 4),
                                    qd + (((kk >> 2) * 128 * p.qbox + off) >> 4), id, kk > 0);
                    }
                    mma_commit(&ctl->freeb[sl]);
                    mma_commit(&ctl->s_full[buf]);
                    if (st + 1 == s_hi) mma_commit(&ctl->kfree[kb]);
                }
                __syncwarp();
            }
            ++k;
        }
        if (elect_one()) mma_commit(&ctl->fin);
        __syncwarp();
        volatile int never = 0;
        mbar_wait(&ctl->fin, 0, &never, p.err);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ weights and sums
        // Four threads a key.  Items of several steps: each takes a quarter of every
        // step's columns.  Items of one step: every other item, half of its columns
        // (the waits and meetings an item costs overlap the other half's work:
        // decode of 16 x 8192 entries takes 9.3 us, in quarters 10.3).
        const int h = (warp - kSumWarp0) >> 2;
        constexpr int share = kOne ? 2 : kQuarters;
        const int part_of = h & (share - 1);
        const int r = (warp & 3) * 32 + lane;                // key of the item
        const uint32_t my = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint64_t sl2 = f2_pack(p.sl2, p.sl2);
        int k = 0, L = 0;
        bool ok = true;
        // an item's entry of this thread, and what it had (asked for one item ahead)
        const auto entry = [&](const Item& t, float* had) -> int {
            const int j = t.chunk * kKeys + r;
            int s = a.idx ? (j < a.topk ? __ldg(a.idx + (size_t)t.b * a.topk + j) : -1) : j;
            if (s < 0 || s >= a.N_cap) s = -1;
            *had = 0.0f;
            if (part_of == 0 && rank == 0 && !a.idx && s >= 0 && a.in) *had = a.in[(size_t)t.b * a.N_cap + s];
            return s;
        };
        Item tn = first_item(p, walk, ctl->ne);
        float had_n = 0.0f;
        int s_n = tn.i < p.items ? entry(tn, &had_n) : -1;
        while (tn.i < p.items && ok) {
            const Item t = tn;
            const int s = s_n;
            const float had = had_n;
            float* dst = a.out + (size_t)t.b * a.N_cap + s;
            next_item(p, walk, ctl->ne, tn);
            if (tn.i < p.items) s_n = entry(tn, &had_n);
            if (!t.live) {
                if (h == 0 && rank == 0 && !a.idx && s >= 0) *dst = had;
                continue;
            }
            if (kOne && (k & 1) != (h >> 1)) {
                ++k;
                ++L;
                continue;
            }
            float sum = 0.0f;
            for (int st = s_lo; st < s_hi; ++st, ++L) {
                const int buf = L % kBufs;
                // this thread's columns of the step: a quarter or half of 128 or 64
                const int n = min(kCols, (p.cols - st * kCols + 63) & ~63) / share, c0 = n * part_of;
                // every wait is warp-collective: the TMEM accesses below are .sync.aligned
                ok = wait(&ctl->s_full[buf], (L / kBufs) & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = c0; c < (kOne ? c0 + n : c0 + 1); c += 32) {
                    // columns of one query row (or rows that see the same): one test for all
                    const int same = ctl->low[buf][c >> 5];
                    float part = 0.0f;
                    if (n >= 32 && same >= 0) {
                        part = sum_columns<32>(my + buf * kCols + c, &ctl->nlse[buf][c], sl2);
                    } else if (same >= 0) {
                        part = sum_columns<16>(my + buf * kCols + c, &ctl->nlse[buf][c], sl2);
                    } else {
#pragma unroll 1
                        for (int d = c; d < c + min(n, 32); d += 16) {
                            float z[16];
                            tmem_ld16(my + buf * kCols + d, z);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float w = ex2(fmaf(z[e], p.sl2, ctl->nlse[buf][d + e]));
                                if (s < ctl->vis[buf][d + e]) part += w;
                            }
                        }
                    }
                    if (same < 0 || s < same) sum += part;   // (what a key may not add may be NaN)
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->s_free[buf]);
            }
            if (!ok) break;
            // the shares' sums meet.  (The others are at most kBufs steps, so kBufs
            // items, ahead: their slot of xs has been read.)
            if (part_of > 0) {
                ctl->xs[k % kXs][part_of - 1][r] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->x_full[k % kXs]);
            } else {
                ok = wait(&ctl->x_full[k % kXs], (k / kXs) & 1);
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < kQuarters - 1; ++q)
                    if (q < share - 1) sum += ctl->xs[k % kXs][q][r];
                if (kCluster) {
                    const int others = (1 << shared) - 1;
                    if (rank > 0) {
                        peer_store(peer_addr(&ctl->cx[k * others + rank - 1][r], 0), sum);
                        __syncwarp();
                        if (lane == 0) peer_arrive(peer_addr(&ctl->c_full[k], 0));
                        ++k;
                        continue;
                    }
                    ok = wait(&ctl->c_full[k], 0);
                    if (!ok) break;
                    asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    for (int q = 0; q < others; ++q) sum += ctl->cx[k * others + q][r];
                }
                if (s >= 0) {
                    // (an entry listed twice receives its weight twice: equal terms, any order)
                    if (a.idx) atomicAdd(dst, sum);
                    else *dst = had + sum;
                }
            }
            ++k;
        }
    }
    // (the MMA warp waited for its final commit: no MMA is in flight)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (kCluster) cluster_meet();                        // (the first CTA's memory outlives the others' stores)
    if (warp == kMmaWarp) tmem_dealloc(tmem, kBufs * kCols);
}

// ---------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn_weights() {
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

// A bf16 tensor [rows, 128] as {64 channels, rows, 2 halves}, so that one copy brings n
// rows as two 64-column halves, each 128-byte-swizzled (two copies took the loading
// warp twice as long to issue).
bool make_map_weights(CUtensorMap* m, const void* ptr, uint64_t rows, int n) {
    auto fn = encode_fn_weights();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, 2};
    cuuint64_t strides[2] = {(cuuint64_t)kD * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)n, 2};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t cluster_config(int C, int clusters, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(C * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of 2^cshift CTAs that run at once on the current device (0: unknown).
int most_clusters(int cshift) {
    static std::atomic<int> known[64][4];                    // plus one
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (const int k = known[dev][cshift].load(std::memory_order_relaxed)) return k - 1;
    const auto kern = weights_tc_kernel<false, true>;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = cluster_config(1 << cshift, 1, attr);
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[dev][cshift].store(n + 1, std::memory_order_relaxed);
    return n;
}

// log2 of the CTAs that share an item: where the tiles are so few that it saves a quarter
// of the steps, the two or so that meeting costs included.  64 query rows of 64 heads over
// 2048 entries take 13 us, without clusters 27; 64 of 128 heads over 8192 31 and 50.
// (With fewer rounds than that at stake, a full cache of 16384 took 35 us for 28.)
int choose_cluster(int items, int steps) {
    const long plain = (long)((items + kSms - 1) / kSms) * steps;
    long best = plain;
    int shift = 0;
    for (int k = 1; k <= 3 && (1 << k) <= steps; ++k) {
        const int C = 1 << k, n = std::min(most_clusters(k), items);
        if (n <= 0) continue;
        const long rounds = (items + n - 1) / n, cost = rounds * ((steps + C - 1) / C + 2);
        if (rounds > kRounds || rounds * (C - 1) > kCx || cost >= best || 4 * cost > 3 * plain) continue;
        best = cost;
        shift = k;
    }
    return shift;
}

}  // namespace

// Served here: bf16 rows of 128 channels.  (Lists with a single step of columns go
// to the mma.sync kernel, whose many small CTAs hide the gather better: 12.7 us
// against 15.1 for 64 lists of 1999 entries and 64 columns.  With 128 columns either side
// wins: 18.8 us there and 16.3 here for 64 lists of 1999, 8.9 and 9.7 for 16, 8.8 and 9.5 for
// 64 lists of 300.)
bool entry_weights_tc_supported(const WeightsArgs& a) {
    return a.dt == DT_BF16 && a.D == kD && (long)a.B * a.n_q * a.H < (1L << 31) - kCols && a.n_q > 0 &&
           (!a.idx || (long)a.n_q * a.H > kCols);
}

cudaError_t launch_entry_weights_tc(const WeightsArgs& a, uint32_t* err, cudaStream_t s) {
    CUtensorMap tm_k, tm_q;
    TcWeights p;
    p.qbox = a.n_q * a.H <= 64 ? 64 : kCols;
    if (!make_map_weights(&tm_k, a.kv_c, (uint64_t)a.B * a.N_cap, kKeys) ||
        !make_map_weights(&tm_q, a.q, (uint64_t)a.B * a.n_q * a.H, p.qbox))
        return cudaErrorInvalidValue;
    p.a = a;
    p.cols = a.n_q * a.H;
    p.steps = (p.cols + kCols - 1) / kCols;
    const long items = (long)(((a.idx ? a.topk : a.N_cap) + kKeys - 1) / kKeys) * a.B;
    if (items > (1L << 31) - 1 - kSms) return cudaErrorInvalidConfiguration;
    p.items = (int)items;
    p.cshift = a.idx ? 0 : choose_cluster(p.items, p.steps);
    const int C = 1 << p.cshift;
    const int groups = (int)std::min<long>(items, C == 1 ? kSms : most_clusters(p.cshift));
    const auto log2_of = [](int v) { return (v & (v - 1)) ? -1 : 31 - __builtin_clz((unsigned)v); };
    p.hshift = log2_of(a.H);
    p.mshift = log2_of(a.m);
    p.sl2 = a.scale * kLog2e;
    p.err = err;
    p.wait_ns = wait_limit_ns();
    p.stall = take_stall();
    const auto kern = C > 1 ? weights_tc_kernel<false, true> : p.steps == 1 ? weights_tc_kernel<true, false> : weights_tc_kernel<false, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    if (C > 1) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = cluster_config(C, groups, attr);
        cfg.stream = s;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_q, p);
        if (e != cudaSuccess) e = cudaGetLastError();
    } else {
        e = launch_dependent(kern, (unsigned)groups, kThreads, kSmem, s, tm_k, tm_q, p);
    }
    count_launch();
    return e;
}

}  // namespace csa
