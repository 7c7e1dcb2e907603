// evict.cu -- which entries a compressed cache of a given budget keeps.
//
// Of element b's candidates (s < n_entries[b] with weight[b, s] >= 0) the
// newest `recent` positions come first, newest before older, then the others
// by (weight descending, index ascending); the first `budget` are kept.
// Both orders are one 32-bit key: 0x80000000 + s for a recent candidate, the
// bits of the weight otherwise (non-negative fp32 values order like their
// bits; -0 is taken as +0), so the kept set is an exact radix select of the
// budget-th largest key, ties to the lowest index.
#include "common.cuh"
#include "kernels.h"

namespace csa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// The candidate's key, or false.
__device__ __forceinline__ bool evict_key(float w, int s, int V, int recent, uint32_t* key) {
    if (!(w >= 0.0f) || s >= V) return false;
    *key = (s >= V - recent) ? 0x80000000u + (uint32_t)s : __float_as_uint(w) & 0x7fffffffu;
    return true;
}

__device__ __forceinline__ int block_sum(int v, int* red) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int t = 0;
    for (int i = 0; i < kWarps; ++i) t += red[i];
    return t;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int red[kWarps];
    __shared__ int wgt[kWarps], weq[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* w = a.weight + (size_t)b * a.N_cap;
    const int V = clampi(a.n_entries ? a.n_entries[b] : a.N_cap, 0, a.N_cap);
    int* idx = a.idx_out + (size_t)b * a.budget;

    int c = 0;
    for (int s = tid; s < V; s += kThreads) c += (w[s] >= 0.0f);
    const int total = block_sum(c, red);

    // the budget-th largest key T and how many of its equals are kept
    uint32_t T = 0;
    int need = 0;
    const bool all = total <= a.budget;
    if (!all && a.budget > 0) {
        if (tid == 0) { s_prefix = 0; s_need = a.budget; }
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            const uint32_t pre = s_prefix;
            const uint32_t hi = shift == 24 ? 0u : (0xffffffffu << (shift + 8));
            for (int s = tid; s < V; s += kThreads) {
                uint32_t k;
                if (evict_key(w[s], s, V, a.recent, &k) && (k & hi) == (pre & hi))
                    atomicAdd(&hist[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = s_need, d = 255;
                for (; d > 0 && hist[d] < left; --d) left -= hist[d];
                s_prefix = pre | ((uint32_t)d << shift);
                s_need = left;
            }
            __syncthreads();
        }
        T = s_prefix;
        need = s_need;
    }

    // ordered emission: each warp owns a contiguous span of entries
    const int per = ((V + kWarps - 1) / kWarps + 31) & ~31;
    const int s_lo = min(warp * per, V), s_hi = min(s_lo + per, V);
    int gt = 0, eq = 0;
    for (int s0 = s_lo; s0 < s_hi; s0 += 32) {
        const int s = s0 + lane;
        uint32_t k = 0;
        const bool cand = s < s_hi && evict_key(w[s], s, V, a.recent, &k);
        gt += __popc(__ballot_sync(0xffffffffu, cand && (all || (a.budget > 0 && k > T))));
        eq += __popc(__ballot_sync(0xffffffffu, cand && !all && a.budget > 0 && k == T));
    }
    if (lane == 0) { wgt[warp] = gt; weq[warp] = eq; }
    __syncthreads();
    int g0 = 0, e0 = 0;
    for (int i = 0; i < warp; ++i) { g0 += wgt[i]; e0 += weq[i]; }
    for (int s0 = s_lo; s0 < s_hi; s0 += 32) {
        const int s = s0 + lane;
        uint32_t k = 0;
        const bool in = s < s_hi;
        const bool cand = in && evict_key(w[s], s, V, a.recent, &k);
        const bool isg = cand && (all || (a.budget > 0 && k > T));
        const bool ise = cand && !all && a.budget > 0 && k == T;
        const uint32_t mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
        const uint32_t below = (1u << lane) - 1u;
        const int eb = e0 + __popc(me & below);          // equals of T before this entry
        const bool keep = isg || (ise && eb < need);
        if (keep) idx[g0 + __popc(mg & below) + min(eb, need)] = s;
        else if (in) w[s] = -1.0f;
        g0 += __popc(mg);
        e0 += __popc(me);
    }
    const int kept = min(total, a.budget);
    for (int j = kept + tid; j < a.budget; j += kThreads) idx[j] = -1;
    if (tid == 0 && a.n_kept) a.n_kept[b] = kept;
}

// ------------------------------------------------------------------ registers
// One CTA per element, its keys held in registers: the weights are read once.
// Radix select in digits of 12, 12 and 8 bits: 12 leading bits cut every power of
// two into 16, so the first histogram's atomics spread over its bins; later rounds
// touch only the boundary bin's keys, and end early once the bin has as many keys
// as are still wanted.  What bounds it is instruction issue on the element's one
// SM: sums over warps are taken by a lane a warp, and only the warp that has the
// boundary looks into its bins.  (A cluster of four CTAs an element, summing its
// histograms over distributed shared memory, took 28 us for 64 elements of 32768:
// reading 16 KB from three peers alone was 5 us.)
constexpr int kBins = 4096, kLastBins = 256;

template <int NT, int kPer>
__global__ void __launch_bounds__(NT) evict_regs_kernel(EvictArgs a) {
    constexpr int NW = NT / 32, Q = kBins / NT / 4;          // warps; quads of bins a thread
    __shared__ __align__(16) int hist[2 * kBins + kLastBins];
    __shared__ int wsum[NW];
    __shared__ int found[3];                                 // bin, keys above it, keys in it
    __shared__ int wgt[NW], weq[NW];
    const int b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_wait();
    float* w = a.weight + (size_t)b * a.N_cap;
    const int V = clampi(a.n_entries ? a.n_entries[b] : a.N_cap, 0, a.N_cap);
    int* idx = a.idx_out + (size_t)b * a.budget;
    const int s0 = warp * (32 * kPer) + lane;  // entries s0 + 32 e: a warp's are consecutive
    const bool idle = s0 - lane >= V;                        // the warp has no entry

    // keys plus one; 0: not a candidate
    uint32_t key[kPer];
    uint32_t gone = 0;                                       // bit e: the entry is marked already
#pragma unroll
    for (int e = 0; e < kPer; ++e) key[e] = 0;
    if (!idle) {
        float x[kPer];                                       // all loads in flight
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = s0 + 32 * e < V ? w[s0 + 32 * e] : -1.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            uint32_t k = 0;
            if (evict_key(x[e], s0 + 32 * e, V, a.recent, &k)) key[e] = k + 1;
            gone |= (x[e] == -1.0f ? 1u : 0u) << e;
        }
    }
    for (int i = tid; i < (2 * kBins + kLastBins) / 4; i += NT) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();

    // T: the least key kept (plus one), with the bits below `shift` zero
    uint32_t T = 0;
    int need = a.budget, total = 0;
    bool all = false, ties = false;
    int shift = 20;
#pragma unroll 1
    for (int round = 0;; ++round) {
        int* h = hist + round * kBins;
        const int bins = shift == 0 ? kLastBins : kBins;
        if (!idle) {
            // (the digits' shifts as constants)
            if (round == 0) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (key[e]) atomicAdd(&h[key[e] >> 20], 1);
            } else if (round == 1) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((key[e] ^ T) >> 20 == 0 && key[e]) atomicAdd(&h[key[e] >> 8 & 4095u], 1);
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((key[e] ^ T) >> 8 == 0 && key[e]) atomicAdd(&h[key[e] & 255u], 1);
            }
        }
        __syncthreads();
        // thread t has the 4 Q bins from b0 on; the highest bins are the first thread's
        const int b0 = 4 * Q * (NT - 1 - tid);
        int4 cnt[Q];
        int mine = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            cnt[q] = make_int4(0, 0, 0, 0);
            if (b0 + 4 * q >= bins) continue;
            cnt[q] = *reinterpret_cast<const int4*>(h + b0 + 4 * q);
            mine += cnt[q].x + cnt[q].y + cnt[q].z + cnt[q].w;
        }
        const int of_warp = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) wsum[warp] = of_warp;
        __syncthreads();
        const int ws = lane < NW ? wsum[lane] : 0;
        int above = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
        if (round == 0) {
            total = __reduce_add_sync(0xffffffffu, ws);
            all = total <= a.budget;
            if (all || a.budget == 0) break;
        }
        if (above < need && above + of_warp >= need) {       // this warp's bins have the boundary
            int run = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            above += run - mine;
            if (above < need && above + mine >= need) {
#pragma unroll
                for (int q = Q - 1; q >= 0; --q) {
                    const int v[4] = {cnt[q].w, cnt[q].z, cnt[q].y, cnt[q].x};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (above < need && above + v[j] >= need) {
                            found[0] = b0 + 4 * q + 3 - j;
                            found[1] = above;
                            found[2] = v[j];
                        }
                        above += v[j];
                    }
                }
            }
        }
        __syncthreads();
        T |= (uint32_t)found[0] << shift;
        need -= found[1];
        if (found[2] == need) break;                         // all of the bin
        if (shift == 0) {
            ties = true;                                     // the first `need` of equal keys
            break;
        }
        shift = shift == 20 ? 8 : 0;
    }
    // kept: every candidate; or the keys from T on; or those above T and `need` equals
    const uint32_t from = all ? 1u : (a.budget == 0 ? 0xffffffffu : (ties ? T + 1 : T));
    // lane e gets the bits of the warp's e-th 32 entries: what is kept, and the equals of T
    uint32_t kw = 0, ew = 0;
    if (!idle) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const uint32_t m = __ballot_sync(0xffffffffu, key[e] >= from);
            if (lane == e) kw = m;
        }
        if (ties) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t m = __ballot_sync(0xffffffffu, key[e] == T);
                if (lane == e) ew = m;
            }
        }
    }
    int gt = __popc(kw), eq = __popc(ew);                    // inclusive over the lanes
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, gt, o), y = __shfl_up_sync(0xffffffffu, eq, o);
        if (lane >= o) {
            gt += x;
            eq += y;
        }
    }
    if (lane == 31) {
        wgt[warp] = gt;
        weq[warp] = eq;
    }
    __syncthreads();
    const int gw = lane < warp ? wgt[lane] : 0, qw = lane < warp ? weq[lane] : 0;
    const int g0 = __reduce_add_sync(0xffffffffu, gw) + gt - __popc(kw);
    const int e0 = __reduce_add_sync(0xffffffffu, qw) + eq - __popc(ew);
    if (!idle) {
        if (ties) {                                          // the lane's share of the `need` first equals
            uint32_t left = ew;
            for (int i = e0; i < need && left; ++i) {
                kw |= left & (0u - left);
                left &= left - 1;
            }
        }
        int at = g0 + (ties ? min(e0, need) : 0);
        for (uint32_t m = kw; m; m &= m - 1, ++at)
            if (at < a.budget) idx[at] = (s0 - lane) + 32 * lane + __ffs(m) - 1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const bool kept = ties ? (__shfl_sync(0xffffffffu, kw, e) >> lane & 1u) : key[e] >= from;
            if (!kept && !(gone >> e & 1u) && s0 + 32 * e < V) w[s0 + 32 * e] = -1.0f;
        }
    }
    const int kept = min(total, a.budget);
    for (int j = kept + tid; j < a.budget; j += NT) idx[j] = -1;
    if (tid == 0 && a.n_kept) a.n_kept[b] = kept;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
    // in registers where a CTA of 256 or 1024 threads holds the entries (64 x 32768 to 2048: 16
    // us; 64 x 65536 by the kernel that reads them again for every digit: 87 us, 39 once cut)
    cudaError_t e = cudaSuccess;
    if (a.N_cap <= 256 * 16) e = launch_dependent(evict_regs_kernel<256, 16>, (unsigned)a.B, 256, 0, s, a);
    else if (a.N_cap <= 1024 * 32) e = launch_dependent(evict_regs_kernel<1024, 32>, (unsigned)a.B, 1024, 0, s, a);
    else
        evict_kernel<<<(unsigned)a.B, kThreads, 0, s>>>(a);
    count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa
