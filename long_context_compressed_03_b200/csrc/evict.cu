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

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
    evict_kernel<<<(unsigned)a.B, kThreads, 0, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace csa
