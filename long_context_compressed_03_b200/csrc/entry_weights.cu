// entry_weights.cu -- the attention weight each compressed entry received.
//
//   out[b, s] = in[b, s] + sum over query rows q that see s, and heads h, of
//               exp(scale * q[b, q, h] . kv_c[b, s] - lse[b, q, h])
// with the attention's own log-sum-exp, so a row's weights over all its keys
// (window included) add to one a head.  s is visible to the row at position
// t iff s < min(floor((t+1)/m), n_entries[b]); with a list (idx) only the
// listed entries receive weight.  Sums are fp32.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 32;
constexpr float kLog2e = 1.4426950408889634f;

// One CTA per 32 entries (or list slots): the keys staged as fp32, a lane per
// key, the (query row, head) pairs dealt to the warps; the warps' sums are
// added in warp order.
template <typename T>
__global__ void __launch_bounds__(kThreads) weights_simt_kernel(WeightsArgs a) {
    extern __shared__ float sm[];
    const int D = a.D, DP = D + 1;
    float* Ks = sm;                       // [32][D + 1]
    float* part = sm + kKeys * DP;        // [warps][32]
    __shared__ int ent[kKeys];
    const int slots = a.idx ? a.topk : a.N_cap;
    const int chunks = (slots + kKeys - 1) / kKeys;
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ne = clampi(a.n_entries ? a.n_entries[b] : a.N_cap, 0, a.N_cap);
    if (tid < kKeys) {
        const int j = chunk * kKeys + tid;
        int s = j < slots ? (a.idx ? a.idx[(size_t)b * a.topk + j] : j) : -1;
        ent[tid] = (s >= 0 && s < a.N_cap) ? s : -1;
    }
    __syncthreads();
    const T* kv = static_cast<const T*>(a.kv_c) + (size_t)b * a.N_cap * D;
    for (int i = tid; i < kKeys * D; i += kThreads) {
        const int k = i / D, d = i - k * D;
        const int s = ent[k];
        Ks[k * DP + d] = (s >= 0 && s < ne) ? to_f32(kv[(size_t)s * D + d]) : 0.0f;
    }
    __syncthreads();
    const int s = ent[lane];
    const float sl2 = a.scale * kLog2e;
    float acc = 0.0f;
    for (int r = warp; r < a.n_q * a.H; r += kWarps) {
        const int qi = r / a.H;
        const int t = a.q_pos ? a.q_pos[(size_t)b * a.n_q + qi] : qi;
        const int vis = t < 0 ? 0 : min((int)(((unsigned)t + 1u) / (unsigned)a.m), ne);
        const size_t row = (size_t)b * a.n_q * a.H + r;
        const float lse = a.lse[row];
        if (!(lse > -INFINITY) && lse == lse) continue;      // an empty row: no weight
        const T* q = static_cast<const T*>(a.q) + row * D;
        float z = 0.0f;
        for (int d = 0; d < D; ++d) z = fmaf(to_f32(q[d]), Ks[lane * DP + d], z);
        if (s >= 0 && s < vis) acc += exp2f(fmaf(z, sl2, -lse * kLog2e));
    }
    part[warp * kKeys + lane] = acc;
    __syncthreads();
    if (warp == 0 && s >= 0) {
        float v = 0.0f;
        for (int i = 0; i < kWarps; ++i) v += part[i * kKeys + lane];
        float* dst = a.out + (size_t)b * a.N_cap + s;
        // listed entries: the same entry twice receives twice its weight
        if (a.idx) atomicAdd(dst, v);
        else *dst = (a.in ? a.in[(size_t)b * a.N_cap + s] : 0.0f) + v;
    }
}

template <typename T>
cudaError_t launch_simt(const WeightsArgs& a, cudaStream_t s) {
    const int slots = a.idx ? a.topk : a.N_cap;
    const size_t smem = sizeof(float) * (kKeys * (a.D + 1) + kWarps * kKeys);
    const unsigned grid = (unsigned)((long)((slots + kKeys - 1) / kKeys) * a.B);
    weights_simt_kernel<T><<<grid, kThreads, smem, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_entry_weights(const WeightsArgs& a, cudaStream_t s) {
    if (a.idx && a.out != a.in) {     // the unlisted entries keep what they had
        const size_t bytes = sizeof(float) * (size_t)a.B * a.N_cap;
        const cudaError_t e = a.in ? cudaMemcpyAsync(a.out, a.in, bytes, cudaMemcpyDeviceToDevice, s)
                                   : cudaMemsetAsync(a.out, 0, bytes, s);
        if (e != cudaSuccess) return e;
    }
    if ((a.idx ? a.topk : a.N_cap) == 0) return cudaSuccess;
    if (a.dt == DT_F32) return launch_simt<float>(a, s);
    return launch_simt<__nv_bfloat16>(a, s);
}

}  // namespace csa
