// entry_weights.cu -- the attention weight each compressed entry received.
//
//   out[b, s] = in[b, s] + sum over query rows q that see s, and heads h, of
//               exp(scale * q[b, q, h] . kv_c[b, s] - lse[b, q, h])
// with the attention's own log-sum-exp, so a row's weights over all its keys
// (window included) add to one a head.  s is visible to the row at position
// t iff s < min(floor((t+1)/m), n_entries[b]); with a list (idx) only the
// listed entries receive weight.  Sums are fp32.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace csa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

// What the entries had (or zero), for the calls that add to listed entries only.
__global__ void __launch_bounds__(kThreads) copy_weights_kernel(float* dst, const float* src, long n) {
    grid_wait();
    const long step = (long)gridDim.x * kThreads;
#pragma unroll 4
    for (long i = (long)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) dst[i] = src ? src[i] : 0.0f;
}

// One CTA per 32 entries (or list slots): the keys staged as fp32, a lane per
// key, the (query row, head) pairs dealt to the warps; the warps' sums are
// added in warp order.
template <typename T>
__global__ void __launch_bounds__(kThreads) weights_simt_kernel(WeightsArgs a) {
    extern __shared__ float sm[];
    grid_wait();
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
    // Rows four at a time share the key's reads, the last few (or few rows) go one by one:
    // 64 query rows of 8 heads over 4 x 1024 fp32 entries of 64 take 30 us; one by one on 8
    // warps 128, by fours on 8 and 16 warps 64 and 37.
    const int n = a.n_q * a.H, fours = n / (4 * kWarps) * (4 * kWarps);
    const T* q0 = static_cast<const T*>(a.q) + (size_t)b * n * D;
    const float* k = Ks + lane * DP;
    const auto rows = [&](int r, auto count) {               // weights of rows r, r + 1, ..
        constexpr int kCount = decltype(count)::value;
        const T* q = q0 + (size_t)r * D;
        float z[kCount];
#pragma unroll
        for (int j = 0; j < kCount; ++j) z[j] = 0.0f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float k0 = k[d], k1 = k[d + 1], k2 = k[d + 2], k3 = k[d + 3];
#pragma unroll
            for (int j = 0; j < kCount; ++j) {
                const float4 x = load4(q + j * D + d);
                z[j] = fmaf(x.w, k3, fmaf(x.z, k2, fmaf(x.y, k1, fmaf(x.x, k0, z[j]))));
            }
        }
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int qi = (r + j) / a.H;
            const int t = a.q_pos ? a.q_pos[(size_t)b * a.n_q + qi] : qi;
            const int vis = t < 0 ? 0 : (int)min(((unsigned)t + 1u) / (unsigned)a.m, (unsigned)ne);
            const float lse = a.lse[(size_t)b * n + r + j];
            if (!(lse > -INFINITY) && lse == lse) continue;  // an empty row: no weight
            if (s >= 0 && s < vis) acc += exp2f(fmaf(z[j], sl2, -lse * kLog2e));
        }
    };
    for (int r = warp * 4; r < fours; r += kWarps * 4) rows(r, std::integral_constant<int, 4>{});
    for (int r = fours + warp; r < n; r += kWarps) rows(r, std::integral_constant<int, 1>{});
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

// ------------------------------------------------------------------ mma.sync
// bf16, D 64 or 128: z = K.Q^T on the tensor cores (m16n8k16, fp32 sums of exact
// products), 32 keys a warp as the A operand straight from global memory (each
// read once, its 64 or 128 registers stay for all heads), the query rows' heads in
// steps of 64 as the B operand from shared memory, double-buffered by cp.async.  A
// thread adds the weights of its keys over its columns, so the sums over heads
// and query rows stay in registers and meet in one quad at the end: no atomics, a
// fixed order.  Decode (one query row) is bound by HBM; with many query rows the
// exponentials and products are the longer part.
constexpr int kMmaWarps = 4;
constexpr int kMmaThreads = kMmaWarps * 32;
constexpr int kMmaKeys = 32 * kMmaWarps;      // keys a CTA
constexpr int kCols = 64;                     // (query row, head) columns a step

// 2^x within 2^-22 of itself, results below 2^-126 as 0: the scores' own rounding (D products
// in fp32) moves a weight by more.
__device__ __forceinline__ float wex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

template <int D>
__global__ void __launch_bounds__(kMmaThreads) weights_mma_kernel(WeightsArgs a, int chunks) {
    constexpr int KS = D / 16;                // k steps
    constexpr int RB = D * 2 + 64;            // bytes of a staged row (64 more: no bank conflicts)
    __shared__ __align__(16) uint8_t Qs[2][kCols * RB];
    __shared__ float Ls[2][kCols];            // lse * log2(e); +inf: no weight
    __shared__ int Vs[2][kCols];              // entries the column's row sees
    grid_wait();
    const int b = blockIdx.x / chunks, chunk = blockIdx.x - b * chunks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tq = lane & 3;
    const int slots = a.idx ? a.topk : a.N_cap;
    const int ne = clampi(a.n_entries ? a.n_entries[b] : a.N_cap, 0, a.N_cap);
    const int cols = a.n_q * a.H;
    const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv_c) + (size_t)b * a.N_cap * D;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (size_t)b * cols * D;

    // columns c0 .. c0 + 63 of the element: the query rows' heads, lse and reach
    const auto stage = [&](int buf, int c0) {
        for (int i = tid; i < kCols * (D / 8); i += kMmaThreads) {
            const int c = i / (D / 8), e = i - c * (D / 8);
            const bool in = c0 + c < cols;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(smem_addr(Qs[buf] + c * RB + e * 16)), "l"(q + (in ? (size_t)(c0 + c) * D + e * 8 : 0)),
                           "r"(in ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (tid < kCols) {
            const int c = c0 + tid;
            float l = INFINITY;
            int vis = 0;
            if (c < cols) {
                const int qi = c / a.H;
                const int t = a.q_pos ? a.q_pos[(size_t)b * a.n_q + qi] : qi;
                vis = t < 0 ? 0 : (int)min(((unsigned)t + 1u) / (unsigned)a.m, (unsigned)ne);
                l = a.lse[(size_t)b * cols + c] * kLog2e;
                if (l == -INFINITY) vis = 0;          // an empty row adds nothing
            }
            Ls[buf][tid] = l;
            Vs[buf][tid] = vis;
        }
    };
    if (cols > 0) stage(0, 0);

    // this thread's keys: rows g and g + 8 of two m16 tiles
    int ent[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = chunk * kMmaKeys + warp * 32 + i * 8 + g;
        int s = j < slots ? (a.idx ? a.idx[(size_t)b * a.topk + j] : j) : -1;
        ent[i] = (s >= 0 && s < a.N_cap) ? s : -1;
    }
    // A operand: 16-byte loads; a row's channels are dealt to the k steps so that a
    // thread's 8 consecutive channels are its fragments of two steps (the B operand is
    // read with the same order, which a dot product does not see)
    uint32_t A[2][KS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool live = ent[i] >= 0 && ent[i] < ne;
        const uint4* row = reinterpret_cast<const uint4*>(kv + (size_t)(live ? ent[i] : 0) * D);
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
            // a key that no row sees may hold anything: zeros in its place
            const uint4 v = live ? __ldg(row + k2 * 4 + tq) : make_uint4(0u, 0u, 0u, 0u);
            A[i >> 1][2 * k2][i & 1] = v.x;
            A[i >> 1][2 * k2][2 + (i & 1)] = v.y;
            A[i >> 1][2 * k2 + 1][i & 1] = v.z;
            A[i >> 1][2 * k2 + 1][2 + (i & 1)] = v.w;
        }
    }
    const float sl2 = a.scale * kLog2e;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

    for (int c0 = 0, buf = 0; c0 < cols; c0 += kCols, buf ^= 1) {
        if (c0 + kCols < cols) {
            stage(buf ^ 1, c0 + kCols);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
#pragma unroll 2
        for (int n0 = 0; n0 < kCols; n0 += 8) {
            float z[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[mt][e] = 0.0f;
            const uint8_t* qrow = Qs[buf] + (n0 + g) * RB;
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
                const uint4 w = *reinterpret_cast<const uint4*>(qrow + (k2 * 4 + tq) * 16);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const uint32_t* x = A[mt][2 * k2];
                    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                                 : "+f"(z[mt][0]), "+f"(z[mt][1]), "+f"(z[mt][2]), "+f"(z[mt][3])
                                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(w.x), "r"(w.y));
                    const uint32_t* y = A[mt][2 * k2 + 1];
                    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                                 : "+f"(z[mt][0]), "+f"(z[mt][1]), "+f"(z[mt][2]), "+f"(z[mt][3])
                                 : "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(w.z), "r"(w.w));
                }
            }
            const int c = n0 + 2 * tq;
            const float2 l = *reinterpret_cast<const float2*>(&Ls[buf][c]);
            const int2 vs = *reinterpret_cast<const int2*>(&Vs[buf][c]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 2 * mt + (e >> 1);
                    const float w = wex2(fmaf(z[mt][e], sl2, (e & 1) ? -l.y : -l.x));
                    if (ent[i] < ((e & 1) ? vs.y : vs.x)) acc[i] += w;
                }
        }
        __syncthreads();
    }
    // over the quad's columns, then one thread a key writes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 1);
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 2);
        if (tq == i && ent[i] >= 0) {
            float* dst = a.out + (size_t)b * a.N_cap + ent[i];
            if (a.idx) atomicAdd(dst, acc[i]);
            else *dst = (a.in ? a.in[(size_t)b * a.N_cap + ent[i]] : 0.0f) + acc[i];
        }
    }
}

template <int D>
cudaError_t launch_mma(const WeightsArgs& a, cudaStream_t s) {
    const int slots = a.idx ? a.topk : a.N_cap;
    const int chunks = (slots + kMmaKeys - 1) / kMmaKeys;
    const cudaError_t e = launch_dependent(weights_mma_kernel<D>, (unsigned)((long)chunks * a.B), kMmaThreads, 0, s, a, chunks);
    count_launch();
    return e;
}

template <typename T>
cudaError_t launch_simt(const WeightsArgs& a, cudaStream_t s) {
    const int slots = a.idx ? a.topk : a.N_cap;
    const size_t smem = sizeof(float) * (kKeys * (a.D + 1) + kWarps * kKeys);
    const unsigned grid = (unsigned)((long)((slots + kKeys - 1) / kKeys) * a.B);
    const cudaError_t e = launch_dependent(weights_simt_kernel<T>, grid, kThreads, smem, s, a);
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_entry_weights(const WeightsArgs& a, cudaStream_t s) {
    if (a.idx && a.out != a.in) {     // the unlisted entries keep what they had
        // (a kernel, and the next one set up meanwhile: 64 lists of 1999 of 8192 entries, calls
        // one after the other, took 18.5 us with cudaMemcpyAsync)
        const long n = (long)a.B * a.N_cap;
        const unsigned grid = (unsigned)std::min<long>((n + 4 * kThreads - 1) / (4 * kThreads), 148L * 8);
        const cudaError_t e = launch_dependent(copy_weights_kernel, grid, kThreads, 0, s, a.out, a.in, n);
        count_launch();
        if (e != cudaSuccess) return e;
    }
    if ((a.idx ? a.topk : a.N_cap) == 0) return cudaSuccess;
    if (entry_weights_tc_supported(a)) {
        uint32_t* err = device_error_word();
        if (!err) return cudaErrorUnknown;
        return launch_entry_weights_tc(a, err, s);
    }
    if (a.dt == DT_BF16 && a.D == 128) return launch_mma<128>(a, s);
    if (a.dt == DT_BF16 && a.D == 64) return launch_mma<64>(a, s);
    if (a.dt == DT_F32) return launch_simt<float>(a, s);
    return launch_simt<__nv_bfloat16>(a, s);
}

}  // namespace csa
