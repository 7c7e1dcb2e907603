// attention.cu -- stage 3: joint-softmax shared-KV MQA over the selected
// compressed entries (CSA) or all visible entries (HCA) plus the sliding
// window of raw rows.
//
// For query row (b, q) at position t, head h:
//   keys = compressed set ∪ { raw row j : raw_pos0[b]+j in [max(0, t-W+1), t] }
//   o = sum_s softmax_s(scale * q.key_s) key_s      (key = value, one KV head)
// ("DS-V4 分析&学习" §1.2, §1.4, §1.5; "百万上下文从「奢侈品」变「日用品」…"
//  §4.3, §5.2 window [max(0,i-W+1), i] and 1/sqrt(head_dim).)
//
// Generic path: one CTA per query row and all H heads (MQA: every head reads
// the same key block, staged once in shared memory as fp32).  Keys stream in
// blocks of 32 through an online (running max / running sum) softmax kept
// in base 2; the compressed part and the window part are one sequence of
// "virtual" keys so both share a single softmax.
//
// With a shared prefix (few rows, many keys) a cluster of CTAs takes a query
// row, each a share of its keys; the states (m, l, O) meet in distributed
// shared memory.  One CTA a row waits for its 32 keys at a time: 10 fp32 rows of
// 8 heads over 574 keys take 53 us on one CTA a row and 12 on 8.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "attn_rows.cuh"
#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kBK = 32;
constexpr int kMaxCluster = 8, kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;

// kSplit: a cluster of CTAs a row, each a run of whole blocks of keys.
template <typename T, int H, int D, bool kSplit>
__global__ void __launch_bounds__(kThreads) attn_generic_kernel(AttnArgs a) {
    constexpr int TPH = kThreads / H;    // threads per head
    constexpr int KPT = kBK / TPH;       // keys per thread in the score step
    constexpr int DPT = D / TPH;         // output dims per thread
    constexpr int DP = D + 1;            // padded row stride (bank spread)
    extern __shared__ float sm[];
    float* Qs = sm;                      // [H][DP]
    float* Ks = Qs + H * DP;             // [kBK][DP]
    float* Ps = Ks + kBK * DP;           // [H][kBK]
    int* valid = reinterpret_cast<int*>(Ps + H * kBK);   // [kBK]
    const T** krow = reinterpret_cast<const T**>(valid + kBK);  // [kBK]

    int C = 1, rank = 0;
    if constexpr (kSplit) {
        grid_wait();
        C = (int)cg::this_cluster().num_blocks();
        rank = (int)cg::this_cluster().block_rank();
    }
    const int row = blockIdx.x / C;
    const int b = row / a.n_q;
    const int t = a.q_pos ? a.q_pos[row] : a.pos0 + (row - b * a.n_q);
    const RowKeys rk = row_keys(a, b, t);
    const int keys = rk.n_comp + rk.n_win;
    const int share = kSplit ? (keys + C * kBK - 1) / (C * kBK) * kBK : keys;
    const int first = kSplit ? min(keys, rank * share) : 0;
    const int total = kSplit ? min(keys, first + share) : keys;

    const T* q = static_cast<const T*>(a.q) + (size_t)row * H * D;
    const T* kvc = static_cast<const T*>(a.kv_c);          // rows from cache_row()
    const T* kvr = static_cast<const T*>(a.kv_raw) + (size_t)b * a.L_raw * D;
    const float qscale = a.scale * kLog2e;
    for (int p = threadIdx.x; p < H * D; p += kThreads) {
        const int h = p / D, c = p - h * D;
        Qs[h * DP + c] = to_f32(q[p]) * qscale;
    }

    const int h = threadIdx.x / TPH, sub = threadIdx.x % TPH;
    float o[DPT];
#pragma unroll
    for (int i = 0; i < DPT; ++i) o[i] = 0.0f;
    float mrun = -INFINITY, lrun = 0.0f;

    for (int base = first; base < total; base += kBK) {
        __syncthreads();
        if (threadIdx.x < kBK) {
            const int kk = base + threadIdx.x;
            const T* ptr = nullptr;
            if (kk < rk.n_comp) {
                const int s = (a.dense ? kk : a.idx[(size_t)row * a.topk + kk]) - a.N_p;
                if (s < 0 && a.N_p > 0) {                  // an entry of the shared prefix
                    ptr = static_cast<const T*>(a.kv_p) + (size_t)kk * D;
                } else if (s >= 0 && s < a.N_cap) {
                    const long r = cache_row(a.pages, a.N_cap, b, s);
                    if (r >= 0) ptr = kvc + (size_t)r * D;
                }
            } else if (kk < total) {
                ptr = kvr + (size_t)(rk.win_lo + kk - rk.n_comp) * D;
            }
            krow[threadIdx.x] = ptr;
            valid[threadIdx.x] = ptr != nullptr;
        }
        __syncthreads();
        for (int p = threadIdx.x; p < kBK * D; p += kThreads) {
            const int j = p / D, c = p - j * D;
            const T* ptr = krow[j];
            Ks[j * DP + c] = ptr ? to_f32(ptr[c]) : 0.0f;
        }
        __syncthreads();

        // scores of this thread's keys for head h (base-2 domain)
        float sc[KPT];
        float bmax = -INFINITY;
#pragma unroll
        for (int jj = 0; jj < KPT; ++jj) {
            const int j = sub * KPT + jj;
            float acc = 0.0f;
            const float* qh = Qs + h * DP;
            const float* kj = Ks + j * DP;
            for (int c = 0; c < D; ++c) acc = fmaf(qh[c], kj[c], acc);
            sc[jj] = valid[j] ? acc : -INFINITY;
            bmax = fmaxf(bmax, sc[jj]);
        }
        for (int off = TPH / 2; off; off >>= 1) bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, off));
        const float mnew = fmaxf(mrun, bmax);
        const float alpha = (mnew == -INFINITY) ? 1.0f : exp2f(mrun - mnew);
        float psum = 0.0f;
#pragma unroll
        for (int jj = 0; jj < KPT; ++jj) {
            const float p = (sc[jj] == -INFINITY) ? 0.0f : exp2f(sc[jj] - mnew);
            Ps[h * kBK + sub * KPT + jj] = p;
            psum += p;
        }
        for (int off = TPH / 2; off; off >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
        lrun = lrun * alpha + psum;
        mrun = mnew;
#pragma unroll
        for (int i = 0; i < DPT; ++i) o[i] *= alpha;
        __syncthreads();
        for (int j = 0; j < kBK; ++j) {
            const float p = Ps[h * kBK + j];
            const float* kj = Ks + j * DP;
#pragma unroll
            for (int i = 0; i < DPT; ++i) o[i] = fmaf(p, kj[i * TPH + sub], o[i]);
        }
    }

    if constexpr (kSplit) {
        // O over the queries, m and l over the weights: then a share of the row's
        // elements a CTA, in a fixed order over the CTAs
        __syncthreads();
#pragma unroll
        for (int i = 0; i < DPT; ++i) Qs[h * DP + i * TPH + sub] = o[i];
        if (sub == 0) {
            Ps[h] = mrun;
            Ps[H + h] = lrun;
        }
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        for (int p = rank * kThreads + threadIdx.x; p < H * D; p += C * kThreads) {
            const int ph = p / D, c = p - ph * D;
            float mc[kMaxCluster], lc[kMaxCluster], oc[kMaxCluster];
            float M = -INFINITY, l = 0.0f, v = 0.0f;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
                mc[k] = -INFINITY;
                lc[k] = oc[k] = 0.0f;
                if (k < C) {
                    const float* pp = cluster.map_shared_rank(Ps, k);
                    mc[k] = pp[ph];
                    lc[k] = pp[H + ph];
                    oc[k] = cluster.map_shared_rank(Qs, k)[ph * DP + c];
                }
                M = fmaxf(M, mc[k]);
            }
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
                const float w = mc[k] == -INFINITY ? 0.0f : exp2f(mc[k] - M);
                l = fmaf(w, lc[k], l);
                v = fmaf(w, oc[k], v);
            }
            // (l = 0: no key; a key that holds NaN makes l NaN, and so the row)
            store_out<T>(static_cast<T*>(a.out) + (size_t)row * H * D + p, l == 0.0f ? 0.0f : v / l);
            if (a.lse_out && c == 0)
                a.lse_out[(size_t)row * H + ph] = l == 0.0f ? -INFINITY : (M + log2f(l)) / kLog2e;
        }
        cluster.sync();                  // the peers read this CTA's shared memory
        return;
    }
    T* out = static_cast<T*>(a.out) + (size_t)row * H * D + (size_t)h * D;
    const float inv = lrun > 0.0f ? 1.0f / lrun : 0.0f;
#pragma unroll
    for (int i = 0; i < DPT; ++i) store_out<T>(out + i * TPH + sub, o[i] * inv);
    if (a.lse_out && sub == 0)
        a.lse_out[(size_t)row * H + h] = lrun > 0.0f ? (mrun + log2f(lrun)) / kLog2e : -INFINITY;
}

// CTAs a row: a power of two whose CTAs fit the SMs at one each and have a block
// of keys each.
int cluster_of(const AttnArgs& a) {
    const long rows = (long)a.B * a.n_q;
    const long keys = (long)a.N_p + a.N_cap + std::min(a.window, a.L_raw);
    int C = 1;
    while (2 * C <= kMaxCluster && rows * 2 * C <= kSms && keys >= 2 * C * kBK) C *= 2;
    return C;
}

template <typename T, int H, int D, bool kSplit>
cudaError_t launch_t(const AttnArgs& a, cudaStream_t s) {
    const int DP = D + 1;
    const size_t smem = sizeof(float) * ((size_t)H * DP + (size_t)kBK * DP + (size_t)H * kBK) +
                        sizeof(int) * kBK + sizeof(void*) * kBK;
    const int C = kSplit ? cluster_of(a) : 1;
    if (kSplit && C == 1) return launch_t<T, H, D, false>(a, s);
    auto kern = attn_generic_kernel<T, H, D, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if constexpr (kSplit) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(a.B * a.n_q * C));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)C;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kern, a);
        count_launch();
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    kern<<<(unsigned)(a.B * a.n_q), kThreads, smem, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <typename T, bool kSplit, int D>
cudaError_t launch_heads(const AttnArgs& a, cudaStream_t s, const char** why) {
    switch (a.H) {
        case 8: return launch_t<T, 8, D, kSplit>(a, s);
        case 16: return launch_t<T, 16, D, kSplit>(a, s);
        case 32: return launch_t<T, 32, D, kSplit>(a, s);
        case 64: return launch_t<T, 64, D, kSplit>(a, s);
        case 128: return launch_t<T, 128, D, kSplit>(a, s);
    }
    *why = "attention: H must be one of 8, 16, 32, 64, 128";
    return cudaErrorNotSupported;
}

template <typename T, bool kSplit = false>
cudaError_t launch_dims(const AttnArgs& a, cudaStream_t s, const char** why) {
    if (a.D == 64) return launch_heads<T, kSplit, 64>(a, s, why);
    if (a.D == 128) return launch_heads<T, kSplit, 128>(a, s, why);
    *why = "attention: D must be 64 or 128";
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_attention_packed(const AttnArgs& a, cudaStream_t s) {
    if (a.vl == nullptr || a.pages.bt != nullptr || !attention_tc_supported(a))
        return cudaErrorNotSupported;
    uint32_t* err = device_error_word();
    if (!err) return cudaErrorUnknown;
    return launch_attention_tc(a, err, s);
}

unsigned long long attention_prefix_workspace(const AttnArgs& a) {
    return attention_prefix_tc_supported(a) ? attention_prefix_tc_workspace(a) : 0;
}

cudaError_t launch_attention_prefix(const AttnArgs& a, void* workspace, cudaStream_t s, const char** why) {
    if (attention_prefix_tc_supported(a)) {
        uint32_t* err = device_error_word();
        if (!err) return cudaErrorUnknown;
        return launch_attention_prefix_tc(a, workspace, err, s);
    }
    // (mma.sync over a row's keys: 4 rows of 16 heads over 4274 keys take 914 us on the
    // generic path without clusters, 29 us there)
    if (a.dt == DT_BF16 && attention_split_supported(a)) return launch_attention_split(a, s);
    if (a.dt == DT_F32) return launch_dims<float, true>(a, s, why);
    return launch_dims<__nv_bfloat16, true>(a, s, why);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t s, const char** why) {
    if (a.B <= 0 || a.n_q <= 0) return cudaSuccess;
    if (a.pages.bt == nullptr && attention_tc_supported(a)) {   // paged caches: decode kernels
        uint32_t* err = device_error_word();
        if (!err) return cudaErrorUnknown;
        return launch_attention_tc(a, err, s);
    }
    if (attention_dec_tc_supported(a)) {
        uint32_t* err = device_error_word();
        if (!err) return cudaErrorUnknown;
        return launch_attention_dec_tc(a, err, s);
    }
    if (attention_split_supported(a)) return launch_attention_split(a, s);
    if (a.dt == DT_F32) return launch_dims<float>(a, s, why);
    if (a.dt == DT_BF16) return launch_dims<__nv_bfloat16>(a, s, why);
    *why = "attention: dt must be F32 or BF16";
    return cudaErrorNotSupported;
}

}  // namespace csa
