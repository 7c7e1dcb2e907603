// rope.cu -- rotary positions of query heads and shared-KV rows.
//
// For a token at position p, pair j of a head's rotated part turns by the
// angle p * f_j (f_j in radians a position, given by the caller):
//   (a, b) -> s * (a cos - b sin, b cos + a sin)          (transpose: -sin)
// with (a, b) = elements (2j, 2j+1) of the part (interleaved) or
// (j, j + d_rot/2) (half).  Arithmetic is fp32; the result is rounded once.
//
// The angle.  p * f reaches 10^6 rad at long contexts, where an fp32 product
// is off by 0.06 rad.  The host turns f_j into a 64-bit fraction of a turn,
// F = frac(f / 2 pi) * 2^64 (rounded in extended precision); p * F mod 2^64
// is then the exact phase of the rounded frequency, whole turns dropping out
// by overflow, for any integer p.  Its top 32 bits feed sincospi: the angle
// is within 2^-32 turns + 2^53 relative of the exact one.
#include "common.cuh"
#include "kernels.h"

namespace csa {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
    T v[N];
};

// cos and sin of token `row`'s pairs for this CTA's tokens, cooperatively;
// void tokens (position < 0) keep ok = 0 and are passed on unrotated.
__device__ __forceinline__ void fill_angles(const RopeArgs& a, long tok0, int n_tok, float2* cs,
                                            int* ok) {
    const int half = a.d_rot / 2;
    for (int i = threadIdx.x; i < n_tok * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        const long tok = tok0 + t;
        const long p = a.pos ? (long)a.pos[tok] : a.pos0 + (tok % a.n) * (long)a.pos_step;
        const uint64_t phase = (uint64_t)p * a.turn[j];
        // the top 32 bits as a signed fraction of a turn in [-1/2, 1/2), in units of pi
        const float x = (float)(int32_t)(phase >> 32) * 0x1p-31f;
        float s, c;
        sincospif(x, &s, &c);
        cs[i] = make_float2(c * a.scale, (a.transpose ? -s : s) * a.scale);
        if (j == 0) ok[t] = p >= 0;
    }
    __syncthreads();
}

// One pair or one passed-on element per thread and step: any size, stride and offset.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_scalar_kernel(RopeArgs a, int tpb) {
    extern __shared__ float2 cs[];
    const int half = a.d_rot / 2;
    int* ok = reinterpret_cast<int*>(cs + (size_t)tpb * half);
    const long total = (long)a.B * a.n;
    const long tok0 = (long)blockIdx.x * tpb;
    const int n_tok = (int)min((long)tpb, total - tok0);
    fill_angles(a, tok0, n_tok, cs, ok);
    const int R = a.H[0] + a.H[1];
    const int ipr = half + (a.D - a.d_rot);
    for (int i = threadIdx.x; i < n_tok * R * ipr; i += blockDim.x) {
        const int rr = i / ipr, it = i - rr * ipr;
        const int t = rr / R, r = rr - t * R;
        const int w = r >= a.H[0];
        const int h = w ? r - a.H[0] : r;
        const T* src = static_cast<const T*>(a.x[w]) + (tok0 + t) * a.xs[w][0] + h * a.xs[w][1];
        T* dst = static_cast<T*>(a.out[w]) + (tok0 + t) * a.os[w][0] + h * a.os[w][1];
        if (it < half) {
            const int ea = a.off + (a.interleaved ? 2 * it : it);
            const int eb = ea + (a.interleaved ? 1 : half);
            if (!ok[t]) {
                const T u = src[ea], v = src[eb];
                dst[ea] = u;
                dst[eb] = v;
                continue;
            }
            const float u = to_f32(src[ea]), v = to_f32(src[eb]);
            const float2 c = cs[t * half + it];
            store_out<T>(dst + ea, u * c.x - v * c.y);
            store_out<T>(dst + eb, v * c.x + u * c.y);
        } else {
            int e = it - half;
            if (e >= a.off) e += a.d_rot;
            dst[e] = src[e];
        }
    }
}

template <typename T>
cudaError_t launch_scalar(const RopeArgs& a, cudaStream_t s) {
    const long total = (long)a.B * a.n;
    const int items = (a.H[0] + a.H[1]) * (a.d_rot / 2 + a.D - a.d_rot);
    const int tpb = items >= 1024 ? 1 : (items >= 256 ? 4 : 16);
    const size_t smem = (size_t)tpb * (a.d_rot / 2) * sizeof(float2) + tpb * sizeof(int);
    rope_scalar_kernel<T><<<(unsigned)((total + tpb - 1) / tpb), kThreads, smem, s>>>(a, tpb);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    if (a.dt == DT_F32) return launch_scalar<float>(a, s);
    return launch_scalar<__nv_bfloat16>(a, s);
}

}  // namespace csa
