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
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace csa {
namespace {

constexpr int kThreads = 256;

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

// 16 bytes of a row as fp32, and back (rounded to nearest).
__device__ __forceinline__ void unpack(const uint4& v, float* f, float) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float* f, __nv_bfloat16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float* f, float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float* f, __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes a step: a CTA takes tpb tokens and all their rows (the heads of both
// tensors, which share the angles), or rpb rows of one token.  A thread keeps one
// item of a row -- a vector (interleaved: its pairs are inside; not rotated: passed
// on), or in the half layout the two vectors whose channels pair up -- and goes
// down the rows.  Its next kDepth - 1 rows are on their way to its own slots of
// shared memory (cp.async, no barrier), the first of them while the angles are made.
// Bound by HBM: every byte is read and written once.  2 x 8192 tokens of 65 x 128
// bf16 take 87 us, 96% of a plain copy's rate; in batches of four rows through
// registers, which drain before the next is asked for, 114 us.  Depths of 3, 6 and 8
// took 4, 3 and 4 us more.
constexpr int kDepth = 4;
template <bool HALF>
__host__ __device__ constexpr size_t ring_bytes() { return (size_t)kDepth * kThreads * (HALF ? 32 : 16); }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// How a call is cut: tokens a CTA; rows a CTA of one token, and such CTAs a token; items
// a row; rows a step of the CTA's threads.  The divisors come with their reciprocals
// (the calls of a few us wait for every division).
struct RopeGrid {
    int tpb, rpb, chunks, ipr, row_step;
    float inv_rot, inv_pass, inv_h[2], inv_step;
};
// x / d for 0 <= x < 2^20, given 1 / d
__device__ __forceinline__ int quot(int x, float inv) { return (int)(((float)x + 0.5f) * inv); }

template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 4)
rope_vec_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeGrid g) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    float2* cs = reinterpret_cast<float2*>(smem + ring_bytes<HALF>());
    const int half = a.d_rot / 2;
    const int tpb = g.tpb, ipr = g.ipr, row_step = g.row_step;
    int* ok = reinterpret_cast<int*>(cs + (size_t)tpb * half);
    const long total = (long)a.B * a.n;
    const int tile = g.chunks == 1 ? (int)blockIdx.x : (int)(blockIdx.x / g.chunks);
    const long tok0 = (long)tile * tpb;
    const int r0 = ((int)blockIdx.x - tile * g.chunks) * g.rpb;
    const int n_tok = (int)min((long)tpb, total - tok0);
    const int R = min(a.H[0] + a.H[1] - r0, g.rpb);
    const int rot_items = (HALF ? half : a.d_rot) / V, pass_items = ipr - rot_items;
    // Rotated items to the first threads, the others to the rest: a warp of both kinds
    // would run the rotation for a third of its lanes.  (So mapped, and with every row's
    // offset computed anew, instruction issue was 79% busy: 90 us for the call above, 97
    // where its tensors' addresses collide in DRAM.)
    const bool rot = (int)threadIdx.x < row_step * rot_items;
    int it, rr0;                                             // the thread's item, and its first row
    if (rot) {
        rr0 = quot(threadIdx.x, g.inv_rot);
        it = threadIdx.x - rr0 * rot_items;
    } else {
        const int u = threadIdx.x - row_step * rot_items;
        rr0 = pass_items ? quot(u, g.inv_pass) : row_step;
        it = u - rr0 * pass_items;
    }
    // the item's element offset in a row (HALF: of the first of its two vectors)
    int e0 = it * V;
    if (rot) e0 += a.off;
    else if (e0 >= a.off) e0 += a.d_rot;
    const int pair0 = HALF ? it * V : it * (V / 2);
    // The CTA's rows: the hx x heads of its tokens, then their hy y heads.  A thread's
    // rows are row_step apart.
    const int hx = min(max(a.H[0] - r0, 0), R), hy = R - hx;
    const int nx = n_tok * hx, rows = n_tok * R;
    struct Rows {                // walks them
        const T* p;
        long inc, wrap;          // to the next row; and, past a token's last row, back to the next token's
        int v, r, t, h, dr, dt;  // row, its head and token; heads a token; steps of r and t
    };
    const auto row = [&](Rows& w, int v) {
        const bool y = v >= nx;
        w.v = v;
        if (y) v -= nx;
        if (tpb == 1) {          // (one token: no row is past its last)
            w.h = 1 << 30;
            w.t = w.dt = 0;
            w.r = v;
            w.dr = row_step;
            return;
        }
        w.h = y ? hy : hx;
        w.t = quot(v, g.inv_h[y]);
        w.r = v - w.t * w.h;
        w.dt = quot(row_step, g.inv_h[y]);
        w.dr = row_step - w.dt * w.h;
    };
    const auto aim = [&](Rows& w, const void* const* ptr, const long(*sd)[2]) {
        const bool y = w.v >= nx;
        const long s0 = sd[y][0], s1 = sd[y][1];
        w.inc = w.dt * s0 + w.dr * s1;
        w.wrap = s0 - w.h * s1;
        const int h0 = y ? max(r0 - a.H[0], 0) : r0;
        w.p = static_cast<const T*>(ptr[y]) + (tok0 + w.t) * s0 + (h0 + w.r) * s1 + e0;
    };
    const auto step = [&](Rows& w, const void* const* ptr, const long(*sd)[2]) {
        const bool x = w.v < nx;
        w.v += row_step;
        if (x && w.v >= nx) {    // from the x heads to the y heads
            row(w, w.v);
            aim(w, ptr, sd);
            return;
        }
        w.t += w.dt;
        w.r += w.dr;
        w.p += w.inc;
        if (w.r >= w.h) {
            w.r -= w.h;
            ++w.t;
            w.p += w.wrap;
        }
    };
    Rows in, out;
    row(in, rr0);
    out = in;
    aim(in, a.x, a.xs);
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;          // [kDepth][1 or 2][kThreads]
    constexpr int kSlot = (HALF ? 2 : 1) * kThreads;
    int left = rr0 < row_step && rows > rr0 ? quot(rows - rr0 + row_step - 1, g.inv_step) : 0;
    int count = left, slot = 0;
    const auto load = [&]() {
        if (left > 0) {
            uint4* d = ring + slot * kSlot;
            cp_async16(d, in.p);
            if (HALF && rot) cp_async16(d + kThreads, in.p + half);
            step(in, a.x, a.xs);
            --left;
        }
        slot = (slot + 1) % kDepth;
        asm volatile("cp.async.commit_group;" ::: "memory");             // (one a step, if empty)
    };
    grid_wait();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) load();
    fill_angles(a, tok0, n_tok, cs, ok);
    aim(out, a.out, a.os);
    for (; count > 0; --count) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        const uint4* d = ring + (slot + 1) % kDepth * kSlot;
        uint4 v = d[0], w = make_uint4(0, 0, 0, 0);
        if (HALF && rot) w = d[kThreads];
        load();                                              // (into the slot read a step ago)
        const int st = out.t;
        T* p = const_cast<T*>(out.p);
        if (rot && ok[st]) {
            const float2* c = cs + st * half + pair0;
            float x[V], y[V];
            unpack(v, x, T());
            if (HALF) {
                unpack(w, y, T());
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 q = c[i];
                    const float p0 = x[i] * q.x - y[i] * q.y, p1 = y[i] * q.x + x[i] * q.y;
                    x[i] = p0;
                    y[i] = p1;
                }
                w = pack(y, T());
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 q = c[i];
                    const float p0 = x[2 * i] * q.x - x[2 * i + 1] * q.y, p1 = x[2 * i + 1] * q.x + x[2 * i] * q.y;
                    x[2 * i] = p0;
                    x[2 * i + 1] = p1;
                }
            }
            v = pack(x, T());
        }
        *reinterpret_cast<uint4*>(p) = v;
        if (HALF && rot) *reinterpret_cast<uint4*>(p + half) = w;
        step(out, a.out, a.os);
    }
}

template <typename T>
bool vec_supported(const RopeArgs& a) {
    constexpr int V = 16 / sizeof(T);
    if (a.D % V || a.off % V || (a.interleaved ? a.d_rot % V : a.d_rot / 2 % V)) return false;
    if (a.D / V > kThreads) return false;
    for (int w = 0; w < 2; ++w)
        if (a.H[w] && (a.xs[w][0] % V || a.xs[w][1] % V || a.os[w][0] % V || a.os[w][1] % V)) return false;
    return true;
}

template <typename T>
cudaError_t launch_vec(const RopeArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const long total = (long)a.B * a.n;
    // in place, the channels that are not rotated are already there
    const bool in_place = (!a.H[0] || a.x[0] == a.out[0]) && (!a.H[1] || a.x[1] == a.out[1]);
    const int R = a.H[0] + a.H[1];
    const int ipr = (a.interleaved ? a.d_rot : a.d_rot / 2) / V + (in_place ? 0 : (a.D - a.d_rot) / V);
    // Rows a CTA: kDepth a thread, fewer where the call has too few rows for
    // the GPU (148 SMs, two CTAs each); whole tokens where a token's rows fit.  With
    // rows for 16 CTAs an SM, up to 8 times that: making one token's angles a CTA, by one
    // warp, cost more than moving its rows.
    const int step = kThreads / ipr, pass = step * kDepth;
    const int want = (int)std::max<long>(std::min<long>(std::max<long>(total * R / (2 * 148), step), pass),
                                         std::min<long>(total * R / (16 * 148), 8L * pass));
    int tpb = 1, rpb = R, chunks = 1;
    if (want >= R) {
        tpb = std::max(1, std::min(want / R, 4096 / (a.d_rot / 2)));      // angles: 32 KB at most
    } else {
        chunks = (R + want - 1) / want;
        rpb = (R + chunks - 1) / chunks;
    }
    const auto inv = [](int d) { return d > 0 ? 1.0f / (float)d : 0.0f; };
    const int rot_items = (a.interleaved ? a.d_rot : a.d_rot / 2) / V;
    const RopeGrid g{tpb, rpb, chunks, ipr, step, inv(rot_items), inv(ipr - rot_items), {inv(a.H[0]), inv(a.H[1])}, inv(step)};
    const long blocks = (total + tpb - 1) / tpb * chunks;
    if (blocks > (1L << 31) - 1) return cudaErrorInvalidConfiguration;
    const size_t smem = (a.interleaved ? ring_bytes<false>() : ring_bytes<true>()) +
                        (size_t)tpb * (a.d_rot / 2) * sizeof(float2) + tpb * sizeof(int);
    auto kern = a.interleaved ? rope_vec_kernel<T, false> : rope_vec_kernel<T, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, (unsigned)blocks, kThreads, smem, s, a, g);
    count_launch();
    return e;
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
    // 16-byte items need sizes and strides that are whole vectors
    if (a.dt == DT_F32) return vec_supported<float>(a) ? launch_vec<float>(a, s) : launch_scalar<float>(a, s);
    return vec_supported<__nv_bfloat16>(a) ? launch_vec<__nv_bfloat16>(a, s) : launch_scalar<__nv_bfloat16>(a, s);
}

}  // namespace csa
