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
// F = frac(f / 2 pi) * 2^64 (to the nearest, from 1 / 2 pi to 128 bits); p * F mod
// 2^64 is then the exact phase of the rounded frequency, whole turns dropping out by
// overflow, for any integer p: within 2^-34 of a turn of p * f where p < 2^31.  The
// nearest quarter turn comes off in integers; the rest, at most 1/8 turn, is cut to 34
// fraction bits and rounded to fp32 (2^-28 of a turn at most, less the closer it is to
// the quarter turn) and feeds sincospi.  So the angle is within 2^-27 of a turn.
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
        const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
        const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));       // [-1/8, 1/8) turn
        float s, c;
        sincospif((float)(int32_t)(rest >> 30) * 0x1p-33f, &s, &c);              // in units of pi
        if (quarter & 1u) {                                  // (a quarter turn on: cos is -sin, sin is cos)
            const float w = c;
            c = -s;
            s = w;
        }
        if (quarter & 2u) {
            c = -c;
            s = -s;
        }
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

// How a call is cut: tokens a CTA; rows a CTA of one token, and such CTAs a token; items
// a row; rows a step of the CTA's threads.  The divisors come with their reciprocals
// (the calls of a few us wait for every division).
struct RopeGrid {
    int tpb, rpb, chunks, ipr, row_step;
    float inv_rot, inv_pass, inv_h[2], inv_step;
};
// x / d for 0 <= x < 2^20, given 1 / d
__device__ __forceinline__ int quot(int x, float inv) { return (int)(((float)x + 0.5f) * inv); }

// A CTA's rows: the hx x heads of its tokens, then their hy y heads.
struct RopeTile {
    long tok0;
    int r0, n_tok, hx, hy, nx, rows, tpb, row_step;
    float inv_x, inv_y;          // 1 / heads
    __device__ __forceinline__ RopeTile(const RopeArgs& a, const RopeGrid& g) {
        const long total = (long)a.B * a.n;
        const int tile = g.chunks == 1 ? (int)blockIdx.x : (int)(blockIdx.x / g.chunks);
        tpb = g.tpb;
        row_step = g.row_step;
        inv_x = g.inv_h[0];
        inv_y = g.inv_h[1];
        tok0 = (long)tile * tpb;
        r0 = ((int)blockIdx.x - tile * g.chunks) * g.rpb;
        n_tok = (int)min((long)tpb, total - tok0);
        const int R = min(a.H[0] + a.H[1] - r0, g.rpb);
        hx = min(max(a.H[0] - r0, 0), R);
        hy = R - hx;
        nx = n_tok * hx;
        rows = n_tok * R;
    }
};
// Walks the rows of one thread, row_step apart.
template <typename T>
struct Rows {
    const T* p;
    long inc, wrap;              // to the next row; and, past a token's last row, back to the next token's
    int v, r, t, h, dr, dt;      // row, its head and token; heads a token; steps of r and t
    __device__ __forceinline__ void row(const RopeTile& c, int at) {
        const bool y = at >= c.nx;
        v = at;
        if (y) at -= c.nx;
        if (c.tpb == 1) {        // (one token: no row is past its last)
            h = 1 << 30;
            t = dt = 0;
            r = at;
            dr = c.row_step;
            return;
        }
        const float inv = y ? c.inv_y : c.inv_x;
        h = y ? c.hy : c.hx;
        t = quot(at, inv);
        r = at - t * h;
        dt = quot(c.row_step, inv);
        dr = c.row_step - dt * h;
    }
    __device__ __forceinline__ void aim(const RopeArgs& a, const RopeTile& c, const void* const* ptr,
                                        const long (*sd)[2], int e0) {
        const bool y = v >= c.nx;
        const long s0 = sd[y][0], s1 = sd[y][1];
        inc = dt * s0 + dr * s1;
        wrap = s0 - h * s1;
        const int h0 = y ? max(c.r0 - a.H[0], 0) : c.r0;
        p = static_cast<const T*>(ptr[y]) + (c.tok0 + t) * s0 + (h0 + r) * s1 + e0;
    }
    __device__ __forceinline__ void step(const RopeArgs& a, const RopeTile& c, const void* const* ptr,
                                         const long (*sd)[2], int e0) {
        const bool x = v < c.nx;
        v += c.row_step;
        if (x && v >= c.nx) {    // from the x heads to the y heads
            row(c, v);
            aim(a, c, ptr, sd, e0);
            return;
        }
        t += dt;
        r += dr;
        p += inc;
        if (r >= h) {
            r -= h;
            ++t;
            p += wrap;
        }
    }
    // the next row without an address
    __device__ __forceinline__ void next(const RopeTile& c) {
        const bool x = v < c.nx;
        v += c.row_step;
        if (x && v >= c.nx) {
            row(c, v);
            return;
        }
        t += dt;
        r += dr;
        if (r >= h) {
            r -= h;
            ++t;
        }
    }
};

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

template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 4)
rope_vec_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeGrid g) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    float2* cs = reinterpret_cast<float2*>(smem + ring_bytes<HALF>());
    const int half = a.d_rot / 2;
    const RopeTile c(a, g);
    const int ipr = g.ipr, row_step = g.row_step;
    int* ok = reinterpret_cast<int*>(cs + (size_t)g.tpb * half);
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
    Rows<T> in, out;
    in.row(c, rr0);
    out = in;
    in.aim(a, c, a.x, a.xs, e0);
    uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;          // [kDepth][1 or 2][kThreads]
    constexpr int kSlot = (HALF ? 2 : 1) * kThreads;
    int left = rr0 < row_step && c.rows > rr0 ? quot(c.rows - rr0 + row_step - 1, g.inv_step) : 0;
    int count = left, slot = 0;
    const auto load = [&]() {
        if (left > 0) {
            uint4* d = ring + slot * kSlot;
            cp_async16(d, in.p);
            if (HALF && rot) cp_async16(d + kThreads, in.p + half);
            in.step(a, c, a.x, a.xs, e0);
            --left;
        }
        slot = (slot + 1) % kDepth;
        asm volatile("cp.async.commit_group;" ::: "memory");             // (one a step, if empty)
    };
    grid_wait();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) load();
    fill_angles(a, c.tok0, c.n_tok, cs, ok);
    out.aim(a, c, a.out, a.os, e0);
    for (; count > 0; --count) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        const uint4* d = ring + (slot + 1) % kDepth * kSlot;
        uint4 v = d[0], w = make_uint4(0, 0, 0, 0);
        if (HALF && rot) w = d[kThreads];
        load();                                              // (into the slot read a step ago)
        const int st = out.t;
        T* p = const_cast<T*>(out.p);
        if (rot && ok[st]) {
            const float2* angle = cs + st * half + pair0;
            float x[V], y[V];
            unpack(v, x, T());
            if (HALF) {
                unpack(w, y, T());
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 q = angle[i];
                    const float p0 = x[i] * q.x - y[i] * q.y, p1 = y[i] * q.x + x[i] * q.y;
                    x[i] = p0;
                    y[i] = p1;
                }
                w = pack(y, T());
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 q = angle[i];
                    const float p0 = x[2 * i] * q.x - x[2 * i + 1] * q.y, p1 = x[2 * i + 1] * q.x + x[2 * i] * q.y;
                    x[2 * i] = p0;
                    x[2 * i + 1] = p1;
                }
            }
            v = pack(x, T());
        }
        *reinterpret_cast<uint4*>(p) = v;
        if (HALF && rot) *reinterpret_cast<uint4*>(p + half) = w;
        out.step(a, c, a.out, a.os, e0);
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

constexpr int kMostPairs = 4096;                             // angles a CTA keeps: 32 KB

// Cuts a call whose rows have rot_items and pass_items.
RopeGrid cut(const RopeArgs& a, int rot_items, int pass_items, long most, long* blocks) {
    const long total = (long)a.B * a.n;
    const int R = a.H[0] + a.H[1], ipr = rot_items + pass_items;
    // Rows a CTA: kDepth a thread, fewer where the call has too few rows for
    // the GPU (148 SMs, two CTAs each); whole tokens where a token's rows fit.  With
    // rows for 16 CTAs an SM, up to `most` times that: making one token's angles a CTA, by one
    // warp, cost more than moving its rows.
    const int step = std::max(kThreads / ipr, 1), pass = step * kDepth;
    const int want = (int)std::max<long>(std::min<long>(std::max<long>(total * R / (2 * 148), step), pass),
                                         std::min<long>(total * R / (16 * 148), most * pass));
    RopeGrid g{1, R, 1, ipr, step, 0.0f, 0.0f, {0.0f, 0.0f}, 0.0f};
    if (want >= R) {
        g.tpb = std::max(1, std::min(want / R, kMostPairs / (a.d_rot / 2)));
    } else {
        g.chunks = (R + want - 1) / want;
        g.rpb = (R + g.chunks - 1) / g.chunks;
    }
    const auto inv = [](int d) { return d > 0 ? 1.0f / (float)d : 0.0f; };
    g.inv_rot = inv(rot_items);
    g.inv_pass = inv(pass_items);
    g.inv_h[0] = inv(a.H[0]);
    g.inv_h[1] = inv(a.H[1]);
    g.inv_step = inv(step);
    *blocks = (total + g.tpb - 1) / g.tpb * g.chunks;
    return g;
}
size_t angle_bytes(const RopeArgs& a, const RopeGrid& g) {
    return (size_t)g.tpb * (a.d_rot / 2) * sizeof(float2) + g.tpb * sizeof(int);
}
// A kernel's shared memory goes with the call's sizes, the limit set for it does not: it is
// the kernel's, so that of a smaller call on another host thread would hold for a larger
// one that is about to be launched.  (Tokens a CTA: kMostPairs at most, at one pair each.)
constexpr size_t kAngleLimit = kMostPairs * (sizeof(float2) + sizeof(int));
constexpr size_t kTileLimit = 32768;                         // of rope_staged_kernel

template <typename K>
cudaError_t allow_smem(K* kern, size_t limit, size_t smem) {
    if (smem > limit) return cudaErrorInvalidValue;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
}
// In place, the channels that are not rotated are already there.
int pass_channels(const RopeArgs& a) {
    const bool in_place = (!a.H[0] || a.x[0] == a.out[0]) && (!a.H[1] || a.x[1] == a.out[1]);
    return in_place ? 0 : a.D - a.d_rot;
}

template <typename T>
cudaError_t launch_vec(const RopeArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    long blocks;
    const RopeGrid g = cut(a, (a.interleaved ? a.d_rot : a.d_rot / 2) / V, pass_channels(a) / V, 8, &blocks);
    if (blocks > (1L << 31) - 1) return cudaErrorInvalidConfiguration;
    const size_t ring = a.interleaved ? ring_bytes<false>() : ring_bytes<true>(), smem = ring + angle_bytes(a, g);
    auto kern = a.interleaved ? rope_vec_kernel<T, false> : rope_vec_kernel<T, true>;
    cudaError_t e = allow_smem(kern, ring + kAngleLimit, smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, (unsigned)blocks, kThreads, smem, s, a, g);
    count_launch();
    return e;
}

// Heads that are whole 16-byte vectors, with a rotated part that is not: the rows pass
// through shared memory, where a thread a pair rotates them.  2 x 4096 tokens of 17 x 80
// bf16, 50 rotated, take 17 us, element by element in global memory 35.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_staged_kernel(const __grid_constant__ RopeArgs a,
                                                               const __grid_constant__ RopeGrid g) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    const int half = a.d_rot / 2;
    const RopeTile c(a, g);
    T* tile = reinterpret_cast<T*>(smem);                    // [rows][D]
    float2* cs = reinterpret_cast<float2*>(tile + (size_t)c.tpb * g.rpb * a.D);
    int* ok = reinterpret_cast<int*>(cs + (size_t)g.tpb * half);
    const int rr0 = (int)threadIdx.x / g.ipr, e0 = ((int)threadIdx.x - rr0 * g.ipr) * V;
    const bool moves = rr0 < c.row_step;                     // (the last threads may have no vector)
    Rows<T> w;
    grid_wait();
    w.row(c, rr0);
    w.aim(a, c, a.x, a.xs, e0);
    while (moves && w.v < c.rows) {
        cp_async16(tile + w.v * a.D + e0, w.p);
        w.step(a, c, a.x, a.xs, e0);
    }
    fill_angles(a, c.tok0, c.n_tok, cs, ok);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    RopeTile pairs = c;                                      // the same rows, a pair a thread
    pairs.row_step = kThreads / half;
    const int r1 = (int)threadIdx.x / half, j = (int)threadIdx.x - r1 * half;
    const int ea = a.off + (a.interleaved ? 2 * j : j), eb = ea + (a.interleaved ? 1 : half);
    w.row(pairs, r1);
    while (r1 < pairs.row_step && w.v < c.rows) {
        if (ok[w.t]) {
            T* row = tile + w.v * a.D;
            const float x = to_f32(row[ea]), y = to_f32(row[eb]);
            const float2 q = cs[w.t * half + j];
            store_out<T>(row + ea, x * q.x - y * q.y);
            store_out<T>(row + eb, y * q.x + x * q.y);
        }
        w.next(pairs);
    }
    __syncthreads();
    w.row(c, rr0);
    w.aim(a, c, a.out, a.os, e0);
    while (moves && w.v < c.rows) {
        *reinterpret_cast<uint4*>(const_cast<T*>(w.p)) = *reinterpret_cast<const uint4*>(tile + w.v * a.D + e0);
        w.step(a, c, a.out, a.os, e0);
    }
}

template <typename T>
bool staged_supported(const RopeArgs& a) {
    constexpr int V = 16 / sizeof(T);
    if (a.D % V || a.D / V > kThreads || (pass_channels(a) == 0 && a.d_rot < a.D)) return false;   // (in place: the pairs only)
    for (int w = 0; w < 2; ++w)
        if (a.H[w] && (a.xs[w][0] % V || a.xs[w][1] % V || a.os[w][0] % V || a.os[w][1] % V)) return false;
    return true;
}

template <typename T>
cudaError_t launch_staged(const RopeArgs& a, cudaStream_t s) {
    long blocks;
    const RopeGrid g = cut(a, a.D / (16 / (int)sizeof(T)), 0, 2, &blocks);    // (a tile: kTileLimit at most)
    if (blocks > (1L << 31) - 1) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)g.tpb * g.rpb * a.D * sizeof(T) + angle_bytes(a, g);
    cudaError_t e = allow_smem(rope_staged_kernel<T>, kTileLimit + kAngleLimit, smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(rope_staged_kernel<T>, (unsigned)blocks, kThreads, smem, s, a, g);
    count_launch();
    return e;
}

// The same for any size, stride and offset: a thread keeps one pair, or one element
// that is passed on, and goes down the rows, kBatch of them in flight.  (With an item's
// row, head and token divided out for each: 46 us for 2 x 4096 tokens of 17 x 80 bf16, 50
// rotated.)
constexpr int kBatch = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_item_kernel(const __grid_constant__ RopeArgs a,
                                                             const __grid_constant__ RopeGrid g) {
    extern __shared__ __align__(16) uint8_t smem[];
    float2* cs = reinterpret_cast<float2*>(smem);
    const int half = a.d_rot / 2;
    int* ok = reinterpret_cast<int*>(cs + (size_t)g.tpb * half);
    const RopeTile c(a, g);
    grid_wait();
    fill_angles(a, c.tok0, c.n_tok, cs, ok);
    // (rows of more items than threads: one row a step, its items in turn)
    const int rr0 = g.ipr <= kThreads ? (int)threadIdx.x / g.ipr : 0;
    if (rr0 >= c.row_step) return;
    for (int it = (int)threadIdx.x - rr0 * g.ipr; it < g.ipr; it += kThreads) {
        const bool rot = it < half;
        int e0 = a.off + (a.interleaved ? 2 * it : it);
        if (!rot) {
            e0 = it - half;
            if (e0 >= a.off) e0 += a.d_rot;
        }
        const int e1 = a.interleaved ? 1 : half;             // from a pair's first element to its second
        Rows<T> in, out;
        in.row(c, rr0);
        out = in;
        in.aim(a, c, a.x, a.xs, e0);
        out.aim(a, c, a.out, a.os, e0);
        while (out.v < c.rows) {
            T u[kBatch], w[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (in.v >= c.rows) continue;
                u[b] = in.p[0];
                if (rot) w[b] = in.p[e1];
                in.step(a, c, a.x, a.xs, e0);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (out.v >= c.rows) continue;
                T* p = const_cast<T*>(out.p);
                if (rot && ok[out.t]) {
                    const float x = to_f32(u[b]), y = to_f32(w[b]);
                    const float2 q = cs[out.t * half + it];
                    store_out<T>(p, x * q.x - y * q.y);
                    store_out<T>(p + e1, y * q.x + x * q.y);
                } else {
                    p[0] = u[b];
                    if (rot) p[e1] = w[b];
                }
                out.step(a, c, a.out, a.os, e0);
            }
        }
    }
}

template <typename T>
cudaError_t launch_items(const RopeArgs& a, cudaStream_t s) {
    long blocks;
    const RopeGrid g = cut(a, a.d_rot / 2, pass_channels(a), 8, &blocks);
    if (blocks > (1L << 31) - 1) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_dependent(rope_item_kernel<T>, (unsigned)blocks, kThreads, angle_bytes(a, g), s, a, g);
    count_launch();
    return e;
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, cudaStream_t s) {
    // 16-byte items need sizes and strides that are whole vectors, 16-byte rows a head of them
    if (vec_supported<T>(a)) return launch_vec<T>(a, s);
    if (staged_supported<T>(a)) return launch_staged<T>(a, s);
    return launch_items<T>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    return a.dt == DT_F32 ? launch_typed<float>(a, s) : launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace csa
