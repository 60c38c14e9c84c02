// Rotary positions: part of each head turned by an angle that grows with the position.
//
// Pair i of the rotated dims (a, b) = (x[2i], x[2i+1]) (interleaved) or (x[i],
// x[i + dims/2]) (halves) becomes m (a cos t - b sin t, a sin t + b cos t) with
// t = position * f_i, f_i the pair's frequency (the host's table: plain, linear, NTK or
// YaRN scaling) and m the scaling's magnitude. The transposed rotation (sin negated) is
// the gradient, and the inverse where m = 1.
//
// Angles: a position of 2^20 times f_0 = 1 leaves an fp32 product no bits for the
// fraction of a turn. The table holds each frequency (computed in 64-bit floating point) in
// turns, as a 64-bit fixed-point fraction, so that position * step wraps modulo one turn
// exactly; the top 32 bits of the wrapped product are the angle that sincospif takes. What
// is left is the frequency's own rounding, at most |position| * 2^-55 turns, and fp32's.
//
// Bound: memory (each value read and written once). cos and sin of a (token, pair) serve
// every head, so a thread takes one chunk of a token's rotated dims for several heads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ds4sp {

constexpr int kRopeMaxDims = 256;

struct RopeTable {
    uint64_t step[kRopeMaxDims / 2];   // turns per position, as a fraction of 2^64
    float m;                           // magnitude of cos and sin
    int dims, offset, half_layout;     // half_layout: 0 = pairs (2i, 2i+1), 1 = (i, i + dims/2)
    int transpose;
};

// (m cos, m sin) of `position` times the pair's frequency.
__device__ __forceinline__ float2 rope_turn(uint64_t step, long long position, float m) {
    const int32_t turns = (int32_t)(((uint64_t)position * step) >> 32);   // modulo one turn
    const int32_t near = (turns + 64) & ~127;                             // exact in fp32
    float s, c;
    sincospif((float)near * 0x1p-31f, &s, &c);
    // the rest of the angle (at most 2^-25 of half a turn), to first order
    const float r = (float)(turns - near) * (0x1p-31f * 3.14159265f);
    return make_float2(m * fmaf(-s, r, c), m * fmaf(c, r, s));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// V values moved as one access of V * sizeof(T) bytes.
template <class T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
};

struct RopeParams {
    RopeTable tab;
    const void* x;
    void* out;
    const int32_t* positions;          // NULL: pos0 + i * pos_step
    long long x_ts, x_hs, o_ts, o_hs;  // token and head strides, in values
    long long pos0, pos_step;
    int n, heads;
    int rot, per_head;                 // chunks of a head: rotated, all of them
    int groups;                        // heads / heads per thread, rounded up
};

// A chunk is V values (two for V = 1 interleaved); a halves-layout chunk is V values of
// the first half and their partners in the second. Chunks [0, rot) of a head are its
// rotated dims, [rot, per_head) the dims copied beside them. Thread: one chunk of one
// token for HPT heads, `groups` apart, so that a warp's accesses of one step are the
// chunks of neighbouring heads.
template <class T, int V, int HPT>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int C = V < 2 ? 2 : V;                      // values of an interleaved chunk
    __shared__ uint64_t step[kRopeMaxDims / 2];
    for (int i = threadIdx.x; i < p.tab.dims / 2; i += 256) step[i] = p.tab.step[i];
    __syncthreads();
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int per_token = p.groups * p.per_head;
    const long long tok = id / per_token;
    if (tok >= p.n) return;
    const int rest = (int)(id - tok * per_token), hg = rest / p.per_head, ch = rest - hg * p.per_head;
    const T* x = static_cast<const T*>(p.x) + tok * p.x_ts;
    T* out = static_cast<T*>(p.out) + tok * p.o_ts;
    using W = Vec<T, V>;
    if (ch >= p.rot) {                                    // a copied chunk
        int d = (ch - p.rot) * V;
        if (d >= p.tab.offset) d += p.tab.dims;
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
            const int h = hg + j * p.groups;
            if (h < p.heads)
                *reinterpret_cast<W*>(out + h * p.o_hs + d) = *reinterpret_cast<const W*>(x + h * p.x_hs + d);
        }
        return;
    }
    const long long pos = p.positions ? (long long)p.positions[tok] : p.pos0 + tok * p.pos_step;
    const float sign = p.tab.transpose ? -1.f : 1.f;
    if (p.tab.half_layout) {
        float2 cs[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            cs[i] = rope_turn(step[ch * V + i], pos, p.tab.m);
            cs[i].y *= sign;
        }
        const int da = p.tab.offset + ch * V, db = da + p.tab.dims / 2;
        W a[HPT], b[HPT];
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
            const int h = hg + j * p.groups;
            if (h < p.heads) {
                a[j] = *reinterpret_cast<const W*>(x + h * p.x_hs + da);
                b[j] = *reinterpret_cast<const W*>(x + h * p.x_hs + db);
            }
        }
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
            const int h = hg + j * p.groups;
            if (h >= p.heads) continue;
            W u, v;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float fa = to_f32(a[j].v[i]), fb = to_f32(b[j].v[i]);
                u.v[i] = from_f32<T>(fa * cs[i].x - fb * cs[i].y);
                v.v[i] = from_f32<T>(fa * cs[i].y + fb * cs[i].x);
            }
            *reinterpret_cast<W*>(out + h * p.o_hs + da) = u;
            *reinterpret_cast<W*>(out + h * p.o_hs + db) = v;
        }
    } else {
        float2 cs[C / 2];
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            cs[i] = rope_turn(step[ch * (C / 2) + i], pos, p.tab.m);
            cs[i].y *= sign;
        }
        const int d = p.tab.offset + ch * C;
        W a[HPT][C / V];
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
            const int h = hg + j * p.groups;
            if (h < p.heads)
#pragma unroll
                for (int w = 0; w < C / V; ++w)
                    a[j][w] = *reinterpret_cast<const W*>(x + h * p.x_hs + d + w * V);
        }
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
            const int h = hg + j * p.groups;
            if (h >= p.heads) continue;
            T r[C];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                const float fa = to_f32(a[j][2 * i / V].v[2 * i % V]);
                const float fb = to_f32(a[j][(2 * i + 1) / V].v[(2 * i + 1) % V]);
                r[2 * i] = from_f32<T>(fa * cs[i].x - fb * cs[i].y);
                r[2 * i + 1] = from_f32<T>(fa * cs[i].y + fb * cs[i].x);
            }
#pragma unroll
            for (int w = 0; w < C / V; ++w) {
                W o;
#pragma unroll
                for (int i = 0; i < V; ++i) o.v[i] = r[w * V + i];
                *reinterpret_cast<W*>(out + h * p.o_hs + d + w * V) = o;
            }
        }
    }
}

}  // namespace ds4sp
