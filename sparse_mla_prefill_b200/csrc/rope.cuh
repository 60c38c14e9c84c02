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
// Bound: memory (each value read and written once). A block takes a few tokens (or a slice
// of one with very many heads): it computes their cos and sin once, into shared memory, for
// all heads, then walks their chunks, four loads in flight per thread.
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

// Quotients by a divisor d of values v with v * d < 2^32, as a multiplication by ceil(2^32 / d).
struct SmallDiv {
    uint32_t d, m;
    __host__ void set(uint32_t divisor) {
        d = divisor;
        m = (uint32_t)(((1ull << 32) + divisor - 1) / divisor);      // 0 (2^32) for a divisor of 1
    }
    __device__ __forceinline__ uint32_t div(uint32_t v) const { return m ? __umulhi(v, m) : v; }
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxHead = 32768;    // values of a head at most: (kRopeMaxHead + kRopeChunks) of
                                       // its chunks times itself is below 2^32
constexpr int kRopeChunks = 4096;      // chunks of a block at most
constexpr int kRopeTurns = 2048;       // (token, pair) of a block at most

struct RopeParams {
    RopeTable tab;
    const void* x;
    void* out;
    const int32_t* positions;          // NULL: pos0 + i * pos_step
    long long x_ts, x_hs, o_ts, o_hs;  // token and head strides, in values
    long long pos0, pos_step;
    int n, heads;
    int rot, per_head;                 // chunks of a head: rotated, all of them
    int tokens;                        // tokens of a block; 1 where a token has several blocks
    int slices;                        // blocks per token (tokens == 1)
    SmallDiv by_head, by_token;        // chunks of a head, of a token
};

// A chunk is V values (two for V = 1 interleaved); a halves-layout chunk is V values of
// the first half and their partners in the second. Chunks [0, rot) of a head are its
// rotated dims, [rot, per_head) the dims copied beside them.
template <class T, int V, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int C = HALVES || V > 1 ? V : 2;            // values of a chunk (of each half)
    constexpr int P = HALVES ? C : C / 2;                 // pairs of a chunk
    constexpr int U = HALVES ? 2 : 4;                     // chunks in flight per thread: 64 bytes
    extern __shared__ float2 turn[];                      // [token][pair]
    using W = Vec<T, V>;
    const int pairs = p.tab.dims / 2, tid = threadIdx.x;
    const int tok0 = p.slices > 1 ? blockIdx.x / p.slices : blockIdx.x * p.tokens;
    const int n_tok = min(p.tokens, p.n - tok0);
    const int c0 = p.slices > 1 ? blockIdx.x % p.slices * kRopeChunks : 0;   // of the token's chunks
    for (int i = tid; i < n_tok * pairs; i += kRopeThreads) {
        const int t = i / pairs;
        const long long pos = p.positions ? (long long)p.positions[tok0 + t] : p.pos0 + (tok0 + t) * p.pos_step;
        const float2 cs = rope_turn(p.tab.step[i - t * pairs], pos, p.tab.m);
        turn[i] = make_float2(cs.x, p.tab.transpose ? -cs.y : cs.y);
    }
    __syncthreads();
    const int h0 = c0 / p.per_head, first = c0 - h0 * p.per_head;
    const int total = p.slices > 1 ? min(kRopeChunks, (int)p.by_token.d - c0) : n_tok * (int)p.by_token.d;
#pragma unroll 1
    for (int base = tid; base < total; base += U * kRopeThreads) {
        const T* src[U];
        T* dst[U];
        const float2* cs[U];                              // NULL: a copied chunk
        W a[U][HALVES ? 2 : C / V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = base + u * kRopeThreads;
            if (c >= total) break;
            const uint32_t t = p.slices > 1 ? 0 : p.by_token.div(c), in_tok = c - t * p.by_token.d + first;
            const uint32_t hh = p.by_head.div(in_tok), h = hh + h0;
            int ch = (int)(in_tok - hh * p.by_head.d), d;
            if (ch < p.rot) {
                cs[u] = turn + t * pairs + ch * P;
                d = p.tab.offset + ch * C;
            } else {
                cs[u] = nullptr;
                d = (ch - p.rot) * V;
                if (d >= p.tab.offset) d += p.tab.dims;
            }
            src[u] = static_cast<const T*>(p.x) + (tok0 + (long long)t) * p.x_ts + h * p.x_hs + d;
            dst[u] = static_cast<T*>(p.out) + (tok0 + (long long)t) * p.o_ts + h * p.o_hs + d;
            a[u][0] = *reinterpret_cast<const W*>(src[u]);
            if (cs[u]) {
                if constexpr (HALVES) a[u][1] = *reinterpret_cast<const W*>(src[u] + pairs);
                else if constexpr (C > V) a[u][1] = *reinterpret_cast<const W*>(src[u] + V);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * kRopeThreads >= total) break;
            if (!cs[u]) {
                *reinterpret_cast<W*>(dst[u]) = a[u][0];
                continue;
            }
            W o[HALVES ? 2 : C / V];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 r = cs[u][i];
                // the pair's places in the loaded vectors
                const int va = HALVES ? 0 : 2 * i / V, ia = HALVES ? i : 2 * i % V;
                const int vb = HALVES ? 1 : (2 * i + 1) / V, ib = HALVES ? i : (2 * i + 1) % V;
                const float fa = to_f32(a[u][va].v[ia]), fb = to_f32(a[u][vb].v[ib]);
                o[va].v[ia] = from_f32<T>(fa * r.x - fb * r.y);
                o[vb].v[ib] = from_f32<T>(fa * r.y + fb * r.x);
            }
            *reinterpret_cast<W*>(dst[u]) = o[0];
            if constexpr (HALVES) *reinterpret_cast<W*>(dst[u] + pairs) = o[1];
            else if constexpr (C > V) *reinterpret_cast<W*>(dst[u] + V) = o[1];
        }
    }
}

}  // namespace ds4sp
