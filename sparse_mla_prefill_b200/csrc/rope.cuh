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
// exactly. The wrapped product's top two bits (rounded) are the quadrant, the 32 below them
// the angle within it, in [-pi/4, pi/4): cos and sin are their Taylor sums in 64-bit floating
// point (off by at most 2^-37), times m, each rounded to fp32 once. What is left is the
// frequency's own rounding, at most |position| * (f_i * 2^-50 + 2^-61) radians, and fp32's. (In
// fp32 throughout, with roundings of cos, of sin, of the angle's remainder and of their products
// with m, rotated rows written in 8 bits were 2.2 times as far from the exact ones. A table of 256
// angles as sums of two fp32 values, with fp32 sums for the rest, measured no faster.)
//
// Bound: memory (each value read and written once). A thread keeps one chunk of the head and
// walks rows (token, head), four loads in flight; the block computes its tokens' cos and sin
// once, into shared memory, for all heads, while its first loads are on their way. Measured:
// 10,240 tokens x 64 heads of 128 bf16 values (336 MB) in 52.4 us, the copy rate; 10,240 x 16
// heads of 64 fp16 values from rows of 192 into rows of 576 (42 MB in 128-byte pieces) in 10.5 us.
// With a thread per chunk that computed its own cos and sin the first took 150 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ds4sp {

constexpr int kRopeMaxDims = 256;

struct RopeTable {
    uint64_t step[kRopeMaxDims / 2];   // turns per position, as a fraction of 2^64
    double m;                          // magnitude of cos and sin
    int dims, offset, half_layout;     // half_layout: 0 = pairs (2i, 2i+1), 1 = (i, i + dims/2)
    int transpose;
};

// (m cos, m sin) of `position` times the pair's frequency, in 64 bits.
__device__ __forceinline__ double2 rope_turn_f64(uint64_t step, long long position, double m) {
    const uint64_t turns = (uint64_t)position * step;                     // modulo one turn
    const uint32_t quadrant = (uint32_t)((turns + (1ull << 61)) >> 62);
    const double t = (double)(int32_t)(uint32_t)(turns >> 30) * (1.5707963267948966 * 0x1p-32);
    const double t2 = t * t;
    double s = fma(t2, -1.0 / 39916800.0, 1.0 / 362880.0);
    s = fma(t2, s, -1.0 / 5040.0);
    s = fma(t2, s, 1.0 / 120.0);
    s = fma(t2, s, -1.0 / 6.0);
    s = m * fma(t * t2, s, t);
    double c = fma(t2, 1.0 / 479001600.0, -1.0 / 3628800.0);
    c = fma(t2, c, 1.0 / 40320.0);
    c = fma(t2, c, -1.0 / 720.0);
    c = fma(t2, c, 1.0 / 24.0);
    c = fma(t2, c, -0.5);
    c = m * fma(t2, c, 1.0);
    const bool swap = quadrant & 1u;
    const double u = swap ? s : c, v = swap ? c : s;
    return make_double2(((quadrant + 1u) & 2u) ? -u : u, (quadrant & 2u) ? -v : v);
}

// The same, each rounded once.
__device__ __forceinline__ float2 rope_turn(uint64_t step, long long position, double m) {
    const double2 cs = rope_turn_f64(step, position, m);
    return make_float2((float)cs.x, (float)cs.y);
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

// Two neighbouring values as fp32, and back, rounded once: one 32-bit word for 16-bit types.
__device__ __forceinline__ float2 pair_f32(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 pair_f32(const __half* v) {
    return __half22float2(*reinterpret_cast<const __half2*>(v));
}
__device__ __forceinline__ float2 pair_f32(const __nv_bfloat16* v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(v));
}
__device__ __forceinline__ void put_pair(float* v, float a, float b) {
    v[0] = a;
    v[1] = b;
}
__device__ __forceinline__ void put_pair(__half* v, float a, float b) {
    *reinterpret_cast<__half2*>(v) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void put_pair(__nv_bfloat16* v, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(v) = __floats2bfloat162_rn(a, b);
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
constexpr int kRopeTurns = 2048;       // (token, pair) of a block at most
constexpr int rope_rows(bool halves) { return halves ? 2 : 4; }    // rows in flight per thread

struct RopeParams {
    RopeTable tab;
    const void* x;
    void* out;
    const int32_t* positions;          // NULL: pos0 + i * pos_step
    long long x_ts, x_hs, o_ts, o_hs;  // token and head strides, in values
    long long pos0, pos_step;
    int n, heads;
    int rot, per_head;                 // chunks of a head: rotated, all of them
    int tokens;                        // tokens of a block (heads * tokens below 2^16 where above 1)
    int groups;                        // rows a block walks side by side
    SmallDiv by_width, by_heads;       // threads of a row, heads of a token
};

// A chunk is V values (two for V = 1 interleaved); a halves-layout chunk is V values of
// the first half and their partners in the second. Chunks [0, rot) of a head are its
// rotated dims, [rot, per_head) the dims copied beside them. blockIdx.y counts chunks by the
// width of a row where a head has more of them than the block threads.
template <class T, int V, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int C = HALVES || V > 1 ? V : 2;            // values of a chunk (of each half)
    constexpr int P = HALVES ? C : C / 2;                 // pairs of a chunk
    constexpr int U = rope_rows(HALVES);                  // 64 bytes of wide accesses
    constexpr int L = HALVES || C > V ? 2 : 1;            // accesses of a chunk
    extern __shared__ float2 turn[];                      // [token][pair]
    using W = Vec<T, V>;
    const int pairs = p.tab.dims / 2, tid = threadIdx.x, apart = HALVES ? pairs : V;
    const int tok0 = blockIdx.x * p.tokens, n_tok = min(p.tokens, p.n - tok0);
    const int group = (int)p.by_width.div(tid), ch = tid - group * (int)p.by_width.d + blockIdx.y * (int)p.by_width.d;
    const bool rot = ch < p.rot;
    const int rows = group < p.groups && ch < p.per_head ? n_tok * p.heads : 0;
    int d = rot ? p.tab.offset + ch * C : (ch - p.rot) * V;
    if (!rot && d >= p.tab.offset) d += p.tab.dims;
    const T* x = static_cast<const T*>(p.x) + tok0 * p.x_ts + d;
    T* out = static_cast<T*>(p.out) + tok0 * p.o_ts + d;
    W a[U][L];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r0 + u * p.groups;
            if (row >= rows) break;
            const int t = p.tokens > 1 ? (int)p.by_heads.div(row) : 0, h = row - t * p.heads;
            const T* src = x + t * p.x_ts + h * p.x_hs;
            a[u][0] = *reinterpret_cast<const W*>(src);
            if (L > 1 && rot) a[u][L - 1] = *reinterpret_cast<const W*>(src + apart);
        }
    };
    load(group);
    for (int i = tid; i < n_tok * pairs; i += kRopeThreads) {
        const int t = i / pairs;
        const long long pos = p.positions ? (long long)p.positions[tok0 + t] : p.pos0 + (tok0 + t) * p.pos_step;
        const float2 cs = rope_turn(p.tab.step[i - t * pairs], pos, p.tab.m);
        turn[i] = make_float2(cs.x, p.tab.transpose ? -cs.y : cs.y);
    }
    __syncthreads();
    float2 cs[P];                                         // of the token held
    int held = -1;
#pragma unroll 1
    for (int r0 = group; r0 < rows; r0 += U * p.groups) {
        if (r0 != group) load(r0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r0 + u * p.groups;
            if (row >= rows) break;
            const int t = p.tokens > 1 ? (int)p.by_heads.div(row) : 0, h = row - t * p.heads;
            if (rot) {
                if (t != held) {
                    held = t;
#pragma unroll
                    for (int i = 0; i < P; ++i) cs[i] = turn[t * pairs + ch * P + i];
                }
                if constexpr (HALVES && V > 1) {
#pragma unroll
                    for (int i = 0; i < P; i += 2) {
                        const float2 fa = pair_f32(&a[u][0].v[i]), fb = pair_f32(&a[u][1].v[i]);
                        put_pair(&a[u][0].v[i], fa.x * cs[i].x - fb.x * cs[i].y, fa.y * cs[i + 1].x - fb.y * cs[i + 1].y);
                        put_pair(&a[u][1].v[i], fa.x * cs[i].y + fb.x * cs[i].x, fa.y * cs[i + 1].y + fb.y * cs[i + 1].x);
                    }
                } else if constexpr (V > 1) {
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 f = pair_f32(&a[u][0].v[2 * i]);
                        put_pair(&a[u][0].v[2 * i], f.x * cs[i].x - f.y * cs[i].y, f.x * cs[i].y + f.y * cs[i].x);
                    }
                } else {
                    const float fa = to_f32(a[u][0].v[0]), fb = to_f32(a[u][1].v[0]);
                    a[u][0].v[0] = from_f32<T>(fa * cs[0].x - fb * cs[0].y);
                    a[u][1].v[0] = from_f32<T>(fa * cs[0].y + fb * cs[0].x);
                }
            }
            T* dst = out + t * p.o_ts + h * p.o_hs;
            *reinterpret_cast<W*>(dst) = a[u][0];
            if (L > 1 && rot) *reinterpret_cast<W*>(dst + apart) = a[u][L - 1];
        }
    }
}

}  // namespace ds4sp
