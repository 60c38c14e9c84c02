// Writing latent rows to a cache as they are produced, and reading them back.
//
// A row of x (fp16, bf16 or fp32) is rotated (optionally, the rotary part of the row:
// rope.cuh's arithmetic, kept in fp32, or in 64 bits for kv_format 5) and stored in the cache's
// format: fp16, the block formats of quant_kv.cuh, or kv_format 5, whose rows the scaled
// attention reads:
//
//   e4m3 codes with one scale 2^e for each block of 64 rows; value = code * 2^e.
//   e is the smallest integer with max|x| <= 448 * 2^e over the block's finite values,
//   within [-40, 40] (all zero: -40); larger values, infinities among them, saturate at
//   +-448 * 2^e, and a NaN stays one. A power of two costs a floating code no precision
//   (only the smallest values lose range) and makes every stored value an exact product.
//   The rows of block b are stored at places 65b .. 65b+63, and place 65b+64 is the
//   block's record: its scale as fp32, then zeros. Places are `dims` bytes.
//
// A write that starts inside a block keeps the rows before it: the block's scale becomes
// the larger of its own and the new rows', and if it grew the earlier codes are rounded
// again to it. Rows after the written ones are left as they are.
//
// Bound: memory. Writing reads x once and stores codes; a CTA holds its block's rows in
// registers between the maximum and the rounding.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "quant_kv.cuh"
#include "rope.cuh"

namespace ds4sp {

constexpr int kFmtE4M3 = 5;
constexpr int kScaleBlock = 64;                 // rows that share a scale
constexpr int kScaleExpMax = 40;
constexpr float kE4M3Max = 448.f;

__host__ __device__ constexpr long long e4m3_place(long long row) { return row + row / kScaleBlock; }

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// The smallest e with top <= 448 * 2^e, in [-40, 40]. top is finite and >= 0.
__device__ __forceinline__ int scale_exponent(float top) {
    if (top == 0.f) return -kScaleExpMax;
    // top < 2^(x+1) with x its exponent; 448 = 1.75 * 2^8
    int e = max((int)(__float_as_uint(top) >> 23) - 127, -126) - 8;
    e = min(max(e, -kScaleExpMax), kScaleExpMax);
    if (top > kE4M3Max * pow2f(e)) ++e;
    return min(e, kScaleExpMax);
}

struct CacheRows {                              // the rows a write takes
    const void* x;
    long long x_ld;                             // in values
    const int32_t* positions;                   // NULL: pos0 + i * pos_step
    long long pos0, pos_step;
    int n, row0, dims;
    int rotate;                                 // apply the table
    int fast;                                   // x's rows are 16-byte aligned, and no chunk of
                                                // eight is partly rotated
};

template <class T>
union Eight {
    uint4 q[sizeof(T) / 2];
    T e[8];
};
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const T* src) {          // 16-byte aligned
    Eight<T> a;
#pragma unroll
    for (int w = 0; w < (int)sizeof(T) / 2; ++w) a.q[w] = __ldg(reinterpret_cast<const uint4*>(src) + w);
    return a;
}

__device__ __forceinline__ long long position_of(const CacheRows& p, int i) {
    return p.positions ? (long long)__ldg(p.positions + i) : p.pos0 + i * p.pos_step;
}

// Whether chunk c of eight values is rotated (p.fast: all of it or none).
__device__ __forceinline__ bool turned(const CacheRows& p, const RopeTable& tab, int c) {
    return p.rotate && 8 * c >= tab.offset && 8 * c < tab.offset + tab.dims;
}

// A 64-bit value cut to fp32, the last bit set where anything was cut off, so that a later
// rounding to fewer bits is the rounding of the 64-bit value. (Turned in fp32, or rounded to it
// in between, one value in some millions lands on the wrong side of a border, a whole step of
// its code.)
__device__ __forceinline__ float cut_odd(double v) {
    return __uint_as_float(__float_as_uint(__double2float_rz(v)) | ((__double2loint(v) & 0x1fffffff) != 0));
}
// How a row's pair of values is turned: in 64 bits, cut as above (kv_format 5),
struct TurnOdd {
    const uint64_t* step;
    long long pos;
    double m;
    __device__ __forceinline__ float2 operator()(int pair, float a, float b) const {
        const double2 cs = rope_turn_f64(step[pair], pos, m);
        const double x = a, y = b;
        return make_float2(cut_odd(x * cs.x - y * cs.y), cut_odd(x * cs.y + y * cs.x));
    }
};
// or as ds4sp_rope does, with the row's cos and sin at hand.
struct TurnBy {
    const float2* cs;
    __device__ __forceinline__ float2 operator()(int pair, float a, float b) const {
        return make_float2(a * cs[pair].x - b * cs[pair].y, a * cs[pair].y + b * cs[pair].x);
    }
};

struct TurnNot {};                              // no row is turned (p.rotate is 0)
// A rotated chunk c of row i, loaded as `a`, in fp32 (p.fast).
template <class T, class Turn>
__device__ __forceinline__ void turn_eight(const CacheRows& p, const RopeTable& tab, const Turn& turn, int i,
                                           int c, const Eight<T>& a, float (&v)[8]) {
    const int r0 = 8 * c - tab.offset, half = tab.dims / 2;
    if (tab.half_layout) {
        const bool upper = r0 >= half;
        const Eight<T> b = load_eight(static_cast<const T*>(p.x) + i * p.x_ld + 8 * c + (upper ? -half : half));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = to_f32(a.e[k]), o = to_f32(b.e[k]);
            const float2 t = turn((upper ? r0 - half : r0) + k, upper ? o : s, upper ? s : o);
            v[k] = upper ? t.y : t.x;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = turn(r0 / 2 + k, to_f32(a.e[2 * k]), to_f32(a.e[2 * k + 1]));
            v[2 * k] = t.x;
            v[2 * k + 1] = t.y;
        }
    }
}

// Eight values of row i (of the n written) at dims 8c .. 8c+7, rotated, in fp32.
template <class T, class Turn>
__device__ __forceinline__ void load_chunk(const CacheRows& p, const RopeTable& tab, const Turn& turn,
                                           int i, int c, float (&v)[8]) {
    constexpr bool kTurns = !std::is_same<Turn, TurnNot>::value;
    const T* row = static_cast<const T*>(p.x) + i * p.x_ld;
    const int d0 = 8 * c;
    if (p.fast) {
        const Eight<T> a = load_eight(row + d0);
        if constexpr (kTurns)
            if (turned(p, tab, c)) {
                turn_eight<T>(p, tab, turn, i, c, a, v);
                return;
            }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = to_f32(a.e[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int d = d0 + k, r = d - tab.offset, half = tab.dims / 2;
        v[k] = to_f32(row[d]);
        if constexpr (kTurns) {
            if (!p.rotate || r < 0 || r >= tab.dims) continue;
            const bool second = tab.half_layout ? r >= half : r & 1;
            const int pair = tab.half_layout ? (second ? r - half : r) : r / 2;
            const int od = tab.half_layout ? (second ? d - half : d + half) : (second ? d - 1 : d + 1);
            const float o = to_f32(row[od]);
            const float2 t = turn(pair, second ? o : v[k], second ? v[k] : o);
            v[k] = second ? t.y : t.x;
        }
    }
}

__device__ __forceinline__ void load_steps(const RopeTable& tab, int rotate, uint64_t* step) {
    if (rotate)
        for (int i = threadIdx.x; i < tab.dims / 2; i += blockDim.x) step[i] = tab.step[i];
    __syncthreads();
}

// ---------------------------------------------------------------- fp16, Q8_0, Q4_0, Q8 K / Q4 V

// The code bytes of eight values of a Q8_0 block of scale d.
__device__ __forceinline__ uint2 q8_codes(const float (&v)[8], float d) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float q = d == 0.f ? 0.f : fminf(fmaxf(rintf(v[k] / d), -127.f), 127.f);
        w[k / 4] |= (uint32_t)(uint8_t)(int8_t)(int)q << (8 * (k % 4));
    }
    return make_uint2(w[0], w[1]);
}

// The codes of eight values of a Q4_0 block of scale d, one per byte.
__device__ __forceinline__ uint2 q4_codes(const float (&v)[8], float d) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t n = d == 0.f ? 8u : (uint32_t)(int)fminf(fmaxf(rintf(v[k] / d) + 8.f, 0.f), 15.f);
        w[k / 4] |= n << (8 * (k % 4));
    }
    return make_uint2(w[0], w[1]);
}

constexpr int kWriteTurns = 1280;               // (256 / 32 + 2) rows of 128 pairs; other widths have fewer

// Four lanes per block of 32 values, eight values each: the block's largest magnitude (and
// for Q4_0 its first extreme) over the four by shuffles, the codes as in quantize_rows_kernel.
// Rows are stored at out + row * row_bytes. FMT: kFmtF16, kFmtQ8, kFmtQ4 or kFmtQ8Q4.
// TURNED: whether rows are rotated. Measured, 122,880 fp16 rows of 576, without a rotation and with
// 64 rotary dims: fp16 rows 49 and 80 us, Q8_0 102 and 143, Q4_0 103 and 148, Q8 K / Q4 V 166 and
// 213 (the last is 254 MB, 39 us at the copy rate: the quotients bound it, not memory).
template <class T, int FMT, bool TURNED>
__global__ void __launch_bounds__(256)
cache_write_kernel(const __grid_constant__ CacheRows p, const __grid_constant__ RopeTable tab, uint8_t* __restrict__ out,
                   int row_bytes) {
    const int chunks = p.dims / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const bool in = id < (long long)p.n * chunks;
    const int i = in ? (int)(id / chunks) : 0, c = in ? (int)(id % chunks) : 0;
    float v[8];
    if constexpr (TURNED) {
        // The turns of the block's rows, from `first` on (at most 256 / chunks + 2 of them, of
        // min(4 chunks, 128) pairs), a thread one at a time.
        __shared__ float2 turns[kWriteTurns];
        const int first = (int)((long long)blockIdx.x * 256 / chunks), pairs = tab.dims / 2;
        const int rows = min((int)(((long long)blockIdx.x * 256 + 255) / chunks) + 1, p.n) - first;
        for (int k = threadIdx.x; k < rows * pairs; k += 256)
            turns[k] = rope_turn(tab.step[k % pairs], position_of(p, first + k / pairs), tab.m);
        __syncthreads();
        load_chunk<T>(p, tab, TurnBy{turns + (in ? i - first : 0) * pairs}, i, c, v);
    } else {
        load_chunk<T>(p, tab, TurnNot{}, i, c, v);
    }
    uint8_t* row = out + (long long)(p.row0 + i) * row_bytes;
    if constexpr (FMT == kFmtF16) {
        if (!in) return;
        uint4 w;
        w.x = pack_half2(v[0], v[1]);
        w.y = pack_half2(v[2], v[3]);
        w.z = pack_half2(v[4], v[5]);
        w.w = pack_half2(v[6], v[7]);
        *reinterpret_cast<uint4*>(row + 16 * c) = w;
    } else {
        // (dims is a multiple of 32: a block's four lanes lie in one warp and one row)
        float m = 0.f, am = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (fabsf(v[k]) > am) {
                am = fabsf(v[k]);
                m = v[k];
            }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {      // strictly larger, or equal from a lower lane
            const float om = __shfl_xor_sync(0xffffffffu, m, off), oam = fabsf(om);
            if (oam > am || (oam == am && (threadIdx.x & off))) {
                am = oam;
                m = om;
            }
        }
        const int b = c / 4, l = c % 4;
        auto scale_bytes = [&](uint8_t* part, int fmt, int dims, __half d16) {
            const int cb = quant_code_bytes(fmt, dims), nb = dims / kQBlock;
            if (l == 0) *reinterpret_cast<__half*>(part + cb + 2 * b) = d16;
            if (b == 0 && l == 1)
                for (int k = cb + 2 * nb; k < quant_row_bytes(fmt, dims); k += 2)
                    *reinterpret_cast<uint16_t*>(part + k) = 0;
        };
        if constexpr (FMT == kFmtQ8 || FMT == kFmtQ8Q4) {
            const __half d16 = __float2half_rn(am / 127.f);
            const uint2 w = q8_codes(v, __half2float(d16));
            if (in) {
                *reinterpret_cast<uint2*>(row + 8 * c) = w;
                scale_bytes(row, kFmtQ8, p.dims, d16);
            }
        }
        if constexpr (FMT == kFmtQ4 || FMT == kFmtQ8Q4) {
            __half d16 = __float2half_rn(m / -8.f);
            if (__half2float(d16) == 0.f) d16 = __float2half_rn(0.f);
            const uint2 w = q4_codes(v, __half2float(d16));
            uint2 hi;                                   // values 16.. of the block: lanes 2, 3
            hi.x = __shfl_xor_sync(0xffffffffu, w.x, 2);
            hi.y = __shfl_xor_sync(0xffffffffu, w.y, 2);
            uint8_t* part = row + (FMT == kFmtQ8Q4 ? quant_row_bytes(kFmtQ8, p.dims) : 0);
            const int dims = FMT == kFmtQ8Q4 ? kValueDims : p.dims;
            if (in && 8 * c < dims) {
                if (l < 2) *reinterpret_cast<uint2*>(part + 16 * b + 8 * l) = make_uint2(w.x | hi.x << 4, w.y | hi.y << 4);
                scale_bytes(part, kFmtQ4, dims, d16);
            }
        }
    }
}

// ---------------------------------------------------------------- e4m3 with a scale per block

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// fp16 values of two e4m3 codes (exact).
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return *reinterpret_cast<const __half2*>(&r);
}

constexpr int kE4M3Threads = 512;               // 64 rows x 8 lanes
constexpr int kE4M3Held = 9;                    // steps of 64 dims held in registers: up to 576 dims

// The larger of `top` and the finite magnitudes of eight values.
__device__ __forceinline__ float top_of(const float (&u)[8], float top) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float a = fabsf(u[k]);
        if (a <= 3.402823466e38f) top = fmaxf(top, a);
    }
    return top;
}
template <class T>
__device__ __forceinline__ float top_of(const Eight<T>& a, float top) {
    float u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = to_f32(a.e[k]);
    return top_of(u, top);
}

// The larger of `top` (a value, or two) and a chunk's magnitudes: infinities included, NaNs not.
__device__ __forceinline__ float larger(float top, float v) { return fmaxf(top, fabsf(v)); }
__device__ __forceinline__ __half2 larger(__half2 top, __half2 v) { return __hmax2(top, __habs2(v)); }
__device__ __forceinline__ __nv_bfloat162 larger(__nv_bfloat162 top, __nv_bfloat162 v) { return __hmax2(top, __habs2(v)); }
template <class T> struct Packed { using type = __half2; };
template <> struct Packed<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct Packed<float> { using type = float; };
template <class T>
__device__ __forceinline__ typename Packed<T>::type top_packed(const Eight<T>& a, typename Packed<T>::type top) {
#pragma unroll
    for (int w = 0; w < (int)sizeof(T) / 2; ++w) {
        const uint32_t u[4] = {a.q[w].x, a.q[w].y, a.q[w].z, a.q[w].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = larger(top, *reinterpret_cast<const typename Packed<T>::type*>(&u[k]));
    }
    return top;
}
__device__ __forceinline__ float top_value(float top) { return top; }
__device__ __forceinline__ float top_value(__half2 top) { return fmaxf(__low2float(top), __high2float(top)); }
__device__ __forceinline__ float top_value(__nv_bfloat162 top) { return fmaxf(__low2float(top), __high2float(top)); }

// Eight values times 2^-e (inv, twice) as codes.
__device__ __forceinline__ uint2 codes_of(const float (&u)[8], unsigned long long inv2) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float2 v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%2, %3};\n\tmul.rn.f32x2 t, t, %4;\n\tmov.b64 {%0, %1}, t;\n\t}"
                : "=f"(v[k].x), "=f"(v[k].y)
                : "f"(u[4 * h + 2 * k]), "f"(u[4 * h + 2 * k + 1]), "l"(inv2));
        w[h] = e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
    return make_uint2(w[0], w[1]);
}
template <class T>
__device__ __forceinline__ uint2 codes_of(const Eight<T>& a, unsigned long long inv2) {
    float u[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float2 f = pair_f32(&a.e[k]);
        u[k] = f.x;
        u[k + 1] = f.y;
    }
    return codes_of(u, inv2);
}

// One CTA per block of 64 rows that the write touches; eight lanes a row, each taking every
// eighth chunk of eight values. HELD (up to 576 dims, aligned): the unrotated values as they
// were loaded stay in registers between the block's maximum and the rounding, all loads in
// flight at once (16-bit values: 64 registers, two CTAs an SM, so that one block's loads run
// under the other's arithmetic), and of a rotated part of up to 64 dims (kTurnedOnce) the one
// chunk that a lane has, turned once. What is not held is a loop of its own and computed twice
// (kTurnedTwice). The three are kernels of their own: in one, the loops' registers were spilled in
// all (45.1 us below, 43.7 without a rotation). Measured, 122,880 bf16 rows of 576 with 64 rotary
// dims: 213 MB in 36.9 us (5.8 TB/s, 0.90 of the copy rate; halves 45.6), 34.7 us without a
// rotation, 80 us with 128 rotary dims; 61,440 fp32 rows (one CTA an SM) in 38.8 us. Turned in fp32
// the last two took 68 and 34.3: 64 bits cost most where they are computed twice, or where no
// other CTA's loads run under them. A CTA that goes on to another block, loading it as it stores
// this one's chunks, spills; the next block prefetched to L2: the same time.
enum HowTurned { kNotTurned, kTurnedOnce, kTurnedTwice };
template <class T, bool HELD, HowTurned TURNED>
__global__ void __launch_bounds__(kE4M3Threads, sizeof(T) == 2 ? 2 : 1)
cache_write_e4m3_kernel(const __grid_constant__ CacheRows p, const __grid_constant__ RopeTable tab,
                        uint8_t* __restrict__ cache) {
    __shared__ uint64_t step[kRopeMaxDims / 2];
    __shared__ uint32_t warp_top[kE4M3Threads / 32];
    const int tid = threadIdx.x, r = tid / 8, l = tid % 8;
    const int blk = p.row0 / kScaleBlock + blockIdx.x;
    const int i = (int)((long long)blk * kScaleBlock + r - p.row0);      // this lane's row of the written ones
    const bool in = i >= 0 && i < p.n;
    const int chunks = p.dims / 8;
    uint8_t* base = cache + (long long)blk * (kScaleBlock + 1) * p.dims;
    float* record = reinterpret_cast<float*>(base + kScaleBlock * p.dims);
    const int old = blockIdx.x == 0 ? p.row0 % kScaleBlock : 0;   // rows kept from before
    // HELD: the chunks of steps in `held` are in registers; rotated ones are [rot0, rot1), at most
    // one a lane where kTurnedOnce: it is turned while the others' loads are on their way.
    const int rot0 = TURNED ? tab.offset / 8 : 0, rot1 = TURNED ? rot0 + tab.dims / 8 : 0;
    constexpr bool one = HELD && TURNED == kTurnedOnce;
    const bool mine = one && in && l < rot1 - rot0;
    const int loop0 = HELD ? rot0 : 0, loop1 = HELD ? (TURNED == kTurnedTwice ? rot1 : rot0) : chunks;
    Eight<T> v[HELD ? kE4M3Held : 1], turn;
    uint32_t held = 0;
    if constexpr (HELD)
        if (in) {
            const T* row = static_cast<const T*>(p.x) + i * p.x_ld + 8 * l;
#pragma unroll
            for (int s = 0; s < kE4M3Held; ++s) {
                const int c = 8 * s + l;
                if (c < chunks && !(c >= rot0 && c < rot1)) {
                    held |= 1u << s;
                    v[s] = load_eight(row + 64 * s);
                }
            }
            if (one && mine) turn = load_eight(row + 8 * rot0);
        }
    const float old_scale = old ? *record : 0.f;
    load_steps(tab, p.rotate, step);

    float top = 0.f, turned_to[8];
    if (in) {
        // (without HELD every chunk goes this way)
        if constexpr (!HELD || TURNED == kTurnedTwice)
#pragma unroll 1
            for (int c = loop0 + l; c < loop1; c += 8) {
                float u[8];
                load_chunk<T>(p, tab, TurnOdd{step, p.rotate ? position_of(p, i) : 0, tab.m}, i, c, u);
                top = top_of(u, top);
            }
        if constexpr (HELD) {
            using Two = typename Packed<T>::type;
            Two two;
            memset(&two, 0, sizeof(two));
#pragma unroll
            for (int s = 0; s < kE4M3Held; ++s)
                if (held >> s & 1u) two = top_packed<T>(v[s], two);
            const float t = top_value(two);
            if (t <= 3.402823466e38f) {
                top = fmaxf(top, t);
            } else {                                      // an infinity: the finite ones
#pragma unroll
                for (int s = 0; s < kE4M3Held; ++s)
                    if (held >> s & 1u) top = top_of<T>(v[s], top);
            }
        }
    }
    if constexpr (one)
        if (mine) {
            turn_eight<T>(p, tab, TurnOdd{step, position_of(p, i), tab.m}, i, rot0 + l, turn, turned_to);
            top = top_of(turned_to, top);
        }
    // (a float that is not negative orders as its bits do)
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if (tid % 32 == 0) warp_top[tid / 32] = most;
    __syncthreads();
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, warp_top[tid % (kE4M3Threads / 32)]));
    int e = scale_exponent(top);
    if (old) {
        const int was = (int)(__float_as_uint(old_scale) >> 23) - 127;
        if (was >= e) {
            e = min(was, kScaleExpMax);                   // (a record this library wrote)
        } else if (r < old) {
            // the earlier rows' codes, rounded again to the larger scale
            const float down = pow2f(max(was, -kScaleExpMax) - e);
#pragma unroll 1
            for (int c = l; c < chunks; c += 8) {
                uint32_t* at = reinterpret_cast<uint32_t*>(base + (long long)r * p.dims + 8 * c);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const float2 a = __half22float2(e4m3x2_half2(at[w] & 0xffffu));
                    const float2 b = __half22float2(e4m3x2_half2(at[w] >> 16));
                    at[w] = e4m3x4(a.x * down, a.y * down, b.x * down, b.y * down);
                }
            }
        }
    }
    for (int k = tid; k < p.dims / 4; k += kE4M3Threads)
        reinterpret_cast<uint32_t*>(record)[k] = k == 0 ? __float_as_uint(pow2f(e)) : 0u;
    if (!in) return;
    const uint32_t inv = __float_as_uint(pow2f(-e));
    const unsigned long long inv2 = (unsigned long long)inv << 32 | inv;
    uint8_t* to = base + (long long)r * p.dims + 8 * l;
    if constexpr (HELD)
#pragma unroll
        for (int s = 0; s < kE4M3Held; ++s)
            if (held >> s & 1u) *reinterpret_cast<uint2*>(to + 64 * s) = codes_of<T>(v[s], inv2);
    if constexpr (one)
        if (mine) *reinterpret_cast<uint2*>(to + 8 * rot0) = codes_of(turned_to, inv2);
    if constexpr (!HELD || TURNED == kTurnedTwice)
#pragma unroll 1
        for (int c = loop0 + l; c < loop1; c += 8) {
            float u[8];
            load_chunk<T>(p, tab, TurnOdd{step, p.rotate ? position_of(p, i) : 0, tab.m}, i, c, u);
            *reinterpret_cast<uint2*>(base + (long long)r * p.dims + 8 * c) = codes_of(u, inv2);
        }
}

// ---------------------------------------------------------------- reading back

struct CacheRead {
    const uint8_t* cache;
    const int32_t* rows;                        // NULL: row0 + i
    int row0, n, cache_rows;
    int dims, out_dims;                         // stored values of the part, values read
    int row_bytes, part_off;                    // formats 0-3: a stored row, where the part starts
    long long out_ld;                           // in values
    int fast;                                   // out's rows are 16-byte aligned
    int block_rows;                             // rows of a block
    SmallDiv by_row;                            // chunks of a row
};

// A stored chunk of eight values, and its scale.
template <int FMT>
struct Stored {
    uint4 w;                                    // fp16 values, or codes in x, y
    float scale;                                // 0: no row
};
template <int FMT>
__device__ __forceinline__ Stored<FMT> load_stored(const CacheRead& p, int row, int c) {
    Stored<FMT> s{make_uint4(0u, 0u, 0u, 0u), 0.f};
    if (row < 0 || row >= p.cache_rows) return s;
    if constexpr (FMT == kFmtF16) {
        s.w = __ldg(reinterpret_cast<const uint4*>(p.cache + (long long)row * p.row_bytes + 16 * c));
        s.scale = 1.f;
    } else {
        const uint8_t* codes;
        if constexpr (FMT == kFmtE4M3) {
            codes = p.cache + e4m3_place(row) * p.dims + 8 * c;
            const long long rec = (long long)(row / kScaleBlock) * (kScaleBlock + 1) + kScaleBlock;
            s.scale = __ldg(reinterpret_cast<const float*>(p.cache + rec * p.dims));
        } else {
            const uint8_t* part = p.cache + (long long)row * p.row_bytes + p.part_off;
            s.scale = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(
                part + quant_code_bytes(FMT, p.dims) + 2 * (c / 4)))));
            codes = part + (FMT == kFmtQ8 ? 8 * c : 16 * (c / 4) + 8 * (c % 2));
        }
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes));
        s.w.x = w.x;
        s.w.y = w.y;
    }
    return s;
}
template <int FMT>
__device__ __forceinline__ void values_of(const Stored<FMT>& s, int c, float (&v)[8]) {
    const uint32_t u[4] = {s.w.x, s.w.y, s.w.z, s.w.w};
    if constexpr (FMT == kFmtF16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    } else if constexpr (FMT == kFmtE4M3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(e4m3x2_half2(u[k / 2] >> (16 * (k % 2)) & 0xffffu));
            v[2 * k] = f.x * s.scale;
            v[2 * k + 1] = f.y * s.scale;
        }
    } else if constexpr (FMT == kFmtQ8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = s.scale * (float)(int8_t)(u[k / 4] >> (8 * (k % 4)) & 0xffu);
    } else {
        const int shift = c % 4 < 2 ? 0 : 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = s.scale * (float)((int)(u[k / 4] >> (8 * (k % 4) + shift) & 0xfu) - 8);
    }
}

// A block reads block_rows rows, a thread eight values at a time, four chunks in flight:
// value = code * scale in fp32, rounded once to T. An index outside the cache reads as a row
// of zeros.
template <class T, int FMT>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheRead p, T* __restrict__ out) {
    constexpr int U = 4;
    const int chunks = (int)p.by_row.d;
    const int first = blockIdx.x * p.block_rows;
    const int total = min(p.block_rows, p.n - first) * chunks;
#pragma unroll 1
    for (int base = threadIdx.x; base < total; base += U * 256) {
        Stored<FMT> s[U];
        int at[U], ch[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = base + u * 256;
            if (k >= total) break;
            const int i = (int)p.by_row.div(k);
            ch[u] = k - i * chunks;
            at[u] = first + i;
            s[u] = load_stored<FMT>(p, p.rows ? __ldg(p.rows + at[u]) : p.row0 + at[u], ch[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * 256 >= total) break;
            float v[8];
            values_of<FMT>(s[u], ch[u], v);
            T* dst = out + at[u] * p.out_ld + 8 * ch[u];
            Eight<T> o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o.e[k] = from_f32<T>(v[k]);
            if (p.fast) {
#pragma unroll
                for (int w = 0; w < (int)sizeof(T) / 2; ++w) reinterpret_cast<uint4*>(dst)[w] = o.q[w];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = o.e[k];
            }
        }
    }
}

}  // namespace ds4sp
