// Sparse MLA attention over a kv_format 5 cache (e4m3 codes, a scale for each block of 64
// rows), on the 5th-generation tensor cores with the codes as they are stored.
//
// The same rows and the same softmax as sparse_attn_mma_kernel: for token t one softmax of
// the 16 heads over the selected compressed rows, then the window's raw rows; key = 576
// values, value = the first 512. Row r's values are code * s_r, so with q split into sums of
// e4m3 terms both products run in e4m3 with fp32 accumulators, and no row is ever expanded:
//
//   q_h = 2^e_h (a0 + a1 / 16 + a2 / 256)    three terms hold an fp16 value's 11 bits
//                                            (2^e_h: the head's largest value at 448)
//   S   = codes . [a0 a1 a2]^T               M = 128 rows, N = 3 x 16, K = 576
//   w   = 2^(s_r 2^e_h scale log2(e) S + log2 s_r - ref_h)      the row's scale joins its
//                                            weight, since w * code = p * value
//   w   = b0 + b1 / 16 + b2 / 2^9 (+ b3 / 2^13 + b4 / 2^18)
//   O^T = codes^T . [b0 .. b_{NT-1}]         M = 128 value dims x 4, N = NT x 16, K = rows
//   out = O / sum(w / s_r)
//
// NT = 3 terms hold the weight's fp16 rounding (pv_mode 0), five the weight to 2^-20, and to
// 2^-28 of a weight of 1 where it is small (pv_mode 1: the result is as right as fp32 sums; four
// terms would leave small weights 2^-23, 3e-6 of the result). Each rounding to
// e4m3 is of what the terms before it left, so nothing is lost but the last one's remainder.
// Products of e4m3 values are exact in the fp32 accumulator.
//
// The last term's spacing is fixed, so a weight p s is held to no less than 2^-16 (three terms) or
// 2^-25 (five) of the token's largest: a row of a block of small scale beside one whose scale is
// 2^r times larger loses about r - 4 bits of its probability (measured, r = 10: 1e-3 or 7e-6 of
// sum p |v|; 2^-16 and 2^-25 are bounds, rows' errors have either sign). A unit that is its item's
// only one, as all are in the few-token form, keeps ten bits more.
//
// What bounds it: shared memory, and the instructions around it. Each unit's rows pass through
// the tensor cores twice, from shared memory: an M = 128, K = 32 instruction takes what its
// operands take at 128 bytes a cycle (measured: 45 cycles for S, 53 for O^T, mostly the 4 KB of
// A), so 128 rows take 18 + 16 of them, about 1,640 cycles, and N costs little, which is why the
// terms are columns. The gather and the roles' own accesses add about 800. Measured, 10,240
// tokens with 512 + 128 rows each, at 1.96 GHz: 575 us (pv_mode 1; each SM 3,500 cycles a unit;
// the softmax is busy for most of them, the tensor pipe for half, shared memory for 70%), 538 us
// (pv_mode 0), against 1,097 us of the fp16 cache's kernel with fp16 probabilities, 1,290 us with
// fp32-staged ones. In calls without a pause the card reaches its power limit within 0.2 s and the
// clock falls to 1.75 GHz: 560 us then becomes 635.
//
// What did not help: gathers by TMA (26 cycles for each 512 bytes), two groups of gather warps,
// more slabs, queries in warps of their own or double-buffered, a vote whose wait runs under the
// weights, sleeping or busier waits. The roles' loops compete for the instruction caches, so
// code size counts.
//
// A slab of rows (128 rows x 128 bytes, the 128-byte swizzle) is the K-major A of S and, as
// it lies, the MN-major A of O^T. There are slabs for two units: O^T frees them one by one (its
// tile m reads slab m only), and the gather of the unit after next follows on its heels (nine
// or ten slabs measured the same).
//
// Roles: warps 0-7 softmax, 8-11 the queries' terms and the output, 12-15 gather (16-byte
// cp.async), warp 16 issues S and warp 17 O^T: an MMA of this size is short
// against a wait's latency, and with two issuers each one's waits run under the other's MMAs.
// The reference ref_h is set above the maximum of the first unit that has rows (by 2^3), and
// raised, O and the sums rescaled, only when a unit exceeds it by 2^8, e4m3 holding weights up
// to 448: for logits of wide spread one unit in six, against three in ten with the maximum
// itself. (By 2^5, one in nine, a prefill took 562 us, but the largest weights were then 2^-5 and
// the result's error 7e-7; 2.8e-7 now, an elementary fp32 form's 3.5e-7.) The only unit of an item
// has its largest weight at 2^7: there is none to come that could exceed it.
// Every wait is bounded; a wait that gives up sets the launch's abort word and every role
// drains.
#pragma once

#include "device_common.cuh"
#include "kv_cache.cuh"
#include "sparse_attn_mma.cuh"

namespace ds4sp {
namespace scaled {

constexpr int H = attn::H, DQK = attn::DQK, DV = attn::DV;
constexpr int M = 128;                          // rows per unit
constexpr int SPLIT_ROWS = attn::BR;            // rows of a unit in split mode
constexpr int QT = 3;                           // terms of a query value
constexpr int TILES = DV / 128;                 // value tiles = slabs of 128 dims
constexpr int SLOTS = 2 * TILES;                // slabs: two units'
constexpr int ROPES = 2;                        // the rows' last 64 dims, two units
constexpr int SLAB = M * 128, ROPE = M * 64;
constexpr int QROWS = QT * H;
constexpr int QSLAB = QROWS * 128, QBYTES = TILES * QSLAB + QROWS * 64;
constexpr int SWARPS = 8, EWARPS = 4, PWARPS = 4;
constexpr int HG = H / 2;                       // heads of a softmax group of four warps
constexpr int EWARP0 = SWARPS, PWARP0 = EWARP0 + EWARPS, SMMA = PWARP0 + PWARPS, OMMA = SMMA + 1;
constexpr int THREADS = (OMMA + 1) * 32;
constexpr int SOFTMAX_BAR = 1;                  // and 2: one per group
constexpr int OUT_BAR = 3;
constexpr float UNSET = 1e30f;                  // minus the reference while no row was attended
constexpr float HEADROOM = 8.f;                 // log2 units a unit may exceed the reference, which is
constexpr float START = 3.f;                    // set so many above a unit's maximum,
constexpr float START_ALONE = -7.f;             // or below it, for an item's only rows (weights up to 2^7)

constexpr int OFF_SLAB = 0;
constexpr int OFF_ROPE = OFF_SLAB + SLOTS * SLAB;
constexpr int OFF_Q = OFF_ROPE + ROPES * ROPE;
constexpr int OFF_P = OFF_Q + QBYTES;                        // two buffers of NT x 128 rows x 16 bytes
constexpr int OFF_SCALE = OFF_P + 2 * 5 * M * H;             // rows' scales, one array per rope slot
constexpr int OFF_QS = OFF_SCALE + ROPES * M * 4;            // heads' logit factors, four tokens
constexpr int OFF_RED = OFF_QS + 4 * H * 4;                  // maxima per lane quarter, two units
constexpr int OFF_SUM = OFF_RED + 2 * 4 * H * 4;             // sums per lane quarter
constexpr int OFF_REF = OFF_SUM + 4 * H * 4;                 // references, two tokens
constexpr int OFF_BAR = OFF_REF + 2 * H * 4;
// barriers
constexpr int B_SLAB_FULL = 0, B_SLAB_EMPTY = B_SLAB_FULL + SLOTS, B_ROPE_FULL = B_SLAB_EMPTY + SLOTS,
              B_ROPE_EMPTY = B_ROPE_FULL + ROPES, B_Q_FULL = B_ROPE_EMPTY + ROPES, B_Q_EMPTY = B_Q_FULL + 1,
              B_S_FULL = B_Q_EMPTY + 1, B_S_EMPTY = B_S_FULL + 2, B_P_FULL = B_S_EMPTY + 2,
              B_P_EMPTY = B_P_FULL + 2, B_O_FULL = B_P_EMPTY + 2, B_O_EMPTY = B_O_FULL + 1,
              B_L_FULL = B_O_EMPTY + TILES, B_L_EMPTY = B_L_FULL + 2, B_DONE = B_L_EMPTY + 2, N_BARS = B_DONE + 1;
constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;             // + alignment slack
static_assert(OFF_ROPE % 1024 == 0 && OFF_Q % 1024 == 0 && QSLAB % 1024 == 0 && OFF_P % 128 == 0 && OFF_BAR % 8 == 0,
              "swizzle atoms and barriers aligned");
static_assert(SMEM_BYTES <= attn::SMEM_LIMIT, "shared memory budget");

// TMEM columns: two S accumulators, the four tiles of O^T, and each row's share of the heads'
// sums (two tokens).
constexpr int TM_S = 0, TM_O = 2 * QROWS, TM_SUM = 480;
template <int NT> constexpr int o_cols() { return NT * H; }
// The columns' order: term t of heads 8g .. 8g+7 (softmax group g) starts at o_col(g, t), so
// that a thread's terms are 16-byte chunks: pairs of terms, and an odd last one beside the
// other group's.
template <int NT>
__host__ __device__ constexpr int o_col(int g, int t) {
    return t < NT / 2 * 2 ? (g * (NT / 2) + t / 2) * H + t % 2 * HG : NT / 2 * 2 * H + g * HG;
}
// Term t of a weight counts 1 / (the product of its steps): what a term leaves, times the step.
// A term of up to 448 leaves up to 16, so 16 always fits; 32 does where the term is at most
// 256, as the second is (it is 16 times what the first left of at most 256).
__host__ __device__ constexpr float term_step(int t) { return t % 2 ? 32.f : 16.f; }
static_assert(TM_O + TILES * o_cols<5>() <= TM_SUM && TM_SUM + 2 * H <= 512, "TMEM columns");

// Shared-memory descriptors (start address added): K-major rows of 128 bytes (8-row groups
// 1024 bytes apart, 128-byte swizzle) or of 64 bytes (512 apart, 64-byte swizzle); the same
// 128-byte atoms read with the dims as M (8-row groups are then steps along K); and P, with
// no swizzle: 16 columns x 8 rows of 128 bytes, row groups 128 bytes apart along K, the next
// 16 columns 2048 bytes apart along N.
__host__ __device__ constexpr uint64_t desc_bits(uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | (uint64_t)swizzle << 61;
}
constexpr uint64_t DESC_128 = desc_bits(16, 1024, 2), DESC_64 = desc_bits(16, 512, 4),
                   DESC_P = desc_bits(128, M * H, 0);

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D; tr: both operands MN-major.
__host__ __device__ constexpr uint32_t idesc(int n, bool tr) {
    return 1u << 4 | (tr ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// n (1 .. 4) MMAs in a row whose operands' addresses step by A_STEP and B_STEP bytes, executed
// by a whole warp and issued by its elected lane (the same one every time). A_BITS, B_BITS: the
// descriptors' layouts (desc_bits); a, b: the operands' addresses. acc0: whether the first
// accumulates; the others do.
template <uint64_t A_BITS, uint64_t B_BITS, int A_STEP, int B_STEP>
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t id, uint32_t acc0, int n) {
    asm volatile(
        "{\n\t.reg .pred p, e, q, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "mov.b32 x, %1;\n\tmov.b32 y, %2;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %7};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.s32 x, x, %8;\n\tadd.s32 y, y, %9;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %7};\n\t"
        "setp.gt.and.s32 q, %5, 1, e;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.s32 x, x, %8;\n\tadd.s32 y, y, %9;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %7};\n\t"
        "setp.gt.and.s32 q, %5, 2, e;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.s32 x, x, %8;\n\tadd.s32 y, y, %9;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %7};\n\t"
        "setp.gt.and.s32 q, %5, 3, e;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem),
        "r"((uint32_t)A_BITS | a >> 4), "r"((uint32_t)B_BITS | b >> 4), "r"(id), "r"(acc0), "r"(n),
        "n"((uint32_t)(A_BITS >> 32)), "n"((uint32_t)(B_BITS >> 32)), "n"(A_STEP >> 4), "n"(B_STEP >> 4)
        : "memory");
}
// An arrival when all MMAs issued so far complete.
__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Shared-memory writes of this thread (or writes it has acquired) before later tcgen05 reads.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// This thread's TMEM lane, eight consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Ties registers written by an earlier tcgen05.ld to a point after tmem_ld_wait().
__device__ __forceinline__ void regs_after_wait(uint32_t (&r)[8]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
__device__ __forceinline__ float warp_max(float v) {         // NaNs are ignored
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// A work item: a token's rows, or in split mode (few tokens) 32 of them. Row r of the item
// is a selected compressed row for r < nsel, then window row s_lo + r - nsel.
constexpr int RATIO = 4;       // raw tokens per compressed row (the one ratio a handle takes)
struct Item {
    int i, t, nv;              // token of the call, absolute token, compressed rows it sees
    int nsel, s_lo;
    int row0, rows;            // the item's rows among the token's, [row0, row0 + rows)
    __device__ __forceinline__ void of_token(const AttnParams& p, int token) {
        i = token;
        t = p.t0 + token;
        nv = (t + 1) / RATIO;
        nsel = min(p.k, nv);
        s_lo = max(0, t - p.n_swa + 1);
        row0 = 0;
        rows = nsel + t - s_lo + 1;
    }
};

// Split mode: item idx is 32-row unit `unit` of token `token` (the units of token 0, then token
// 1, ...).
constexpr int MAX_SPLIT_ITEMS = 512;
struct SplitItems {
    uint8_t token[MAX_SPLIT_ITEMS], unit[MAX_SPLIT_ITEMS];
};
static_assert(attn::SPLIT_MAX_TOKENS <= 256 && attn::SPLIT_MAX_UNITS <= 256, "an item's token and unit are bytes");

// This CTA's units in order: rows [128 u, 128 u + rows()) of its m-th item.
struct Cursor {
    int m, idx, u;
    Item it;
    bool valid;
    __device__ __forceinline__ void take(const AttnParams& p, const SplitItems& items) {
        valid = idx < p.n_items;
        u = 0;
        if (!valid) return;
        if (!p.split) {
            it.of_token(p, p.n_q - 1 - idx);                 // heaviest (latest) first
            return;
        }
        it.of_token(p, items.token[idx]);
        it.row0 = SPLIT_ROWS * items.unit[idx];
        it.rows = min(SPLIT_ROWS, it.rows - it.row0);
    }
    __device__ __forceinline__ void start(const AttnParams& p, const SplitItems& items) {
        m = 0;
        idx = blockIdx.x;
        take(p, items);
    }
    __device__ __forceinline__ void next_item(const AttnParams& p, const SplitItems& items) {
        ++m;
        idx += gridDim.x;
        take(p, items);
    }
    __device__ __forceinline__ bool last() const { return M * (u + 1) >= it.rows; }
    __device__ __forceinline__ void advance(const AttnParams& p, const SplitItems& items) {
        if (last()) next_item(p, items);
        else ++u;
    }
    __device__ __forceinline__ int rows() const { return min(M, it.rows - M * u); }
};

// fp16 -> e4m3 codes of a pair, and what they leave, times `step` (exact: the difference of an
// fp16 value and its rounding to fewer bits is an fp16 value).
__device__ __forceinline__ uint32_t e4m3x2_of(__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 left_of(__half2 v, uint32_t codes, float step) {
    return __hmul2(__hsub2(v, e4m3x2_half2(codes)), __float2half2_rn(step));
}

// Two fp32 values in one operation.
struct F2 {
    unsigned long long b;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 of_f2(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v.b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}

}  // namespace scaled

template <int NT>
__global__ void __launch_bounds__(scaled::THREADS, 1)
sparse_attn_scaled_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ scaled::SplitItems items) {
    using namespace scaled;
    constexpr int OC = o_cols<NT>(), PBUF = NT * M * H;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_u32);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto bar = [&](int b) { return base + OFF_BAR + 8u * b; };
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);

    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(bar(B_SLAB_FULL + s), PWARPS * 32);    // the producers' copies
            mbar_init(bar(B_SLAB_EMPTY + s), 1);             // the O^T tile that read it
        }
        for (int s = 0; s < ROPES; ++s) {
            mbar_init(bar(B_ROPE_FULL + s), PWARPS * 32);
            mbar_init(bar(B_ROPE_EMPTY + s), SWARPS);        // the softmax: S has run, the scales are read
        }
        mbar_init(bar(B_Q_FULL), EWARPS);
        mbar_init(bar(B_Q_EMPTY), 1);
        mbar_init(bar(B_O_FULL), 1);
        for (int t = 0; t < TILES; ++t) mbar_init(bar(B_O_EMPTY + t), EWARPS);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S_FULL + i), 1);
            mbar_init(bar(B_S_EMPTY + i), SWARPS);
            mbar_init(bar(B_P_FULL + i), SWARPS);
            mbar_init(bar(B_P_EMPTY + i), 1);
            mbar_init(bar(B_L_FULL + i), SWARPS);
            mbar_init(bar(B_L_EMPTY + i), EWARPS);
        }
        mbar_init(bar(B_DONE), 2);
        fence_mbar_init();
    }
    if (warp == SMMA) {
        tmem_alloc(smem_u32(tmem_ptr), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    grid_dependency_wait();
    grid_dependents_launch();

    bool abort = false;
    auto wait = [&](int b, uint32_t parity) {
        if (!abort) abort = !mbar_wait_small(bar(b), parity, p.wc);
        return !abort;
    };
    Cursor c;
    c.start(p, items);

    if (warp >= PWARP0 && warp < SMMA) {
        // ================================================================ gather
        // A warp copies rows 16 i + 4 pw + (0 .. 3), so that a short unit's rows are spread over the
        // four; this thread resolves row r.
        const int pw = warp - PWARP0, r = 16 * (lane >> 2) + 4 * pw + (lane & 3);
        const uint8_t* raw = reinterpret_cast<const uint8_t*>(p.kv_raw);
        const uint8_t* cmp = reinterpret_cast<const uint8_t*>(p.kv_cmp);
        // The top-k entry of a unit's row r, fetched a unit ahead.
        auto entry = [&](const Cursor& cu) {
            const int gr = cu.it.row0 + M * cu.u + r;
            return cu.valid && r < cu.rows() && gr < cu.it.nsel ? __ldg(p.topk + (size_t)cu.it.i * p.k + gr) : -1;
        };
        // Where row r's values are, and its scale. A row that is not attended (behind the
        // last, or skipped) gets scale 0, so weight 0, and the token's own raw row as its
        // values: that row is attended too, so 0 times its values adds nothing, whatever
        // they are.
        auto resolve = [&](const Cursor& cu, int j, bool& ok) {
            const int gr = cu.it.row0 + M * cu.u + r;
            ok = r < cu.rows();
            int row = cu.it.t;
            if (ok && gr >= cu.it.nsel) row = cu.it.s_lo + gr - cu.it.nsel;
            if (!ok || gr >= cu.it.nsel) return raw + (size_t)e4m3_place(row) * DQK;
            ok = j >= 0 && j < (p.vis_mask ? p.mask_cols : cu.it.nv);
            if (!ok && !(p.vis_mask && j == -1)) record_status(p.wc.status, kStatusBounds);
            if (ok && p.vis_mask) ok = p.vis_mask[(size_t)cu.it.t * p.mask_ld + j] != 0;
            return ok ? cmp + (size_t)e4m3_place(j) * DQK : raw + (size_t)e4m3_place(row) * DQK;
        };
        // Four rows at a time: lane l takes chunk l % 8 of row l / 8 of the four, so an instruction
        // covers four whole 128-byte lines.
        const int ch = lane & 7, r4 = lane >> 3, r0 = 4 * pw + r4;
        const uint32_t to_slab = r0 * 128 + ((ch ^ (r0 & 7)) << 4);
        const uint32_t to_rope = r0 * 64 + ((ch ^ ((r0 >> 1) & 3)) << 4);
        int j = entry(c);
        for (int g = 0; c.valid; ++g) {
            const int b = g & 1;
            const uint32_t phase = ((g >> 1) & 1) ^ 1;
            bool ok;
            const uint8_t* mine = resolve(c, j, ok);
            const int sixteens = (c.rows() + 31) / 32 * 2;   // O^T reads whole groups of 32 rows
            const int place = c.it.row0 + M * c.u + r;
            const int row = place < c.it.nsel ? j : c.it.s_lo + place - c.it.nsel;
            const uint8_t* scale = (place < c.it.nsel ? cmp : raw) + ((size_t)(row / kScaleBlock) * (kScaleBlock + 1) + kScaleBlock) * DQK;
            const uint8_t* src[8];
#pragma unroll
            for (int it = 0; it < 8; ++it)
                src[it] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), 4 * it + r4)) + ch * 16;
            c.advance(p, items);
            j = entry(c);
#pragma unroll
            for (int s = 0; s < TILES; ++s) {
                if (!__all_sync(0xffffffffu, wait(B_SLAB_EMPTY + b * TILES + s, phase))) {
                    abort = true;                            // the whole warp gives up together
                    break;
                }
                const uint32_t dst = base + OFF_SLAB + (b * TILES + s) * SLAB + to_slab;
#pragma unroll
                for (int it = 0; it < 8; ++it)
                    if (it < sixteens) cp_async_16(dst + it * 2048, src[it] + s * 128, true);
                cp_async_arrive_noinc(bar(B_SLAB_FULL + b * TILES + s));
            }
            if (abort || !__all_sync(0xffffffffu, wait(B_ROPE_EMPTY + b, phase))) break;
            if (ch < 4) {
                const uint32_t dst = base + OFF_ROPE + b * ROPE + to_rope;
#pragma unroll
                for (int it = 0; it < 8; ++it)
                    if (it < sixteens) cp_async_16(dst + it * 1024, src[it] + DV, true);
            }
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(base + OFF_SCALE + (b * M + r) * 4),
                         "l"(ok ? scale : raw), "r"(ok ? 4 : 0)
                         : "memory");
            cp_async_arrive_noinc(bar(B_ROPE_FULL + b));
        }
        if (p.prefetch_bytes > 0 && !abort) {
            // This CTA's slice of the region the next kernel reads, in pieces of up to 32 KB.
            const long long per = (p.prefetch_bytes / gridDim.x + 15) / 16 * 16;
            const long long lo = per * blockIdx.x, hi = min(p.prefetch_bytes, lo + per);
            if (lane == 0)
                for (long long off = lo + (long long)pw * 32768; off < hi; off += PWARPS * 32768LL)
                    prefetch_l2(p.prefetch + off, (uint32_t)min(32768LL, hi - off));
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else if (warp >= SMMA) {
        // ================================================================ MMA issuers
        auto wait_w = [&](int b, uint32_t parity) {          // the whole warp gives up together
            abort = !__all_sync(0xffffffffu, wait(b, parity));
            return !abort;
        };
        if (warp == SMMA) {                                  // S of each unit
            for (int g = 0; c.valid && !abort; ++g, c.advance(p, items)) {
                const int b = g & 1;
                const uint32_t phase = (g >> 1) & 1;
                if (c.u == 0 && !wait_w(B_Q_FULL, c.m & 1)) break;
                if (!wait_w(B_S_EMPTY + b, phase ^ 1)) break;
                tc_fence_after();
                const uint32_t d = tmem + TM_S + b * QROWS;
#pragma unroll 1
                for (int s = 0; s < TILES; ++s) {
                    if (!wait_w(B_SLAB_FULL + b * TILES + s, phase)) break;
                    fence_async_proxy();
                    umma_e4m3<DESC_128, DESC_128, 32, 32>(d, base + OFF_SLAB + (b * TILES + s) * SLAB, base + OFF_Q + s * QSLAB,
                                                          idesc(QROWS, false), s, 4);
                }
                if (abort || !wait_w(B_ROPE_FULL + b, phase)) break;
                fence_async_proxy();
                umma_e4m3<DESC_64, DESC_64, 32, 32>(d, base + OFF_ROPE + b * ROPE, base + OFF_Q + TILES * QSLAB,
                                                    idesc(QROWS, false), 1, 2);
                commit_elected(bar(B_S_FULL + b));
                if (c.last()) commit_elected(bar(B_Q_EMPTY));
            }
        } else {                                             // O^T
            for (int g = 0; c.valid && !abort; ++g, c.advance(p, items)) {
                const int b = g & 1, steps = (c.rows() + 31) / 32;
                const bool first = c.u == 0;
                if (!wait_w(B_P_FULL + b, (g >> 1) & 1)) break;
                const uint32_t d = tmem + TM_O;
#pragma unroll 1
                for (int t = 0; t < TILES; ++t) {
                    // (a token's first unit overwrites tile by tile, behind the output's reads)
                    if (first && !wait_w(B_O_EMPTY + t, (c.m & 1) ^ 1)) break;
                    tc_fence_after();
                    umma_e4m3<DESC_128, DESC_P, 32 * 128, 32 * H>(d + t * OC, base + OFF_SLAB + (b * TILES + t) * SLAB,
                                                                  base + OFF_P + b * PBUF, idesc(OC, true), !first, steps);
                    commit_elected(bar(B_SLAB_EMPTY + b * TILES + t));
                }
                if (abort) break;
                commit_elected(bar(B_P_EMPTY + b));
                if (c.last()) commit_elected(bar(B_O_FULL));
            }
        }
        commit_elected(bar(B_DONE));
        if (lane == 0) mbar_wait_drain(bar(B_DONE), 0, p.wc);
        __syncwarp();
    } else if (warp < SWARPS) {
        // ================================================================ softmax
        // Two groups of four warps, eight heads each: a thread has one row of each unit.
        const int hg = warp / 4, qd = warp % 4, r = 32 * qd + lane;
        const uint32_t lanes = (uint32_t)(32 * qd) << 16;    // the warp's TMEM lanes
        const float* scales = reinterpret_cast<const float*>(smem + OFF_SCALE);
        const float* qs = reinterpret_cast<const float*>(smem + OFF_QS) + hg * HG;
        const int group_bar = SOFTMAX_BAR + hg;
        F2 nref[HG / 2], sum[HG / 2], cq[HG / 2];            // minus the references, sums, logit factors
        for (int g = 0; c.valid; ++g, c.advance(p, items)) {
            const bool first = c.u == 0;
            wait(B_P_EMPTY + (g & 1), ((g >> 1) & 1) ^ 1);   // O^T of the unit before last: its weights
            wait(B_S_FULL + (g & 1), (g >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            // (S was issued after its issuer saw the unit's rows, and scales, arrive.)
            const float sv = scales[(g & 1) * M + r];
            const bool valid = sv > 0.f;
            const int sexp = (int)(__float_as_uint(sv) >> 23) - 127;
            if (first) {
                const float4* q4 = reinterpret_cast<const float4*>(qs + (c.m & 3) * H);
#pragma unroll
                for (int q = 0; q < HG / 4; ++q) {
                    const float4 f = q4[q];
                    cq[2 * q] = f2(f.x, f.y);
                    cq[2 * q + 1] = f2(f.z, f.w);
                }
            }
            // No row of the item attended before this unit: the units before it, if there are
            // any, were all hidden and left sums and O of zero.
            const bool none = first || of_f2(nref[0]).x == UNSET;
            if (none)
#pragma unroll
                for (int q = 0; q < HG / 2; ++q) nref[q] = sum[q] = f2(0.f, 0.f);
            F2 x[HG / 2];                                    // log2 of the row's weights
            {
                uint32_t d0[8], d1[8], d2[8];
                const uint32_t at = tmem + lanes + TM_S + (g & 1) * QROWS + hg * HG;
                tmem_ld_x8(at, d0);
                tmem_ld_x8(at + H, d1);
                tmem_ld_x8(at + 2 * H, d2);
                tmem_ld_wait();
                regs_after_wait(d0);
                regs_after_wait(d1);
                regs_after_wait(d2);
                const F2 part = f2(0.0625f, 0.0625f), s2 = f2(sv, sv);
                const F2 lsv = f2((float)sexp, (float)sexp);     // log2 of the row's scale
                auto two = [](const uint32_t (&d)[8], int q) { return f2(__uint_as_float(d[2 * q]), __uint_as_float(d[2 * q + 1])); };
#pragma unroll
                for (int q = 0; q < HG / 2; ++q)
                    x[q] = fma2(fma2(fma2(two(d2, q), part, two(d1, q)), part, two(d0, q)), mul2(cq[q], s2), lsv);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(B_S_EMPTY + (g & 1)));
                mbar_arrive(bar(B_ROPE_EMPTY + (g & 1)));
            }
            float w[HG];                                     // x - ref, then the weights
            float top = -INFINITY;
            auto against_ref = [&] {
#pragma unroll
                for (int q = 0; q < HG / 2; ++q) {
                    const float2 d = of_f2(add2(x[q], nref[q]));
                    w[2 * q] = d.x;
                    w[2 * q + 1] = d.y;
                    top = fmaxf(top, fmaxf(d.x, d.y));
                }
            };
            against_ref();
            if (none || named_barrier_or(group_bar, 128, abort || (valid && top > HEADROOM))) {
                // A new reference: the first rows' maximum, or one raised by this unit.
                float* red = reinterpret_cast<float*>(smem + OFF_RED) + ((g & 1) * H + hg * HG) * 4;   // [head][quarter]
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float mx = warp_max(valid ? w[h] : -INFINITY);      // above the old reference
                    if (lane == 0) red[4 * h + qd] = mx;
                }
                if (named_barrier_or(group_bar, 128, abort)) break;
                float alpha[HG], most = -INFINITY;
                // (A single row keeps START: its reference, nearer 0 than the row's own negative
                // logarithm, is exact there, so its weight is 1/8 and the output the row's values.)
                const float start = none && c.last() && c.it.rows > 1 ? START_ALONE : START;
#pragma unroll
                for (int h = 0; h < HG; ++h) {
                    const float4 m4 = *reinterpret_cast<const float4*>(red + 4 * h);
                    const float mu = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
                    const float up = (none ? mu > -INFINITY : mu > HEADROOM) ? mu + start : 0.f;
                    most = fmaxf(most, mu);
                    alpha[h] = fast_exp2(-up);
                    w[h] = -up;
                }
#pragma unroll
                for (int q = 0; q < HG / 2; ++q) {
                    nref[q] = add2(nref[q], f2(w[2 * q], w[2 * q + 1]));
                    if (!none) sum[q] = mul2(sum[q], f2(alpha[2 * q], alpha[2 * q + 1]));
                }
                against_ref();
                if (!none) {
                    // O^T of the units before has run; this one's waits for the weights below.
                    wait(B_P_EMPTY + ((g - 1) & 1), ((g - 1) >> 1) & 1);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int t = 0; t < TILES; ++t) {
                        const uint32_t at = tmem + lanes + TM_O + t * OC;
                        uint32_t o[NT][8];
#pragma unroll
                        for (int k = 0; k < NT; ++k) tmem_ld_x8(at + o_col<NT>(hg, k), o[k]);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < NT; ++k) {
                            regs_after_wait(o[k]);
#pragma unroll
                            for (int h = 0; h < HG; ++h) o[k][h] = __float_as_uint(__uint_as_float(o[k][h]) * alpha[h]);
                            tmem_st_x8(at + o_col<NT>(hg, k), o[k]);
                        }
                    }
                    tmem_st_wait();
                }
                if (most == -INFINITY)                       // (the same in the whole group)
#pragma unroll
                    for (int q = 0; q < HG / 2; ++q) nref[q] = f2(UNSET, UNSET);
            }
            // Weights, their share of the sums, and their terms: w = hi + lo, two fp16 values;
            // two terms of hi, and NT - 2 of what they leave, lo joining it (NT = 5).
            const float inv = valid ? __uint_as_float((uint32_t)(127 - sexp) << 23) : 0.f;   // 1 / s_r
            uint32_t codes[NT][2];
#pragma unroll
            for (int q = 0; q < HG / 2; ++q) {
                const float wx = valid ? fast_exp2(w[2 * q]) : 0.f, wy = valid ? fast_exp2(w[2 * q + 1]) : 0.f;
                const F2 w2 = f2(wx, wy);
                sum[q] = fma2(w2, f2(inv, inv), sum[q]);
                __half2 v = __floats2half2_rn(wx, wy);
                F2 lo;
                if (NT == 5) {
                    const float2 hi = __half22float2(v);
                    constexpr float up = term_step(0) * term_step(1);
                    lo = fma2(f2(hi.x, hi.y), f2(-up, -up), mul2(w2, f2(up, up)));
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t == 2 && NT == 5) {
                        const float2 l2 = of_f2(lo);
                        v = __hadd2(v, __floats2half2_rn(l2.x, l2.y));
                    }
                    const uint32_t tc = e4m3x2_of(v);
                    if (t + 1 < NT) v = left_of(v, tc, term_step(t));
                    codes[t][q / 2] = q & 1 ? __byte_perm(codes[t][q / 2], tc, 0x5410) : tc;
                }
            }
            const uint32_t pbuf = OFF_P + (g & 1) * PBUF + r * H;
#pragma unroll
            for (int t = 0; t + 1 < NT; t += 2)
                st_shared_v4(base + pbuf + o_col<NT>(hg, t) / H * (M * H),
                             make_uint4(codes[t][0], codes[t][1], codes[t + 1][0], codes[t + 1][1]));
            if (NT % 2)
                *reinterpret_cast<uint2*>(smem + pbuf + o_col<NT>(hg, NT - 1) / H * (M * H) + hg * HG) =
                    make_uint2(codes[NT - 1][0], codes[NT - 1][1]);
            fence_async_proxy();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P_FULL + (g & 1)));
            if (c.last()) {
                // The row's share of the item's sums, for the output warps to add.
                wait(B_L_EMPTY + (c.m & 1), ((c.m >> 1) & 1) ^ 1);
                __syncwarp();
                uint32_t bits[8];
#pragma unroll
                for (int q = 0; q < HG / 2; ++q) {
                    const float2 f = of_f2(sum[q]);
                    bits[2 * q] = __float_as_uint(f.x);
                    bits[2 * q + 1] = __float_as_uint(f.y);
                }
                tmem_st_x8(tmem + lanes + TM_SUM + (c.m & 1) * H + hg * HG, bits);
                if (p.split && qd == 0 && lane == 0)
#pragma unroll
                    for (int q = 0; q < HG / 2; ++q) {
                        const float2 f = of_f2(nref[q]);
                        float* at = reinterpret_cast<float*>(smem + OFF_REF) + (c.m & 1) * H + hg * HG + 2 * q;
                        at[0] = -f.x;
                        at[1] = -f.y;
                    }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_L_FULL + (c.m & 1)));
            }
        }
    } else {
        // ================================================================ queries, output
        const int ew = warp - EWARP0, et = tid - EWARP0 * 32;
        const int qh = et / 8, ql = et % 8;                  // this thread's head, and its eighth
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        bool have = false;                                   // an item whose output is to come
        int om = 0, oi = 0, oidx = 0;                        // its number, its token, its index
        for (;;) {
            if (c.valid) {
                // The terms of the next item's queries into shared memory, once the last S of
                // the item before has read its own; and the heads' logit factors.
                const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)c.it.i * H + qh) * DQK);
                uint4 qv[9];
                __half2 top2 = __float2half2_rn(0.f);
#pragma unroll
                for (int k = 0; k < 9; ++k) qv[k] = __ldg(src + 8 * (k < 8 ? k ^ (qh & 1) : k) + ql);
                if (c.idx + (int)gridDim.x < p.n_items && !p.split) {
                    // The item after it: its queries, read once, come from memory.
                    const char* nx = reinterpret_cast<const char*>(p.q + (size_t)(c.it.i - (int)gridDim.x) * H * DQK);
                    for (int at = et * 128; at < H * DQK * 2; at += EWARPS * 32 * 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(nx + at));
                }
#pragma unroll
                for (int k = 0; k < 9; ++k) {
                    const uint32_t u[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __half2*>(&u[x])));
                }
                float top = fmaxf(__low2float(top2), __high2float(top2));
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                // (2^15 is fp16's largest power of two: it makes whole steps of the first term of
                // fp16's smallest values, so nothing is lost there. An infinity makes the head's
                // factor NaN.)
                const int e = max(scale_exponent(fminf(top, 65504.f)), -15);
                const __half2 up = __float2half2_rn(pow2f(-e));
                const float factor = top < INFINITY ? pow2f(e) * p.scale_log2 : NAN;
                uint32_t w[9][QT][2];
#pragma unroll
                for (int k = 0; k < 9; ++k) {
                    const uint32_t u[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&u[x]), up);
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            const uint32_t two = e4m3x2_of(v);
                            if (t + 1 < QT) v = left_of(v, two, 16.f);
                            w[k][t][x / 2] = x & 1 ? __byte_perm(w[k][t][x / 2], two, 0x5410) : two;
                        }
                    }
                }
                if (have) wait(B_Q_EMPTY, om & 1);           // (a wait that gave up: all stop below)
                __syncwarp();
                if (ql == 0) reinterpret_cast<float*>(smem + OFF_QS)[(c.m & 3) * H + qh] = factor;
                // dims 64k + 8ql ..: half a 16-byte chunk of row t * 16 + qh (whose swizzles are
                // qh's, t * 16 being whole atoms). Odd heads take k ^ 1, so that a warp's four
                // heads cover both halves of the banks.
                uint8_t* at[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    at[k] = smem + OFF_Q + qh * 128 + (((4 * (k ^ (qh & 1)) + ql / 2) ^ (qh & 7)) << 4) + 8 * (ql & 1);
                uint8_t* last = smem + OFF_Q + TILES * QSLAB + qh * 64 + (((ql / 2) ^ ((qh >> 1) & 3)) << 4) + 8 * (ql & 1);
#pragma unroll
                for (int t = 0; t < QT; ++t) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint2*>(at[k & 1] + (k / 2) * QSLAB + t * H * 128) = make_uint2(w[k][t][0], w[k][t][1]);
                    *reinterpret_cast<uint2*>(last + t * H * 64) = make_uint2(w[8][t][0], w[8][t][1]);
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q_FULL));
            }
            if (!have && !c.valid) break;
            const bool output = have;
            const int m = om, oi_ = oi, oidx_ = oidx;
            have = c.valid;
            om = c.m;
            oi = c.it.i;
            oidx = c.idx;
            if (c.valid) c.next_item(p, items);
            if (!output) continue;
            wait(B_L_FULL + (m & 1), (m >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            // The sums: 16 heads over the quarter's 32 rows, halving the heads a lane holds;
            // then the four quarters.
            float sum[H];
            {
                uint32_t bits[16];
                tmem_ld_x16(tmem + lanes + TM_SUM + (m & 1) * H, bits);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    asm volatile("" : "+r"(bits[h]));        // after the wait
                    sum[h] = __uint_as_float(bits[h]);
                }
            }
#pragma unroll
            for (int n = 8, off = 16; n >= 1; n >>= 1, off >>= 1) {
                const bool up = lane & off;
#pragma unroll
                for (int h = 0; h < n; ++h) {
                    const float give = up ? sum[h] : sum[h + n], keep = up ? sum[h + n] : sum[h];
                    sum[h] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            }
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 1);
            float* sums = reinterpret_cast<float*>(smem + OFF_SUM);
            if ((lane & 1) == 0) sums[ew * H + (lane >> 1)] = sum[0];   // lane bits 4..1 chose heads' bits 3..0
            wait(B_O_FULL, m & 1);
            if (named_barrier_or(OUT_BAR, EWARPS * 32, abort)) break;
            tc_fence_after();
            const int hl = lane & 15;
            const float L = (sums[hl] + sums[H + hl]) + (sums[2 * H + hl] + sums[3 * H + hl]);
            named_barrier(OUT_BAR, EWARPS * 32);             // read before the next item's are written
            const float ref = reinterpret_cast<const float*>(smem + OFF_REF)[(m & 1) * H + hl];
            const float mul = p.split ? 1.f : L > 0.f || !(L == L) ? 1.f / L : 0.f;
            float* out = p.split ? p.part_o + (size_t)oidx_ * H * DV : p.out + (size_t)oi_ * H * DV;
            if (p.split && ew == 0 && lane < H) {
                p.part_ml[(size_t)oidx_ * 2 * H + hl] = ref;
                p.part_ml[(size_t)oidx_ * 2 * H + H + hl] = L;
            }
            // A tile at a time, eight heads at a time.
            F2 by[H / 2];
#pragma unroll
            for (int h = 0; h < H; h += 2)
                by[h / 2] = f2(__shfl_sync(0xffffffffu, mul, h), __shfl_sync(0xffffffffu, mul, h + 1));
#pragma unroll 1
            for (int t = 0; t < TILES; ++t) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int h0 = half * HG;
                    uint32_t o[NT][8];
#pragma unroll
                    for (int k = 0; k < NT; ++k) tmem_ld_x8(tmem + lanes + TM_O + t * OC + o_col<NT>(half, k), o[k]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < NT; ++k) regs_after_wait(o[k]);
                    if (half == 1) {                             // the tile is read (and the sums)
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(B_O_EMPTY + t));
                            if (t + 1 == TILES) mbar_arrive(bar(B_L_EMPTY + (m & 1)));
                        }
                    }
                    float* to = out + h0 * DV + 128 * t + 32 * ew + lane;
#pragma unroll
                    for (int h = 0; h < HG; h += 2) {
                        auto two = [&](int k) { return f2(__uint_as_float(o[k][h]), __uint_as_float(o[k][h + 1])); };
                        F2 v = two(NT - 1);
#pragma unroll
                        for (int k = NT - 2; k >= 0; --k) v = fma2(v, f2(1.f / term_step(k), 1.f / term_step(k)), two(k));
                        const float2 f = of_f2(mul2(v, by[(h0 + h) / 2]));
                        to[h * DV] = f.x;
                        to[(h + 1) * DV] = f.y;
                    }
                }
            }
        }
    }

    if (abort) give_up(p.wc);
    linger_if(abort);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == SMMA) tmem_dealloc(tmem, 512);
}

}  // namespace ds4sp
