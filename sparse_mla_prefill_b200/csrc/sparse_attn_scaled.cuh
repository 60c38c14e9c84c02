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
//   w   = b0 + b1 / 16 + ... + b_{NT-1} / 16^(NT-1)
//   O^T = codes^T . [b0 .. b_{NT-1}]         M = 128 value dims x 4, N = NT x 16, K = rows
//   out = O / sum(w / s_r)
//
// NT = 5 carries w to 2^-20 (pv_mode 1: the result is right to fp32 sums), NT = 3 to 2^-12
// (pv_mode 0: as fp16 probabilities). Each rounding to e4m3 is of what the terms before it
// left, so the terms' sum is w but for the last one's rounding, and products of e4m3 values
// are exact in the fp32 accumulator.
//
// What bounds it: each unit's rows pass through the tensor cores twice, from shared memory.
// An M = 128, K = 32 instruction takes about 50 cycles whatever N up to 80 (measured: its
// 4 KB of A), so 128 rows take 18 + 16 of them, about 1,750 cycles. N costs nothing, which
// is why the terms are columns.
//
// A slab of rows (128 rows x 128 bytes, the 128-byte swizzle) is the K-major A of S and, as
// it lies, the MN-major A of O^T. Slabs form a ring of nine: O^T frees them one by one (its
// tile m reads slab m only), and the gather of a later unit follows on its heels.
//
// Roles: warps 0-3 softmax (a row per thread), 4-7 the queries' terms and the output, 8-11
// gather (16-byte cp.async), warp 12 issues the MMAs: S of unit g + 1 before O^T of unit g,
// so that the softmax of a unit has a whole unit's tensor time to finish.
// The reference ref_h is the first unit's maximum and is raised (O and the sums rescaled)
// only when a unit exceeds it by 2^8: e4m3 holds weights up to 448.
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
constexpr int SLOTS = 9;                        // slab ring
constexpr int ROPES = 3;                        // ring of the rows' last 64 dims
constexpr int SLAB = M * 128, ROPE = M * 64;
constexpr int QROWS = QT * H;
constexpr int QSLAB = QROWS * 128, QBYTES = TILES * QSLAB + QROWS * 64;
constexpr int SWARPS = 4, EWARPS = 4, PWARPS = 4;
constexpr int EWARP0 = SWARPS, PWARP0 = EWARP0 + EWARPS, MWARP = PWARP0 + PWARPS;
constexpr int THREADS = (MWARP + 1) * 32;
constexpr int SOFTMAX_BAR = 1;
constexpr float HEADROOM = 8.f;                 // log2 units a unit may exceed the reference

constexpr int OFF_SLAB = 0;
constexpr int OFF_ROPE = OFF_SLAB + SLOTS * SLAB;
constexpr int OFF_Q = OFF_ROPE + ROPES * ROPE;
constexpr int OFF_P = OFF_Q + QBYTES;                        // two buffers of NT x 128 rows x 16 bytes
constexpr int OFF_SCALE = OFF_P + 2 * 5 * M * H;             // rows' scales, one array per rope slot
constexpr int OFF_QS = OFF_SCALE + ROPES * M * 4;            // heads' logit factors, four tokens
constexpr int OFF_RED = OFF_QS + 4 * H * 4;                  // per softmax warp: maxima
constexpr int OFF_SUM = OFF_RED + SWARPS * H * 4;            // per softmax warp: sums, two tokens
constexpr int OFF_REF = OFF_SUM + 2 * SWARPS * H * 4;        // references, two tokens
constexpr int OFF_BAR = OFF_REF + 2 * H * 4;
// barriers
constexpr int B_SLAB_FULL = 0, B_SLAB_EMPTY = B_SLAB_FULL + SLOTS, B_ROPE_FULL = B_SLAB_EMPTY + SLOTS,
              B_ROPE_EMPTY = B_ROPE_FULL + ROPES, B_Q_FULL = B_ROPE_EMPTY + ROPES, B_Q_EMPTY = B_Q_FULL + 1,
              B_S_FULL = B_Q_EMPTY + 1, B_S_EMPTY = B_S_FULL + 2, B_P_FULL = B_S_EMPTY + 2,
              B_P_EMPTY = B_P_FULL + 2, B_O_FULL = B_P_EMPTY + 2, B_O_EMPTY = B_O_FULL + 1,
              B_L_FULL = B_O_EMPTY + 1, B_L_EMPTY = B_L_FULL + 2, B_DONE = B_L_EMPTY + 2, N_BARS = B_DONE + 1;
constexpr int OFF_TMEM = OFF_BAR + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;             // + alignment slack
static_assert(OFF_ROPE % 1024 == 0 && OFF_Q % 1024 == 0 && QSLAB % 1024 == 0 && OFF_P % 128 == 0 && OFF_BAR % 8 == 0,
              "swizzle atoms and barriers aligned");
static_assert(SMEM_BYTES <= attn::SMEM_LIMIT, "shared memory budget");

// TMEM columns: two S accumulators, then the four tiles of O^T.
constexpr int TM_S = 0, TM_O = 2 * QROWS;
template <int NT> constexpr int o_cols() { return NT * H; }
static_assert(TM_O + TILES * o_cols<5>() <= 512, "TMEM columns");

// Shared-memory descriptors (start address added): K-major rows of 128 bytes (8-row groups
// 1024 bytes apart, 128-byte swizzle) or of 64 bytes (512 apart, 64-byte swizzle); the same
// 128-byte atoms read with the dims as M (8-row groups are then steps along K); and P, with
// no swizzle: 16 heads x 8 rows of 128 bytes, row groups 128 bytes apart along K, terms
// 2048 bytes apart along N.
__host__ __device__ constexpr uint64_t desc_bits(uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | (uint64_t)swizzle << 61;
}
constexpr uint64_t DESC_128 = desc_bits(16, 1024, 2), DESC_64 = desc_bits(16, 512, 4),
                   DESC_P = desc_bits(128, M * H, 0);
__device__ __forceinline__ uint64_t desc_at(uint64_t bits, uint32_t addr) { return bits | (addr >> 4); }

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D; tr: both operands MN-major.
__host__ __device__ constexpr uint32_t idesc(int n, bool tr) {
    return 1u << 4 | (tr ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// Shared-memory writes of this thread (or writes it has acquired) before later tcgen05 reads.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Ties registers written by an earlier tcgen05.ld to a point after tmem_ld_wait().
__device__ __forceinline__ void regs_after_wait(uint32_t (&r)[16]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

__device__ __forceinline__ float warp_max(float v) {         // NaNs are ignored
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// This CTA's units in order: item idx, the u-th of its nu units of rows. In split mode an
// item is one unit of 32 rows (token_rows).
struct Cursor {
    int m, idx, u, nu;
    TokenRows tr;
    bool valid;
    __device__ __forceinline__ void take(const AttnParams& p) {
        valid = idx < p.n_items;
        u = 0;
        if (!valid) return;
        tr = token_rows(p, idx);
        nu = p.split ? 1 : (tr.nrows + M - 1) / M;
    }
    __device__ __forceinline__ void start(const AttnParams& p) {
        m = 0;
        idx = blockIdx.x;
        take(p);
    }
    __device__ __forceinline__ void next_item(const AttnParams& p) {
        ++m;
        idx += gridDim.x;
        take(p);
    }
    __device__ __forceinline__ void advance(const AttnParams& p) {
        if (++u == nu) next_item(p);
    }
    __device__ __forceinline__ int first_row(const AttnParams& p) const { return p.split ? SPLIT_ROWS * tr.u0 : M * u; }
    __device__ __forceinline__ int rows(const AttnParams& p) const {      // of this unit
        return min(p.split ? SPLIT_ROWS : M, tr.nrows - first_row(p));
    }
};

}  // namespace scaled

template <int NT>
__global__ void __launch_bounds__(scaled::THREADS, 1) sparse_attn_scaled_kernel(const __grid_constant__ AttnParams p) {
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
            mbar_init(bar(B_ROPE_EMPTY + s), 1 + SWARPS);    // S, and the scales' readers
        }
        mbar_init(bar(B_Q_FULL), EWARPS);
        mbar_init(bar(B_Q_EMPTY), 1);
        mbar_init(bar(B_O_FULL), 1);
        mbar_init(bar(B_O_EMPTY), EWARPS);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S_FULL + i), 1);
            mbar_init(bar(B_S_EMPTY + i), SWARPS);
            mbar_init(bar(B_P_FULL + i), SWARPS);
            mbar_init(bar(B_P_EMPTY + i), 1);
            mbar_init(bar(B_L_FULL + i), SWARPS);
            mbar_init(bar(B_L_EMPTY + i), EWARPS);
        }
        mbar_init(bar(B_DONE), 1);
        fence_mbar_init();
    }
    if (warp == MWARP) {
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
    auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, p.wc, abort); };
    Cursor c;
    c.start(p);

    if (warp >= PWARP0 && warp < MWARP) {
        // ================================================================ gather
        const int pw = warp - PWARP0, r = 32 * pw + lane;    // this thread resolves row r
        // Place of the unit's row r: 2 * place + 1 (compressed) or 2 * place; -1: none. The
        // top-k entry of a unit is fetched a unit ahead.
        auto entry = [&](const Cursor& cu) {
            const int gr = cu.first_row(p) + r;
            return cu.valid && gr < cu.tr.nsel && r < cu.rows(p) ? __ldg(p.topk + (size_t)cu.tr.i * p.k + gr) : -1;
        };
        auto resolve = [&](const Cursor& cu, int j) {
            const int gr = cu.first_row(p) + r;
            if (r >= cu.rows(p)) return -1;
            if (gr >= cu.tr.nsel) {
                const int row = cu.tr.s_lo + gr - cu.tr.nsel;
                return 2 * (int)e4m3_place(row);
            }
            const bool in = j >= 0 && j < (p.vis_mask ? p.mask_cols : cu.tr.nv);
            if (!in && !(p.vis_mask && j == -1)) record_status(p.wc.status, kStatusBounds);
            if (!in || (p.vis_mask && p.vis_mask[(size_t)cu.tr.t * p.mask_ld + j] == 0)) return -1;
            return 2 * (int)e4m3_place(j) + 1;
        };
        const uint8_t* raw = reinterpret_cast<const uint8_t*>(p.kv_raw);
        const uint8_t* cmp = reinterpret_cast<const uint8_t*>(p.kv_cmp);
        int slot = 0, rope = 0;
        uint32_t slab_phase = 1, rope_phase = 1;
        int j = entry(c);
        while (c.valid) {
            const int place = resolve(c, j);
            const bool copied = 32 * pw < c.rows(p);         // O^T reads whole groups of 32 rows
            Cursor nx = c;
            nx.advance(p);
            j = entry(nx);
            c = nx;
#pragma unroll 1
            for (int s = 0; s < TILES; ++s) {
                if (!__all_sync(0xffffffffu, wait(B_SLAB_EMPTY + slot, slab_phase))) {
                    abort = true;                            // the whole warp gives up together
                    break;
                }
                if (copied) {
                    const uint32_t dst = base + OFF_SLAB + slot * SLAB + 32 * pw * 128;
#pragma unroll
                    for (int it = 0; it < 8; ++it) {         // four rows of 128 bytes
                        const int rl = 4 * it + (lane >> 3), ch = lane & 7;
                        const int pl = __shfl_sync(0xffffffffu, place, rl);
                        const uint8_t* src = (pl & 1 ? cmp : raw) + (size_t)(max(pl, 0) >> 1) * DQK + s * 128 + ch * 16;
                        cp_async_16(dst + rl * 128 + ((ch ^ (rl & 7)) << 4), pl < 0 ? raw : src, pl >= 0);
                    }
                }
                cp_async_arrive_noinc(bar(B_SLAB_FULL + slot));
                if (++slot == SLOTS) {
                    slot = 0;
                    slab_phase ^= 1;
                }
            }
            if (abort || !__all_sync(0xffffffffu, wait(B_ROPE_EMPTY + rope, rope_phase))) break;
            if (copied) {
                const uint32_t dst = base + OFF_ROPE + rope * ROPE + 32 * pw * 64;
#pragma unroll
                for (int it = 0; it < 4; ++it) {             // eight rows of 64 bytes
                    const int rl = 8 * it + (lane >> 2), ch = lane & 3;
                    const int pl = __shfl_sync(0xffffffffu, place, rl);
                    const uint8_t* src = (pl & 1 ? cmp : raw) + (size_t)(max(pl, 0) >> 1) * DQK + DV + ch * 16;
                    cp_async_16(dst + rl * 64 + ((ch ^ ((rl >> 1) & 3)) << 4), pl < 0 ? raw : src, pl >= 0);
                }
            }
            {
                // The row's scale, 0 for no row: place q of a block's row lies in block q / 65.
                const int q = max(place, 0) >> 1;
                const uint8_t* src = (place & 1 ? cmp : raw) + ((size_t)(q / (kScaleBlock + 1)) * (kScaleBlock + 1) + kScaleBlock) * DQK;
                const int n = place >= 0 ? 4 : 0;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(base + OFF_SCALE + (rope * M + r) * 4),
                             "l"(place >= 0 ? src : raw), "r"(n)
                             : "memory");
            }
            cp_async_arrive_noinc(bar(B_ROPE_FULL + rope));
            if (++rope == ROPES) {
                rope = 0;
                rope_phase ^= 1;
            }
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
    } else if (warp == MWARP) {
        // ================================================================ MMA issuer
        if (lane == 0) {
            int slot = 0, rope = 0;
            uint32_t slab_phase = 0, rope_phase = 0;
            int pv_slot = 0, pv_rows = 0;
            bool pv_first = false, pv_last = false;
            int pv_m = 0;
            // O^T of unit g: its weights, the slabs from pv_slot on.
            auto issue_o = [&](int g) {
                if (!wait(B_P_FULL + (g & 1), (g >> 1) & 1)) return false;
                if (pv_first && !wait(B_O_EMPTY, (pv_m & 1) ^ 1)) return false;
                tc_fence_after();
                const uint64_t b0 = desc_at(DESC_P, base + OFF_P + (g & 1) * PBUF);
                const int steps = (pv_rows + 31) / 32;
#pragma unroll 1
                for (int t = 0; t < TILES; ++t) {
                    const uint64_t a0 = desc_at(DESC_128, base + OFF_SLAB + pv_slot * SLAB);
                    const uint32_t d = tmem + TM_O + t * OC;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps) umma_e4m3(d, a0 + k * (32 * 128 >> 4), b0 + k * (32 * H >> 4), idesc(OC, true), !pv_first || k > 0);
                    umma_commit(bar(B_SLAB_EMPTY + pv_slot));
                    if (++pv_slot == SLOTS) pv_slot = 0;
                }
                umma_commit(bar(B_P_EMPTY + (g & 1)));
                if (pv_last) umma_commit(bar(B_O_FULL));
                return true;
            };
            int g = 0;
            for (; c.valid; ++g) {
                if (c.u == 0 && !wait(B_Q_FULL, c.m & 1)) break;
                if (!wait(B_S_EMPTY + (g & 1), ((g >> 1) & 1) ^ 1)) break;
                tc_fence_after();
                const uint32_t d = tmem + TM_S + (g & 1) * QROWS;
                bool ok = true;
#pragma unroll 1
                for (int s = 0; s < TILES && ok; ++s) {
                    ok = wait(B_SLAB_FULL + slot, slab_phase);
                    if (!ok) break;
                    fence_async_proxy();
                    const uint64_t a0 = desc_at(DESC_128, base + OFF_SLAB + slot * SLAB);
                    const uint64_t b0 = desc_at(DESC_128, base + OFF_Q + s * QSLAB);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_e4m3(d, a0 + 2 * k, b0 + 2 * k, idesc(QROWS, false), s > 0 || k > 0);
                    if (++slot == SLOTS) {
                        slot = 0;
                        slab_phase ^= 1;
                    }
                }
                if (!ok || !wait(B_ROPE_FULL + rope, rope_phase)) break;
                fence_async_proxy();
                {
                    const uint64_t a0 = desc_at(DESC_64, base + OFF_ROPE + rope * ROPE);
                    const uint64_t b0 = desc_at(DESC_64, base + OFF_Q + TILES * QSLAB);
#pragma unroll
                    for (int k = 0; k < 2; ++k) umma_e4m3(d, a0 + 2 * k, b0 + 2 * k, idesc(QROWS, false), true);
                }
                umma_commit(bar(B_S_FULL + (g & 1)));
                umma_commit(bar(B_ROPE_EMPTY + rope));
                if (++rope == ROPES) {
                    rope = 0;
                    rope_phase ^= 1;
                }
                const bool last = c.u + 1 == c.nu;
                if (last) umma_commit(bar(B_Q_EMPTY));
                if (g > 0 && !issue_o(g - 1)) break;
                pv_rows = c.rows(p);
                pv_first = c.u == 0;
                pv_last = last;
                pv_m = c.m;
                c.advance(p);
            }
            if (!abort && g > 0) issue_o(g - 1);
            umma_commit(bar(B_DONE));
            mbar_wait_drain(bar(B_DONE), 0, p.wc);
        }
        __syncwarp();
    } else if (warp < SWARPS) {
        // ================================================================ softmax
        const int r = tid;                                   // this thread's row of each unit
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;  // the warp's TMEM lanes
        const float* scales = reinterpret_cast<const float*>(smem + OFF_SCALE);
        const float* qs = reinterpret_cast<const float*>(smem + OFF_QS);
        float* red = reinterpret_cast<float*>(smem + OFF_RED);
        float ref[H], sum[H], cq[H];
        int rope = 0;
        uint32_t rope_phase = 0;
        for (int g = 0; c.valid; ++g, c.advance(p)) {
            const bool first = c.u == 0;
            wait(B_ROPE_FULL + rope, rope_phase);
            wait(B_S_FULL + (g & 1), (g >> 1) & 1);
            __syncwarp();
            tc_fence_after();
            float acc[H];
            {
                uint32_t d0[16], d1[16], d2[16];
                const uint32_t at = tmem + lanes + TM_S + (g & 1) * QROWS;
                tmem_ld_x16(at, d0);
                tmem_ld_x16(at + 16, d1);
                tmem_ld_x16(at + 32, d2);
                tmem_ld_wait();
                regs_after_wait(d0);
                regs_after_wait(d1);
                regs_after_wait(d2);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    acc[h] = fmaf(fmaf(__uint_as_float(d2[h]), 0.0625f, __uint_as_float(d1[h])), 0.0625f, __uint_as_float(d0[h]));
            }
            const float sv = scales[rope * M + r];
            if (first) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    cq[h] = qs[(c.m & 3) * H + h];
                    ref[h] = 0.f;
                    sum[h] = 0.f;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(B_S_EMPTY + (g & 1)));
                mbar_arrive(bar(B_ROPE_EMPTY + rope));
            }
            if (++rope == ROPES) {
                rope = 0;
                rope_phase ^= 1;
            }
            const bool valid = sv > 0.f;
            const int sexp = (int)(__float_as_uint(sv) >> 23) - 127;
            const float lsv = (float)sexp;                   // log2 of the row's scale
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                acc[h] = fmaf(acc[h], cq[h] * sv, lsv);      // log2 of the row's weight
                top = fmaxf(top, acc[h] - ref[h]);
            }
            if (named_barrier_or(SOFTMAX_BAR, SWARPS * 32, first || abort || (valid && top > HEADROOM))) {
                // A new reference: the first unit's maximum, or one raised by this unit.
                if (named_barrier_or(SOFTMAX_BAR, SWARPS * 32, abort)) break;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float mx = warp_max(valid ? acc[h] : -INFINITY);
                    if (lane == 0) red[warp * H + h] = mx;
                }
                named_barrier(SOFTMAX_BAR, SWARPS * 32);
                float alpha[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float mu = fmaxf(fmaxf(red[h], red[H + h]), fmaxf(red[2 * H + h], red[3 * H + h]));
                    const float was = first ? (mu > -INFINITY ? mu : 0.f) : ref[h];
                    ref[h] = mu > was + HEADROOM ? mu : was;
                    alpha[h] = fast_exp2(was - ref[h]);
                    sum[h] *= alpha[h];
                }
                if (!first) {
                    // O^T of the units before has run; this one's waits for the weights below.
                    wait(B_P_EMPTY + ((g - 1) & 1), ((g - 1) >> 1) & 1);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int col = 0; col < TILES * OC; col += H) {
                        uint32_t o[16];
                        tmem_ld_x16(tmem + lanes + TM_O + col, o);
                        tmem_ld_wait();
                        regs_after_wait(o);
#pragma unroll
                        for (int h = 0; h < H; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * alpha[h]);
                        tmem_st_x16(tmem + lanes + TM_O + col, o);
                    }
                    tmem_st_wait();
                }
            }
            // Weights, their share of the sums, and their terms.
            const float inv = __uint_as_float((uint32_t)(127 - sexp) << 23);   // 1 / s_r
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float w = valid ? fast_exp2(acc[h] - ref[h]) : 0.f;
                acc[h] = w;
                sum[h] = fmaf(w, valid ? inv : 0.f, sum[h]);
            }
            wait(B_P_EMPTY + (g & 1), ((g >> 1) & 1) ^ 1);   // O^T of the unit before last
            __syncwarp();
            const uint32_t prow = base + OFF_P + (g & 1) * PBUF + r * H;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t w4[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    w4[q] = e4m3x4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
                    if (t + 1 < NT) {                        // what this term leaves, times 16
                        const float2 lo = __half22float2(e4m3x2_half2(w4[q] & 0xffffu));
                        const float2 hi = __half22float2(e4m3x2_half2(w4[q] >> 16));
                        acc[4 * q] = (acc[4 * q] - lo.x) * 16.f;
                        acc[4 * q + 1] = (acc[4 * q + 1] - lo.y) * 16.f;
                        acc[4 * q + 2] = (acc[4 * q + 2] - hi.x) * 16.f;
                        acc[4 * q + 3] = (acc[4 * q + 3] - hi.y) * 16.f;
                    }
                }
                st_shared_v4(prow + t * (M * H), make_uint4(w4[0], w4[1], w4[2], w4[3]));
            }
            fence_async_proxy();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P_FULL + (g & 1)));
            if (c.u + 1 == c.nu) {
                // The item's sums: 16 heads over 32 lanes, halving the heads a lane holds.
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
                // lane bits 4..1 chose heads' bits 3..0
                wait(B_L_EMPTY + (c.m & 1), ((c.m >> 1) & 1) ^ 1);
                __syncwarp();
                if ((lane & 1) == 0)
                    reinterpret_cast<float*>(smem + OFF_SUM)[((c.m & 1) * SWARPS + warp) * H + (lane >> 1)] = sum[0];
                if (tid == 0)
#pragma unroll
                    for (int h = 0; h < H; ++h) reinterpret_cast<float*>(smem + OFF_REF)[(c.m & 1) * H + h] = ref[h];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_L_FULL + (c.m & 1)));
            }
        }
    } else {
        // ================================================================ queries, output
        const int ew = warp - EWARP0, et = tid - EWARP0 * 32;
        const int qh = et / 8, ql = et % 8;                  // this thread's head, and its eighth
        const uint32_t lanes = (uint32_t)(32 * ew) << 16;
        uint4 qv[9];
        auto load_q = [&](const Cursor& cu) {
            const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)cu.tr.i * H + qh) * DQK);
#pragma unroll
            for (int k = 0; k < 9; ++k) qv[k] = __ldg(src + 8 * k + ql);
        };
        // The terms of item m's queries into shared memory, and the heads' logit factors.
        auto store_q = [&](int m) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 9; ++k) {
                const uint32_t u[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
                    if (fabsf(f.x) < INFINITY) top = fmaxf(top, fabsf(f.x));
                    if (fabsf(f.y) < INFINITY) top = fmaxf(top, fabsf(f.y));
                }
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const int e = scale_exponent(top);
            const float up = pow2f(-e);
            if (ql == 0) reinterpret_cast<float*>(smem + OFF_QS)[(m & 3) * H + qh] = pow2f(e) * p.scale_log2;
#pragma unroll
            for (int k = 0; k < 9; ++k) {
                const uint32_t u[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
                float v[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[x]));
                    v[2 * x] = fmaf(f.x * up, 0.f, f.x * up);        // an infinity becomes NaN
                    v[2 * x + 1] = fmaf(f.y * up, 0.f, f.y * up);
                }
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    uint32_t w[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        w[x] = e4m3x4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                        if (t + 1 < QT) {
                            const float2 lo = __half22float2(e4m3x2_half2(w[x] & 0xffffu));
                            const float2 hi = __half22float2(e4m3x2_half2(w[x] >> 16));
                            v[4 * x] = (v[4 * x] - lo.x) * 16.f;
                            v[4 * x + 1] = (v[4 * x + 1] - lo.y) * 16.f;
                            v[4 * x + 2] = (v[4 * x + 2] - hi.x) * 16.f;
                            v[4 * x + 3] = (v[4 * x + 3] - hi.y) * 16.f;
                        }
                    }
                    // dims 64k + 8ql ..: half a 16-byte chunk of row t * 16 + qh
                    const int row = t * H + qh, ch = 4 * (k & 1) + ql / 2;
                    uint8_t* at = k < 8 ? smem + OFF_Q + (k / 2) * QSLAB + row * 128 + ((ch ^ (row & 7)) << 4)
                                        : smem + OFF_Q + TILES * QSLAB + row * 64 + (((ql / 2) ^ ((row >> 1) & 3)) << 4);
                    *reinterpret_cast<uint2*>(at + 8 * (ql & 1)) = make_uint2(w[0], w[1]);
                }
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_Q_FULL));
        };
        if (c.valid) {
            load_q(c);
            store_q(0);
        }
        while (c.valid) {
            const Cursor it = c;
            c.next_item(p);
            if (c.valid) {
                load_q(c);
                if (!__all_sync(0xffffffffu, wait(B_Q_EMPTY, it.m & 1))) break;   // the last S has read it
                store_q(c.m);
            }
            const bool ok = wait(B_L_FULL + (it.m & 1), (it.m >> 1) & 1) && wait(B_O_FULL, it.m & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float* sums = reinterpret_cast<const float*>(smem + OFF_SUM) + (it.m & 1) * SWARPS * H;
            const int hl = lane & 15;
            const float L = (sums[hl] + sums[H + hl]) + (sums[2 * H + hl] + sums[3 * H + hl]);
            const float ref = reinterpret_cast<const float*>(smem + OFF_REF)[(it.m & 1) * H + hl];
            const float mul = p.split ? 1.f : L > 0.f || !(L == L) ? 1.f / L : 0.f;
            float* out = p.split ? p.part_o + (size_t)it.tr.item * H * DV : p.out + (size_t)it.tr.i * H * DV;
            if (p.split && ew == 0 && lane < H) {
                p.part_ml[(size_t)it.tr.item * 2 * H + hl] = ref;
                p.part_ml[(size_t)it.tr.item * 2 * H + H + hl] = L;
            }
#pragma unroll 1
            for (int t = 0; t < TILES; ++t) {
                uint32_t o[NT][16];
#pragma unroll
                for (int k = 0; k < NT; ++k) tmem_ld_x16(tmem + lanes + TM_O + t * OC + k * H, o[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < NT; ++k) regs_after_wait(o[k]);
                if (t + 1 == TILES) {                        // O^T and the sums are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(B_O_EMPTY));
                        mbar_arrive(bar(B_L_EMPTY + (it.m & 1)));
                    }
                }
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float v = __uint_as_float(o[NT - 1][h]);
#pragma unroll
                    for (int k = NT - 2; k >= 0; --k) v = fmaf(v, 0.0625f, __uint_as_float(o[k][h]));
                    out[h * DV + 128 * t + 32 * ew + lane] = v * __shfl_sync(0xffffffffu, mul, h);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MWARP) tmem_dealloc(tmem, 512);
}

}  // namespace ds4sp
