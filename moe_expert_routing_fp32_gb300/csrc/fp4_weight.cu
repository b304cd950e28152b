// fp4_weight.cu -- bf16 rows times 4-bit weights, for the few rows per expert
// of a decoding step.
//
//   STORE:   y[r, n] = x[r] . W[g, n]
//   SWIGLU:  act[r, n] = SiLU(x[r] . W[g, n]) (x[r] . W[g, I + n])
// for the rows r of group g, W[g, n, k] = e2m1 code * block scale.
//
// What bounds it is reading the weights, K (1/2 + 1/block) bytes a weight row,
// each used for a handful of rows.  A multiprocessor gets about 45 weights a
// cycle from memory: three instruction issues a weight for everything.  (mma.sync
// with the weights taken to f16 in registers needs 2.8 to 3.5 and ran at half the
// memory's rate: 22 us where the weights of 8 experts, K = N = 4096, take 10.5.)
// So the block-scaled tensor cores take the codes as they are, and the rows
// become 4-bit operands without loss:
//
// Digits.  With u = 2^(e - 1) for a block whose largest magnitude has the exponent
// e, x / u lies in (-4, 4) and is written to the base 8 in DIGITS digits of -4..4,
//   x = u sum_d digit_d 8^-d,
// all of them e2m1 values.  A row becomes DIGITS rows of codes under one scale
// per block, u relative to the row's largest; a product's columns of one row's
// digits are added up as sum_d 8^-d by the epilogue, which multiplies the row's
// own power of two on.  The digits hold 36 bits: magnitudes down to 2^-27 of their
// block's largest are exact, smaller ones off by at most 2^-35 of it.  (NV scales
// reach over 2^17 only: a block below 2^-17 of its row's largest counts as if it
// were there.)  Products and sums are those of the tensor cores, exact and fp32.
//
// Weights are the MMA's 128-row operand, two of them side by side (gate and up,
// or 256 columns of y); up to 8 rows are its 96 columns.  A stage holds 256
// columns of K.  The work is the list of (tile, stage) steps, cut into equal
// runs, one per CTA: a tile that two or more CTAs share is added up from its
// parts by the one that comes last (an atomic counter finds it; the parts are
// added in the order of K, so the result does not depend on who that is).
//
// A row with infinities or NaN has them left out of its digits and added by the
// epilogue, weight by weight: slow, but what the products give.
//
// 256 rows on 63 experts, K = 2048, N = 4096: 56 us (floor 44.6, 0.80 of the memory's
// rate; 86 with mma.sync).  One row on 8 experts, K = 4096, I = 2048: 20-21 us with the digits,
// 18 of them the product (floor 10.5; starting, the first loads and the joining of parts take
// the rest).  Four rows on one expert: 11.3-12.7.
//
// Beyond 8 rows a group a second tile reads the weights again, and the 96 digit columns a
// tile cost a third of bf16's rate at best: the FFN on 64 experts, H = 4096, I = 2048, MX,
// takes 142 us with one row each, 166 with 8, 272 with 16 and 526 with 32; on rows
// quantised first (csrc/fp4_gemm.cu) 147, 140, 142 and 147.
//
// Roles (8 warps): 0 TMA of the weights (which start before the rows' digits are
// ready), 3 TMA of the digits, 1 MMA, 2 setup, 4-7 epilogue.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "fp4_mma.cuh"
#include "internal.h"

namespace moe {

moe_status_t fp4_check(int format, int scale_exp);

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int THREADS = 256;
constexpr int TOK = 8;                       // rows of a tile
constexpr int DIGITS = 12;
constexpr int NB = TOK * DIGITS;             // 96 columns of an MMA
constexpr int BK = 256;                      // elements of K per stage: 128 bytes
constexpr int A_BYTES = 128 * BK / 2;        // of one of the two weight operands
constexpr int B_BYTES = NB * BK / 2;
constexpr int STAGES = 4;
constexpr int SF_COL = 4 * NB;               // two accumulators of two operands, then scales
constexpr int SF_SET = 24;                   // two scale tiles of each of three operands
constexpr int TMEM_COLS = 512;
constexpr int PART = TOK * 256;              // floats of a tile's partial sums

template <int FMT>
struct Cfg {
    static constexpr int TILES = BK / Fp4<FMT>::TILE_K;          // scale tiles per stage along K
    static constexpr int SF_BYTES = TILES * kScaleTile;
    static constexpr int W_LOAD = 2 * (A_BYTES + SF_BYTES), X_LOAD = B_BYTES + SF_BYTES;
    static constexpr int STAGE = W_LOAD + X_LOAD;
    static constexpr int BAR_OFF = STAGES * STAGE;
    static constexpr int NBARS = 2 * STAGES + 5;                 // full, empty, tfull, tempty, drain
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int OFFS_OFF = MISC_OFF + 16;
    static constexpr int smem(int G) { return 1024 + OFFS_OFF + (2 * G + 2) * 4; }
    // block scale of a row's largest block: 2^TOP; and how far below it others go
    static constexpr int TOP = FMT == MOE_FP4_MX ? 20 : 8, RANGE = FMT == MOE_FP4_MX ? 60 : 17;
    static_assert(STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");
    static_assert(smem(MAX_GROUPS) <= 227 * 1024, "shared memory");
    static_assert(SF_COL + 2 * SF_SET <= TMEM_COLS, "scale columns");
};
constexpr int MIN_E = 27;                    // biased exponent a row's largest counts as at least

// Workspace: digits [n * DIGITS, K / 2] bytes, their scale tiles, row factors
// (negative: the row holds infinities or NaN), counters of shared tiles, parts.
struct Ws {
    size_t q, sf, scale, counter, part, total;
};

struct Params {
    CUtensorMap tmA, tmSA;     // weights' codes [G, rows, K / 2] and scale tiles
    CUtensorMap tmB, tmSB;     // digits
    const uint16_t *x;
    const uint8_t *q, *sf;     // weights, for rows with infinities or NaN
    const float *row_scale;
    unsigned int *counter;     // [tiles]
    float *part;               // [2 * CTAs][TOK][256]
    const int32_t *offsets;
    int32_t G, n, K, N;        // N: output columns
    int32_t wrows;             // rows of a group's weights
    int32_t nt;                // column tiles
    float alpha;               // 2^scale_exp
    void *out;
    int32_t out_f32;
    int32_t *dev_status;
};

// ------------------------------------------------------------------ digits
constexpr int PREP_THREADS = 256;
struct PrepParams {
    const uint16_t *x;
    const int32_t *offsets;
    int32_t G, n, K;
    uint8_t *q, *sf;
    float *row_scale;
    unsigned int *counter;
    int32_t n_counter;
    int32_t parts;             // CTAs of a row
};

// A CTA takes 1024 columns of a row (and looks the whole row through for its
// largest value); two threads share 8 columns, one the upper six digits and one
// the lower.  Rounding to the sixth digit at once gives the same as digit after
// digit: what the first five take off is an even multiple of the sixth's unit.
constexpr int PREP_VECS = PREP_THREADS / 2;
template <int FMT>
__global__ void __launch_bounds__(PREP_THREADS) digits_kernel(const PrepParams p) {
    using C = Cfg<FMT>;
    constexpr int LANES = Fp4<FMT>::BLOCK / 8;         // lanes that share a block
    constexpr int HALF = DIGITS / 2;
    __shared__ int4 s_max[PREP_THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // from here on everything before this call has ended: the products may start
    // on the weights and the offsets, and wait for the digits
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.parts));
    const int part = static_cast<int>(blockIdx.x) - row * p.parts;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * PREP_THREADS + tid; i < p.n_counter;
         i += static_cast<int64_t>(gridDim.x) * PREP_THREADS)
        p.counter[i] = 0u;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.x + static_cast<int64_t>(row) * p.K);
    const int nv = p.K / 8;
    const int i = part * PREP_VECS + (tid & (PREP_VECS - 1)), half = tid / PREP_VECS;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (i < nv) v = __ldg(src + i);
    uint32_t m = 0;
    int bad = 0;
    for (int k = tid; k < nv; k += PREP_THREADS) {
        const uint4 q = __ldg(src + k);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = w[j] & 0x7FFFu, b = (w[j] >> 16) & 0x7FFFu;
            if (a < 0x7F80u) m = max(m, a); else bad = 1;
            if (b < 0x7F80u) m = max(m, b); else bad = 1;
        }
    }
    // the row's group is the last one that starts at or in front of it: how many do,
    // and the last of their starts
    int g = -1, at = -1, end = -1;
    for (int g0 = 0; g0 <= p.G; g0 += PREP_THREADS) {
        const int o = g0 + tid <= p.G ? __ldg(p.offsets + g0 + tid) : -1;
        const bool in = g0 + tid < p.G && o <= row;
        g += __syncthreads_count(in);
        if (in) at = max(at, o);
        end = max(end, o);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    bad = __any_sync(0xffffffffu, bad);
    at = __reduce_max_sync(0xffffffffu, at);
    end = __reduce_max_sync(0xffffffffu, end);
    if (lane == 0) s_max[warp] = make_int4(static_cast<int>(m), bad, at, end);
    __syncthreads();
    int start = -1;
#pragma unroll
    for (int k = 0; k < PREP_THREADS / 32; ++k) {
        const int4 w = s_max[k];
        m = max(m, static_cast<uint32_t>(w.x));
        bad |= w.y;
        start = max(start, w.z);
        end = max(end, w.w);
    }
    const int e_row = max(static_cast<int>(m >> 7), MIN_E);
    // 1 / u of a block is 2^(127 - e_row) 2^(1 - rel), both within fp32's exponents
    const float inv_row = pow2f(max(127 - e_row, -126));
    const int one = e_row == 254 ? 0 : 1;
    // u * 2^-TOP of the largest block
    if (tid == 0 && part == 0) {
        const float f = pow2f(e_row - 127 - 1 - C::TOP);
        p.row_scale[row] = bad ? -f : f;
    }
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {                      // infinities and NaN count as zero
        if ((w[j] & 0x7F80u) == 0x7F80u) w[j] &= 0xFFFF0000u;
        if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] &= 0xFFFFu;
    }
    uint32_t am = amax8(w);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    if (i >= nv) return;
    const int rel = max(static_cast<int>(am >> 7) - e_row, -C::RANGE);          // <= 0
    const float inv = pow2f(one - rel);
    float t[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {                      // x / u: two exact products
        t[2 * j] = __uint_as_float(w[j] << 16) * inv_row * inv;
        t[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * inv_row * inv;
    }
    if (half)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = t[j] * 32768.0f;           // 8^(HALF - 1)
            t[j] = (s - rintf(s)) * 8.0f;
        }
    uint8_t *dst = p.q + (static_cast<int64_t>(row) * DIGITS + half * HALF) * (p.K / 2) + i * 4;
#pragma unroll
    for (int d = 0; d < HALF; ++d) {
        float r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = rintf(t[j]);
            t[j] = (t[j] - r[j]) * 8.0f;
        }
        *reinterpret_cast<uint32_t *>(dst) = e2m1x8(r);
        dst += p.K / 2;
    }
    // (bad offsets are the product's to report; what is written stays in bounds)
    if (start < 0 || g >= p.G || row >= end) return;
    const int local = row - start;
    const int e = C::TOP + rel;
    const uint32_t byte = FMT == MOE_FP4_MX ? static_cast<uint32_t>(127 + e)
                          : e >= -6         ? static_cast<uint32_t>((e + 7) << 3)
                                            : 1u << (e + 9);
    const int b = i / LANES;                           // block: its lanes share the digits' rows
    uint8_t *sf = p.sf + ((static_cast<int64_t>(start / TOK) + g + local / TOK) *
                              (p.K / Fp4<FMT>::TILE_K) + (b >> 2)) * kScaleTile + (b & 3);
    const int digit_row = (local % TOK) * DIGITS + half * HALF;
    for (int d = lane % LANES; d < HALF; d += LANES)
        sf[scale_row_offset(digit_row + d)] = static_cast<uint8_t>(byte);
}

// ------------------------------------------------------------------ products
// The digits' columns at a and at b (one statement: nothing may touch the registers
// before the wait).
__device__ __forceinline__ void tmem_read12x2(uint32_t a, uint32_t b, uint32_t (&x)[DIGITS],
                                              uint32_t (&y)[DIGITS]) {
    static_assert(DIGITS == 12, "three loads of four columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%25];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%26];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%12, %13, %14, %15}, [%27];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%16, %17, %18, %19}, [%28];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%20, %21, %22, %23}, [%29];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(x[0]), "=&r"(x[1]), "=&r"(x[2]), "=&r"(x[3]),
          "=&r"(x[4]), "=&r"(x[5]), "=&r"(x[6]), "=&r"(x[7]),
          "=&r"(x[8]), "=&r"(x[9]), "=&r"(x[10]), "=&r"(x[11]),
          "=&r"(y[0]), "=&r"(y[1]), "=&r"(y[2]), "=&r"(y[3]),
          "=&r"(y[4]), "=&r"(y[5]), "=&r"(y[6]), "=&r"(y[7]),
          "=&r"(y[8]), "=&r"(y[9]), "=&r"(y[10]), "=&r"(y[11])
        : "r"(a), "r"(a + 4), "r"(a + 8), "r"(b), "r"(b + 4), "r"(b + 8)
        : "memory");
}
// sum_d 8^-d v_d
__device__ __forceinline__ float add_digits(const uint32_t (&v)[DIGITS]) {
    float s = __uint_as_float(v[DIGITS - 1]);
#pragma unroll
    for (int d = DIGITS - 2; d >= 0; --d) s = fmaf(s, 0.125f, __uint_as_float(v[d]));
    return s;
}

// Half a stage of NV (or all of MX): two scale tiles of each operand to one of
// two sets of columns in turn, then the MMAs that use them.
template <int FMT>
__device__ __forceinline__ void issue_tiles(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb,
                                            uint32_t sf_col, int steps, bool accumulate) {
    constexpr uint32_t ID0 = idesc<FMT>(128, NB, 0), ID2 = idesc<FMT>(128, NB, 2);
    constexpr uint32_t S1 = Cfg<FMT>::SF_BYTES / 16, A1 = A_BYTES / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        copy_scales<1>(sf_col + 4 * i, sa + i * (kScaleTile / 16));
        copy_scales<1>(sf_col + 8 + 4 * i, sa + S1 + i * (kScaleTile / 16));
        copy_scales<1>(sf_col + 16 + 4 * i, sb + i * (kScaleTile / 16));
    }
    constexpr int PER = FMT == MOE_FP4_MX ? 4 : 2;       // MMAs of 64 columns of K
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (j >= steps) break;
        const int i = FMT == MOE_FP4_MX ? j / 2 : j;
        const uint32_t id = FMT == MOE_FP4_MX && (j & 1) ? ID2 : ID0;
        const uint32_t acc = j > 0 || accumulate ? 1u : 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            mma_fp4<FMT, 1>(d + h * NB, a + h * A1 + j * 2, b + j * 2, id, sf_col + 8 * h + 4 * i,
                            sf_col + 16 + 4 * i, acc);
    }
}

struct Tile {
    int g, row0, cnt, n_blk;
};
// The (tile, stage) steps in equal runs, the first `extra` one step longer.
struct Runs {
    int base, extra;
    __device__ __forceinline__ Runs(int steps, int ctas) : base(steps / ctas), extra(steps - base * ctas) {}
    __device__ __forceinline__ int at(int i) const { return base * i + min(i, extra); }
    __device__ __forceinline__ int owner(int s) const {       // the run that holds step s
        const int longer = extra * (base + 1);
        return s < longer ? s / (base + 1) : extra + (s - longer) / base;
    }
};

// What a row's infinities and NaN add to its product with weight row `wr`.
template <int FMT>
__device__ __noinline__ float odd_terms(const Params &p, int row, int64_t wr) {
    const uint16_t *x = p.x + static_cast<int64_t>(row) * p.K;
    const uint8_t *q = p.q + wr * (p.K / 2);
    const uint8_t *sf = p.sf + wr / 128 * (p.K / Fp4<FMT>::TILE_K) * kScaleTile +
                        scale_row_offset(static_cast<int>(wr % 128));
    float s = 0.0f;
    for (int k = 0; k < p.K; ++k) {
        const uint16_t b = __ldg(x + k);
        if ((b & 0x7F80u) != 0x7F80u) continue;
        const uint32_t c = __ldg(q + k / 2) >> (4 * (k & 1)) & 15u;
        const int blk = k / Fp4<FMT>::BLOCK;
        const uint32_t sb = __ldg(sf + (blk >> 2) * kScaleTile + (blk & 3));
        const uint32_t e = c >> 1 & 3u, m = c & 1u;
        const float mag = e == 0 ? 0.5f * m : static_cast<float>(2u + m) * 0.25f * (1u << e);
        float scale;
        if (FMT == MOE_FP4_MX)
            scale = sb == 255u ? __uint_as_float(0x7FC00000u)
                               : (sb == 0 ? __uint_as_float(1u << 22) : pow2f(static_cast<int>(sb) - 127));
        else
            scale = (sb & 127u) == 127u ? __uint_as_float(0x7FC00000u) : e4m3_value(sb);
        s += bf16_bits_to_float(b) * ((c & 8u ? -mag : mag) * scale);
    }
    return s;
}

// Whether a wait succeeded in every thread of the epilogue's four warps, which share
// barrier 1: they go on or leave their loop together.  A warp that gave up alone would
// leave the others at a barrier that it never reaches.
__device__ __forceinline__ bool all_warps(bool ok) {
    uint32_t all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(ok ? 1u : 0u)
        : "memory");
    return all != 0;
}

template <int FMT, bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1) weight_kernel(const __grid_constant__ Params p) {
    using C = Cfg<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;       // [2]
    uint64_t *tempty = tfull + 2;           // [2]
    uint64_t *drain = tempty + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    volatile int *s_bad = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 8);
    volatile int *s_last = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 12);
    int *s_off = reinterpret_cast<int *>(smem + C::OFFS_OFF);
    int *s_prefix = s_off + p.G + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 1) {
        tmem_alloc(s_tmem, TMEM_COLS);
        tmem_relinquish();
    } else if (warp == 2 && elect_one()) {
        *s_abort = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);          // each producer arms its share
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    } else if (warp == 3 && elect_one()) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        tma_prefetch_desc(&p.tmSA);
        tma_prefetch_desc(&p.tmSB);
    }
    // tiles of the groups before each (the offsets are not the digits' kernel's)
    for (int g = tid; g <= p.G; g += THREADS) s_off[g] = __ldg(p.offsets + g);
    if (tid == 0) *s_bad = 0;
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        bool bad = false;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int tiles = 0;
            if (g < p.G) {
                const int a = s_off[g], b = s_off[g + 1];
                if (a < 0 || b < a || b > p.n) bad = true;
                tiles = b > a ? ((b - a + TOK - 1) / TOK) * p.nt : 0;
            }
            int inc = tiles;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += o;
            }
            if (g < p.G) s_prefix[g] = run + inc - tiles;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) s_prefix[p.G] = run;
        if (__any_sync(0xffffffffu, bad) && lane == 0) *s_bad = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // a kernel that follows may start to get ready (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (*s_bad && tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
    const int kst = (p.K + BK - 1) / BK;
    const int steps = *s_bad ? 0 : s_prefix[p.G] * kst;
    // two steps each at least, as far as they go
    const int ctas = max(1, min(static_cast<int>(gridDim.x), (steps + 1) / 2));
    const int me = static_cast<int>(blockIdx.x);
    const Runs runs(steps, ctas);
    const int run_at = me < ctas ? runs.at(me) : 0, run_end = me < ctas ? runs.at(me + 1) : 0;
    const uint32_t tmem = *s_tmem;
    const int64_t ktiles = p.K / Fp4<FMT>::TILE_K;

    auto decode = [&](int tile, int &g) {
        while (s_prefix[g + 1] <= tile) ++g;
        const int start = s_off[g], cnt = s_off[g + 1] - start;
        const int local = tile - s_prefix[g], chunks = (cnt + TOK - 1) / TOK;
        const int n_blk = local / chunks, c = local - n_blk * chunks;    // chunks side by side:
        return Tile{g, start + c * TOK, min(TOK, cnt - c * TOK), n_blk};  // they share weights
    };

    if (warp == 0 || warp == 3) {
        // ================= TMA producers: warp 0 the weights, warp 3 the digits
        if (elect_one()) {
            const bool weights = warp == 0;
            if (!weights) asm volatile("griddepcontrol.wait;" ::: "memory");
            int stage = 0, g = 0;
            uint32_t phase = 0;
            int armed[STAGES];
            for (int s = 0; s < STAGES; ++s) armed[s] = -1;
            bool ok = true;
            for (int u = run_at; u < run_end && ok && !*s_abort;) {
                const int tile = u / kst, k0 = u - tile * kst, k1 = min(kst, k0 + run_end - u);
                const Tile t = decode(tile, g);
                const int n0 = t.n_blk * (SWIGLU ? 128 : 256), n1 = SWIGLU ? p.N + n0 : n0 + 128;
                const int64_t blk = static_cast<int64_t>(t.g) * (p.wrows / 128);
                const int sa0 = static_cast<int>((blk + n0 / 128) * ktiles);
                const int sa1 = static_cast<int>((blk + n1 / 128) * ktiles);
                const int start = s_off[t.g];
                const int sb = static_cast<int>(
                    (static_cast<int64_t>(start / TOK) + t.g + (t.row0 - start) / TOK) * ktiles);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!wait_phase(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    armed[stage] = static_cast<int>(phase);
                    uint8_t *s = smem + stage * C::STAGE;
                    uint8_t *b = s + 2 * A_BYTES, *sf = b + B_BYTES;
                    const int c = kb * (BK / 2), kt = kb * C::TILES;
                    mbar_arrive_expect_tx(&full[stage], weights ? C::W_LOAD : C::X_LOAD);
                    if (weights) {
                        tma_load_3d(s, &p.tmA, &full[stage], c, n0, t.g);
                        tma_load_3d(s + A_BYTES, &p.tmA, &full[stage], c, n1, t.g);
                        tma_load_2d(sf, &p.tmSA, &full[stage], 0, sa0 + kt);
                        tma_load_2d(sf + C::SF_BYTES, &p.tmSA, &full[stage], 0, sa1 + kt);
                    } else {
                        tma_load_2d(b, &p.tmB, &full[stage], c, t.row0 * DIGITS);
                        tma_load_2d(sf + 2 * C::SF_BYTES, &p.tmSB, &full[stage], 0, sb + kt);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                u += k1 - k0;
            }
            if (*s_abort)
                for (int s = 0; s < STAGES; ++s)
                    if (armed[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(armed[s]));
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer
        if (elect_one()) {
            int stage = 0;
            uint32_t phase = 0, n = 0, set = 0;
            const uint32_t base = smem_u32(smem) >> 4;
            bool issued = false, ok = true;
            for (int u = run_at; u < run_end && ok && !*s_abort; ++n) {
                const int k0 = u % kst, k1 = min(kst, k0 + run_end - u);
                if (!wait_phase(&tempty[n & 1], ((n >> 1) & 1) ^ 1, s_abort, p.dev_status)) break;
                tc_fence_after();
                const uint32_t d = tmem + (n & 1) * (2 * NB);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!wait_phase(&full[stage], phase, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = base + static_cast<uint32_t>(stage) * (C::STAGE / 16);
                    const uint32_t a = at + OPERAND_LO, b = a + 2 * A_BYTES / 16;
                    const uint32_t sa = at + (2 * A_BYTES + B_BYTES) / 16 + SCALES_LO;
                    const uint32_t sb = sa + 2 * C::SF_BYTES / 16;
                    const int left = (p.K - kb * BK) / 64;       // MMA steps of this slice (2 or more)
                    constexpr int PER = FMT == MOE_FP4_MX ? 4 : 2;
#pragma unroll
                    for (int h = 0; h < 4 / PER; ++h) {
                        if (h * PER >= left) break;
                        issue_tiles<FMT>(d, a + h * PER * 2, b + h * PER * 2,
                                         sa + h * 2 * (kScaleTile / 16), sb + h * 2 * (kScaleTile / 16),
                                         tmem + SF_COL + set * SF_SET, left - h * PER, kb > k0 || h > 0);
                        set ^= 1;
                    }
                    issued = true;
                    tc_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit(&tfull[n & 1]);
                u += k1 - k0;
            }
            if (*s_abort && issued) {
                // unwinding: every MMA issued so far ends before TMEM is freed
                tc_commit(drain);
                mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ================= epilogue: thread = weight row `r` of both operands
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t n = 0;
        int g = 0;
        for (int u = run_at; u < run_end; ++n) {
            const int tile = u / kst, k0 = u - tile * kst, k1 = min(kst, k0 + run_end - u);
            u += k1 - k0;
            const Tile t = decode(tile, g);
            const uint32_t acc = tmem + lanes + (n & 1) * (2 * NB);
            const bool whole = k1 - k0 == kst;
            const int n0 = t.n_blk * (SWIGLU ? 128 : 256);
            const int64_t w0 = static_cast<int64_t>(t.g) * p.wrows + n0 + r;
            const bool second = SWIGLU || n0 + 128 < p.N;          // N = 128 mod 256: no such columns
            float scale[TOK];
#pragma unroll
            for (int j = 0; j < TOK; ++j) scale[j] = __ldg(p.row_scale + t.row0 + min(j, t.cnt - 1));
            // the CTAs of this tile, and where one of them leaves its part: a CTA has
            // parts of its first and of its last tile
            const int c0 = runs.owner(tile * kst), c1 = runs.owner(tile * kst + kst - 1);
            auto part_of = [&](int c) {
                return p.part + static_cast<int64_t>(2 * c + (c == c0 && runs.at(c) < tile * kst)) * PART + r;
            };
            // the parts of c .. c + 3, their loads all at once
            float w[4][2][TOK];
            auto load_parts = [&](int c) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float *q = part_of(min(c + k, c1));
#pragma unroll
                    for (int j = 0; j < TOK; ++j) {
                        if (j >= t.cnt) break;
                        w[k][0][j] = __ldcg(q + j * 256);
                        w[k][1][j] = __ldcg(q + j * 256 + 128);
                    }
                }
            };
            // A tile of few parts whose others are all there already (this CTA's is the
            // last, as a rule the first in K): they are fetched while its own MMAs run,
            // and its own part needs not be written.
            bool rest = false;
            if (!whole && c1 - c0 < 4) {
                if (tid == 128) {
                    unsigned int count;
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                                 : "=r"(count)
                                 : "l"(p.counter + tile)
                                 : "memory");
                    *s_last = count == static_cast<unsigned>(c1 - c0);
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                rest = *s_last != 0;
                asm volatile("bar.sync 1, 128;" ::: "memory");     // s_last is free again
                if (rest) {
                    __threadfence();
                    load_parts(c0);
                }
            }
            if (!all_warps(wait_phase(&tfull[n & 1], (n >> 1) & 1, s_abort, p.dev_status))) break;
            tc_fence_after();
            float v[2][TOK];
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                if (j >= t.cnt) break;
                uint32_t a[DIGITS], b[DIGITS];
                __syncwarp();
                tmem_read12x2(acc + j * DIGITS, acc + NB + j * DIGITS, a, b);
                v[0][j] = add_digits(a);
                v[1][j] = add_digits(b);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[n & 1]);
            if (!whole && !rest) {
                // the last of the tile's CTAs adds the parts up
                float *mine = part_of(me);
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    if (j >= t.cnt) break;
                    __stcg(mine + j * 256, v[0][j]);
                    __stcg(mine + j * 256 + 128, v[1][j]);
                }
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (tid == 128)
                    *s_last = atomicAdd(p.counter + tile, 1u) == static_cast<unsigned>(c1 - c0);
                asm volatile("bar.sync 1, 128;" ::: "memory");
                const bool last = *s_last != 0;
                asm volatile("bar.sync 1, 128;" ::: "memory");     // s_last is free again
                if (!last) continue;
                __threadfence();
            }
            if (!whole) {
                float own[2][TOK];
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    own[0][j] = v[0][j];
                    own[1][j] = v[1][j];
                    v[0][j] = v[1][j] = 0.0f;
                }
                for (int c = c0; c <= c1; c += 4) {
                    if (!rest) load_parts(c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (c + k > c1) break;
                        const bool is_own = c + k == me;
#pragma unroll
                        for (int j = 0; j < TOK; ++j) {
                            if (j >= t.cnt) break;
                            v[0][j] += is_own ? own[0][j] : w[k][0][j];
                            v[1][j] += is_own ? own[1][j] : w[k][1][j];
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                if (j >= t.cnt) break;
                const int row = t.row0 + j;
                // The exponent of the weights first: a sum of digits lies within 2^-52 and
                // 2^42 (NV; alpha is 1 for MX), so alpha's 2^60 either way leaves it in fp32's
                // range, whatever the row.  The row's own power of two first would not: 2^118
                // times such a sum is infinite where a small alpha makes it 1e20.
                const float f = fabsf(scale[j]);
                float a = v[0][j] * p.alpha * f, b = v[1][j] * p.alpha * f;
                if (scale[j] < 0.0f) {
                    a += odd_terms<FMT>(p, row, w0) * p.alpha;
                    if (second) b += odd_terms<FMT>(p, row, w0 + (SWIGLU ? p.N : 128)) * p.alpha;
                }
                if (SWIGLU) a = __fdividef(a, 1.0f + __expf(-a)) * b;
                const int64_t o = static_cast<int64_t>(row) * p.N + n0 + r;
                if (p.out_f32) {
                    float *out = static_cast<float *>(p.out) + o;
                    out[0] = a;
                    if (!SWIGLU && second) out[128] = b;
                } else {
                    uint16_t *out = static_cast<uint16_t *>(p.out) + o;
                    out[0] = float_to_bf16_bits(a);
                    if (!SWIGLU && second) out[128] = float_to_bf16_bits(b);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side
template <typename K, typename P>
cudaError_t start(K kernel, int64_t grid, int block, int smem, const P &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int MAX_CTAS = 256;          // at least the multiprocessors of the GPUs this runs on

Ws layout(int64_t n, int64_t K, int64_t G) {
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    Ws w;
    const size_t blocks = static_cast<size_t>(n / TOK + G);       // 128-row blocks of scales
    w.q = 0;
    w.sf = up(static_cast<size_t>(n) * DIGITS * (K / 2));
    w.scale = w.sf + up(blocks * (K / 64) * kScaleTile);          // NV's, MX takes half
    w.part = w.scale + up(static_cast<size_t>(n) * 4);
    w.counter = w.part + static_cast<size_t>(2 * MAX_CTAS) * PART * 4;
    w.total = w.counter;                                          // + the counters
    return w;
}
size_t workspace_of(int64_t n, int64_t K, int64_t N, int64_t G) {
    return layout(n, K, G).total +
           static_cast<size_t>((n / TOK + std::min(n, G)) * ceil_div(N, 128)) * 4;
}

struct Product {
    const moe_bf16_t *x;
    const int32_t *offsets;
    int G;
    const moe_fp4_t *w;
    int n, K, N;
    bool swiglu;
};

moe_status_t check_sizes(int64_t n, int64_t K, int64_t N, int64_t G) {
    if (G <= 0 || n < 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (G > MAX_GROUPS || K % 128 != 0 || N % 128 != 0 || K > (1 << 20) || N > (1 << 20))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    // digit rows, steps and scale tiles are numbered in 32 bits
    const int64_t lim = int64_t{1} << 31;
    if (n * DIGITS >= lim - 1024 || (n / TOK + G) * (N / 128) * ceil_div(K, BK) >= lim || (n / TOK + G) * (K / 64) >= lim ||
        G * (2 * N / 128) * (K / 64) >= lim)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status_t check(const Product &d) {
    if (!d.w) return MOE_ERR_INVALID_ARG;
    moe_status_t st = check_sizes(d.n, d.K, d.N, d.G);
    if (st == MOE_OK) st = fp4_check(d.w->format, d.w->scale_exp);
    if (st != MOE_OK) return st;
    if (!d.offsets || !d.w->q || !d.w->sf || !a16(d.w->q) || !a16(d.w->sf))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

template <int FMT, bool SWIGLU>
cudaError_t launch(const Product &d, uint32_t flags, void *out, uint8_t *ws, int32_t *dev_status,
                   cudaStream_t stream) {
    using C = Cfg<FMT>;
    constexpr int TK = Fp4<FMT>::TILE_K;
    auto kernel = weight_kernel<FMT, SWIGLU>;
    static std::mutex mu;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !attr_done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(MAX_GROUPS));
            if (e != cudaSuccess) return e;
            if (dev < 64) attr_done[dev] = true;
        }
    }
    const Ws L = layout(d.n, d.K, d.G);
    const int64_t ktiles = d.K / TK, blocks = d.n / TOK + d.G;
    Params p{};
    p.wrows = SWIGLU ? 2 * d.N : d.N;
    if (!code_map(&p.tmA, d.w->q, 3, d.G, p.wrows, d.K, 128) ||
        !scale_map(&p.tmSA, d.w->sf, static_cast<int64_t>(d.G) * (p.wrows / 128) * ktiles, C::TILES) ||
        !code_map(&p.tmB, ws + L.q, 2, 1, static_cast<int64_t>(d.n) * DIGITS, d.K, NB) ||
        !scale_map(&p.tmSB, ws + L.sf, blocks * ktiles, C::TILES))
        return cudaErrorInvalidValue;
    p.x = d.x;
    p.q = d.w->q;
    p.sf = d.w->sf;
    p.row_scale = reinterpret_cast<float *>(ws + L.scale);
    p.counter = reinterpret_cast<unsigned int *>(ws + L.counter);
    p.part = reinterpret_cast<float *>(ws + L.part);
    p.offsets = d.offsets;
    p.G = d.G;
    p.n = d.n;
    p.K = d.K;
    p.N = d.N;
    p.nt = static_cast<int>(ceil_div(d.N, SWIGLU ? 128 : 256));
    p.alpha = pow2f(d.w->scale_exp);
    p.out = out;
    p.out_f32 = (flags & MOE_Y_F32) != 0;
    p.dev_status = dev_status;
    const int64_t tiles = (d.n / TOK + std::min(d.n, d.G)) * static_cast<int64_t>(p.nt);
    const PrepParams q{d.x, d.offsets, d.G, d.n, d.K, ws + L.q, ws + L.sf,
                       reinterpret_cast<float *>(ws + L.scale),
                       reinterpret_cast<unsigned int *>(ws + L.counter), static_cast<int32_t>(tiles),
                       static_cast<int32_t>(ceil_div(d.K / 8, PREP_VECS))};
    const cudaError_t e = start(digits_kernel<FMT>, static_cast<int64_t>(d.n) * q.parts, PREP_THREADS, 0, q, stream);
    if (e != cudaSuccess) return e;
    const int64_t steps = tiles * ceil_div(d.K, BK);
    const int64_t grid = std::max<int64_t>(
        1, std::min<int64_t>(std::min(num_sms(), MAX_CTAS), (steps + 1) / 2));
    return start(kernel, grid, THREADS, C::smem(d.G), p, stream);
}

moe_status_t run(const Product &d, uint32_t flags, void *out, void *workspace, int32_t *dev_status,
                 cudaStream_t s) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const bool mx = d.w->format == MOE_FP4_MX;
    cudaError_t e;
    if (d.swiglu)
        e = mx ? launch<MOE_FP4_MX, true>(d, flags, out, ws, dev_status, s)
               : launch<MOE_FP4_NV, true>(d, flags, out, ws, dev_status, s);
    else
        e = mx ? launch<MOE_FP4_MX, false>(d, flags, out, ws, dev_status, s)
               : launch<MOE_FP4_NV, false>(d, flags, out, ws, dev_status, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool bad_workspace(void *ws, size_t have, size_t need) {
    return !ws || have < need || (reinterpret_cast<uintptr_t>(ws) & 255);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_weight_workspace_size(int32_t n, int32_t K, int32_t N, int32_t G,
                                                      size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_sizes(n, K, N, G);
    if (st != MOE_OK) return st;
    *bytes = workspace_of(n, K, N, G);
    return MOE_OK;
}

static moe_status_t product(const Product &d, uint32_t flags, void *out, void *workspace,
                            size_t workspace_bytes, int32_t *dev_status, moe_stream_t stream) {
    const moe_status_t st = check(d);
    if (st != MOE_OK) return st;
    if (d.n == 0) return MOE_OK;
    if (!d.x || !a16(d.x) || !out || !a16(out)) return MOE_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes, workspace_of(d.n, d.K, d.N, d.G)))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    if (!encode_fn()) return MOE_ERR_CUDA;
    return run(d, flags, out, workspace, dev_status, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_fp4_weight_matmul(const moe_bf16_t *x, const int32_t *offsets, int32_t G,
                                              const moe_fp4_t *w, int32_t n, int32_t K, int32_t N,
                                              uint32_t flags, void *y, void *workspace,
                                              size_t workspace_bytes, int32_t *dev_status,
                                              moe_stream_t stream) {
    return product(Product{x, offsets, G, w, n, K, N, false}, flags, y, workspace, workspace_bytes,
                   dev_status, stream);
}

extern "C" moe_status_t moe_fp4_weight_swiglu(const moe_bf16_t *x, const int32_t *offsets, int32_t G,
                                              const moe_fp4_t *w13, int32_t n, int32_t K, int32_t I,
                                              uint32_t flags, void *act, void *workspace,
                                              size_t workspace_bytes, int32_t *dev_status,
                                              moe_stream_t stream) {
    return product(Product{x, offsets, G, w13, n, K, I, true}, flags, act, workspace, workspace_bytes,
                   dev_status, stream);
}

extern "C" moe_status_t moe_fp4_weight_mlp(const moe_bf16_t *expanded_x, const int32_t *offsets,
                                           int32_t G, const moe_fp4_t *w13, const moe_fp4_t *w2,
                                           int32_t n, int32_t H, int32_t I, uint32_t flags,
                                           moe_bf16_t *act, void *y, void *workspace,
                                           size_t workspace_bytes, int32_t *dev_status,
                                           moe_stream_t stream) {
    const Product up{expanded_x, offsets, G, w13, n, H, I, true}, down{act, offsets, G, w2, n, I, H, false};
    moe_status_t st = check(up);
    if (st == MOE_OK) st = check(down);
    if (st != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    if (!expanded_x || !a16(expanded_x) || !act || !a16(act) || !y || !a16(y))
        return MOE_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes,
                      std::max(workspace_of(n, H, I, G), workspace_of(n, I, H, G))))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    if (!encode_fn()) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = run(up, 0, act, workspace, dev_status, s);
    if (st != MOE_OK) return st;
    return run(down, flags, y, workspace, dev_status, s);
}
