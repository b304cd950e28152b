// fp4_gemm.cu -- grouped expert matmuls on microscaled 4-bit operands.
//
// With A[r] = sum over blocks of scale * code along K and W[g] likewise,
//   STORE:    y[r, n] = A[r] . W[g, n]                      (bf16 or fp32)
//   SWIGLU:   act[r, n] = bf16(SiLU(A[r] . W[g, n]) * (A[r] . W[g, I + n]))
//   SWIGLU_Q: act quantised again (the next product's operand)
// for the rows r of group g, accumulated in fp32 by the block-scaled
// tcgen05.mma (kind::mxf4 for blocks of 32, kind::mxf4nvf4 for blocks of 16),
// which multiplies the scales in.
//
// A persistent kernel takes tiles of CG * 128 rows x 256 columns in list
// order, on one CTA (CG = 1) or a pair (CG = 2, tcgen05 cta_group::2, half of
// B in each CTA).  A stage of the shared-memory ring holds 256 columns of K:
// the operands as 128-byte rows (the swizzled K-major tiles a bf16 slice of 64
// has), and the scale tiles, which are copied into tensor memory ahead of the
// MMAs that use them.
//
// What bounds it.  An MMA of 256 x 256 x 64 takes 128 cycles (measured; 10
// PFLOP/s at 2.07 GHz, the rate of the K = 64 form that is used throughout; the
// chip's published dense 4-bit rate is 13.5), and issuing one, or one of the scale copies, takes its
// thread some 30 to 40, so a slice of 256 columns (512 cycles of MMAs; 4 of them
// and 6 to 12 copies) leaves one thread no room for anything else; and tensor
// memory holds no two 256-column accumulators beside the scales, so with one
// accumulator per tile the MMAs stop while it is drained.  Both go away by
// halves: a tile is two half tiles of 128 columns, each with an issuing thread
// of its own, and the half tiles take three 128-column accumulators in turn.
// The thread of half 0 runs ahead on the staged slices while half 1 waits for an
// accumulator, from then on stays ahead, and half 0 is drained while half 1
// still computes.  (One thread with 256-column MMAs on two accumulators that
// share 64 columns, drained first, against the halves as they then were: 690 us
// to 658, SwiGLU 131072 x 4096 x 4096.)  What is left, in cycles a tile of K = 4096 with a quarter of the
// SMs running (so without the power cap): MMAs and hand-overs alone 9,470 (8,192
// ideal), with the operands' loads 9,930 (they alone 6,870, 83 bytes a cycle), and
// with the output 11,130: an SM's loads and stores add up.  In long runs on all
// SMs the power cap takes a fifth of the clock.
//
// Measured (one GB300): SwiGLU 131072 x 4096 x 4096 (MX) 650 us, 6.8 PFLOP/s at
// 2.07 GHz; in a loop 694-735 us, 6.0-6.3 PFLOP/s, at the power cap's 1.68 GHz.
// 131072 x 2048 x 4096 to fp32 (NV) 545-572 us, 2.6 GB at 4.5-4.8 TB/s: of 8,520 cycles a
// tile (a quarter of the SMs) the loads alone take 3,420 and with the stores
// 7,260.  Weights of 41 experts for 64 rows (365 MB) 60 us, 6.1 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

moe_status_t fp4_check(int format, int scale_exp);

namespace {

constexpr int BM = 128;                    // rows of a tile per CTA
constexpr int BN = 256;                    // columns of a tile
constexpr int HN = 128;                    // columns of a half tile
constexpr int BK = 256;                    // elements of K per stage: 128 bytes
constexpr int MAX_GROUPS = 1024;
constexpr int A_BYTES = BM * BK / 2;
constexpr int NACC = 3;                    // accumulators of HN columns
constexpr int SF_COL = NACC * HN;          // scales: the columns behind them
constexpr int SF_SET = 16;                 // columns of a scale set: two tiles of A, two of B
constexpr int TMEM_COLS = 512;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;   // A and B producers, two issuers, epilogue
constexpr int EPI_BYTES = 32 * 128;        // an output box: 32 rows of 128 bytes

enum { MODE_STORE = 0, MODE_SWIGLU = 1, MODE_SWIGLU_Q = 2 };

struct Params {
    CUtensorMap tmA;        // codes of A: [n, K / 2] bytes, 128-row boxes of 128 bytes
    CUtensorMap tmB;        // codes of W: [G, rows, K / 2] bytes, likewise
    CUtensorMap tmSA;       // scale tiles of A and W: [tiles, 128] 32-bit words
    CUtensorMap tmSB;
    CUtensorMap tmO;        // output, 32-row x 128-byte boxes (pair kernel, not SWIGLU_Q)
    const int32_t *offsets;
    int32_t G, n, K, N;     // N: output columns
    int32_t nt;             // column tiles per row block
    int32_t wrows;          // rows of one group's weights (2N for SwiGLU)
    float alpha;            // 2^(scale exponents)
    void *out;
    int32_t out_f32;
    uint8_t *q;             // SWIGLU_Q
    uint8_t *sf;
    float unit, inv_unit;
    int32_t *dev_status;
};

template <int FMT, int CG>
struct Cfg {
    // four one-CTA stages, or five pair stages and the output boxes, fill shared memory
    static constexpr int STAGES = CG == 1 ? 4 : 5;
    static constexpr int BOXES = CG == 1 ? 0 : EPI_WARPS;
    static constexpr int TILES = BK / Fp4<FMT>::TILE_K;          // scale tiles per stage along K
    static constexpr int B_HALF = HN / CG * BK / 2;              // this CTA's rows of a half of B
    static constexpr int SF_BYTES = TILES * kScaleTile;          // of 128 rows
    static constexpr int A_LOAD = A_BYTES + SF_BYTES;
    static constexpr int B_LOAD = 2 * B_HALF + 2 * SF_BYTES;
    static constexpr int STAGE = A_LOAD + B_LOAD;
    static constexpr int EPI_OFF = STAGES * STAGE;
    static constexpr int BAR_OFF = EPI_OFF + BOXES * EPI_BYTES;
    static constexpr int NBARS = 2 * STAGES + 2 * NACC + 2;      // full, empty, tfull, tempty, drain
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int OFFS_OFF = MISC_OFF + 16;
    // the group offsets and tile prefixes take the rest
    static constexpr int smem(int G) { return 1024 + OFFS_OFF + (2 * G + 2) * 4; }
    static constexpr int MAX_G = (227 * 1024 - 1024 - OFFS_OFF - 8) / 8;
    static_assert(MAX_G >= (CG == 1 ? MAX_GROUPS : 256), "shared memory");
    static_assert(STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");
    static_assert(SF_COL + 2 * 2 * SF_SET <= TMEM_COLS, "scale columns");
};

// Instruction descriptor of the block-scaled MMA: e2m1 operands, both K-major,
// fp32 accumulator; scale type e8m0 (MX) or e4m3 (NV); the scales of a K = 64
// step start at byte `id` of their 32-bit column entries.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int id) {
    return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) |
           (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(FMT == MOE_FP4_MX ? 1 : 0) << 23) |
           (static_cast<uint32_t>(M >> 7) << 27) | (static_cast<uint32_t>(id) << 29);
}

// One lane of a converged warp.  The loops below that issue TMA and tcgen05
// instructions run under this test and not under `lane == 0`: the compiler then
// knows that one lane is active and feeds the instructions' uniform operands
// directly.  Measured: 43 cycles an MMA or scale copy to issue against 80,
// where an MMA of 256 x 256 x 64 takes 128 and a slice of four needs six to
// twelve copies besides.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Bounded wait (as mbar_wait_bounded) whose first 64 polls read no timer: a
// %globaltimer read takes far longer than a hand-over between two roles, and
// here one sits on the path from a finished accumulator to the next tile's
// first MMA.  No wait here publishes ordinary memory between CTAs (operands
// come by TMA, accumulators through tensor memory, each with its own ordering),
// so CTA scope is enough.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort,
                                       int32_t *dev_status) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*abort) return false;
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs || it > (1u << 30)) {
                *abort = 1;
                report(dev_status, MOE_DEV_TIMEOUT);
                return false;
            }
        }
    }
}
// Arrive on a barrier of the pair's even CTA once this warp's tensor memory
// loads have ended (tcgen05.wait::ld and the fence before it order those; a
// cluster-scope release would also wait for its output stores).
__device__ __forceinline__ void arrive_drained(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *abort,
                                           int32_t *dev_status) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, dev_status);
}

// Shared-memory descriptors are kept as their low words, whose address field
// steps by plain additions; the high words are constants.  It leaves the issuing
// threads, which share their schedulers with the epilogue's arithmetic, fewer
// instructions: 246 cycles a slice of four MMAs and four copies against 315.
//   operands: 128-byte swizzled K-major rows, 1 KB between groups of eight
//   scales:   rows of 16 bytes, 128 bytes between groups of eight, no swizzle
constexpr uint32_t OPERAND_LO = 1u << 16, OPERAND_HI = 0x40004040u;
constexpr uint32_t SCALES_LO = 8u << 16, SCALES_HI = 0x00004008u;

// D (+)= A * B^T with the scales at sa (rows of A) and sb (rows of B).
// CG = 2: M = 256 over a CTA pair, each CTA holding its 128 rows of A (and
// their scales), half the rows of B and the scales of all of them.
#define MOE_MMA_FP4(GROUP, KIND)                                                              \
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"                               \
                 "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"                       \
                 "setp.ne.b32 p, %6, 0;\n\t"                                                  \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND                               \
                 " [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d),                           \
                 "r"(a), "r"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate), "n"(OPERAND_HI)  \
                 : "memory")
template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                        uint32_t sa, uint32_t sb, uint32_t accumulate) {
    if (FMT == MOE_FP4_MX && CG == 1)
        MOE_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
    else if (FMT == MOE_FP4_MX)
        MOE_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
    else if (CG == 1)
        MOE_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else
        MOE_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
}
#undef MOE_MMA_FP4

// One 512-byte scale tile (32 rows of 16 bytes) into four columns of tensor
// memory, repeated in its four lane quarters (CG = 2: in both CTAs, each from
// its own shared memory).  The tensor pipe takes one thread's copies and MMAs in
// the order they were issued.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
    if (CG == 1)
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
                     "r"(lo), "n"(SCALES_HI)
                     : "memory");
    else
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
                     "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
                     "r"(lo), "n"(SCALES_HI)
                     : "memory");
}

// One half tile's MMAs over STEPS * 64 columns of K of a stage (4, or 2 in a
// last slice of 128 columns): operand tiles a and b, scale tiles sa and sb
// (descriptors' low words).  Two scale tiles of A and two of B at a time go to one
// of this thread's two sets of columns, in turn, so that a set is not rewritten
// while the MMAs just in front still read it.
template <int FMT, int CG, int STEPS>
__device__ __forceinline__ void issue_slice(uint32_t d, uint32_t a, uint32_t b, uint32_t sa,
                                            uint32_t sb, uint32_t sf_col, uint32_t &set,
                                            bool accumulate) {
    constexpr int PER = FMT == MOE_FP4_MX ? 4 : 2;       // MMAs per set
    constexpr uint32_t ID0 = idesc<FMT>(128 * CG, HN, 0), ID2 = idesc<FMT>(128 * CG, HN, 2);
#pragma unroll
    for (int h = 0; h < (STEPS + PER - 1) / PER; ++h) {
        const uint32_t sa_t = sf_col + set * SF_SET, sb_t = sa_t + 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            copy_scales<CG>(sa_t + 4 * i, sa + (2 * h + i) * (kScaleTile / 16));
            copy_scales<CG>(sb_t + 4 * i, sb + (2 * h + i) * (kScaleTile / 16));
        }
        set ^= 1;
#pragma unroll
        for (int j = 0; j < (STEPS < PER ? STEPS : PER); ++j) {
            const int kk = h * PER + j;
            const int i = FMT == MOE_FP4_MX ? j / 2 : j;
            mma_fp4<FMT, CG>(d, a + kk * 2, b + kk * 2,          // 32 bytes further along K
                             FMT == MOE_FP4_MX && (j & 1) ? ID2 : ID0, sa_t + 4 * i, sb_t + 4 * i,
                             (kk > 0 || accumulate) ? 1u : 0u);
        }
    }
}

struct Tile {
    int g, row0, row_end, n_blk;
};

// Checks the group offsets and lists the tiles: s_prefix[g] = tiles (of BMT
// rows) of the groups before g.  Returns false for bad offsets.  All threads.
template <int BMT>
__device__ bool list_tiles(const Params &p, int *s_off, int *s_prefix, volatile int *s_bad) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int g = tid; g <= p.G; g += blockDim.x) s_off[g] = p.offsets[g];
    if (tid == 0) *s_bad = 0;
    __syncthreads();
    if (tid < 32) {
        int run = 0;
        bool bad = false;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int tiles = 0;
            if (g < p.G) {
                const int a = s_off[g], b = s_off[g + 1];
                if (a < 0 || b < a || b > p.n) bad = true;
                tiles = b > a ? ((b - a + BMT - 1) / BMT) * p.nt : 0;
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
    __syncthreads();
    return *s_bad == 0;
}

// Tiles of a group: rows fastest while the group has fewer rows than its
// weights (a weight tile is read from L2 by its row blocks one after the
// other), columns fastest otherwise.  A role's tiles only ascend, so the group
// is found by walking on from the last one's (`g`); a search per tile costs the
// roles several hundred cycles of latency each.
template <int BMT>
__device__ __forceinline__ Tile decode_tile(const Params &p, int tile, int &g, const int *s_off,
                                            const int *s_prefix) {
    while (s_prefix[g + 1] <= tile) ++g;
    Tile t;
    const int start = s_off[g], end = s_off[g + 1], cnt = end - start;
    const int local = tile - s_prefix[g];
    const bool nfast = cnt > p.wrows;
    const int inner = nfast ? p.nt : (cnt + BMT - 1) / BMT;
    const int hi = static_cast<int>(static_cast<unsigned>(local) / static_cast<unsigned>(inner));
    const int lo = local - hi * inner;
    t.g = g;
    t.n_blk = nfast ? lo : hi;
    t.row0 = start + (nfast ? hi : lo) * BMT;
    t.row_end = end;
    return t;
}

// Two fp32 values in a 64-bit register, for the packed arithmetic.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// SiLU(alpha g) / alpha of two gate sums, g / (1 + 2^(c g)) with c = -alpha log2 e.
// With G = alpha g, the product c g is rounded before the exponential: for
// negative gates that is 2.3 |G| 2^-24 of the result (2^-17 at G = -60), beside
// which the hardware exponential and reciprocal are a few 2^-22; act's own
// rounding is 2^-9.  Below G = -87.3 the sum passes 2^126, the reciprocal is
// flushed and the result is zero, |G| 2^-126 at most from the true one.
__device__ __forceinline__ uint64_t silu2(float x, float y, uint64_t c) {
    const uint64_t g = pair(x, y);
    const float2 t = unpair(mul2(g, c));
    const float2 d = unpair(add2(pair(ex2(t.x), ex2(t.y)), pair(1.0f, 1.0f)));
    return mul2(g, pair(rcp(d.x), rcp(d.y)));
}

// 64 act columns of one row (bf16 pairs, from column col on): codes and scale
// bytes, as moe_fp4_quantize forms them.  act is rounded to bf16 before, as the
// unquantised form is, so that both forms hold the same values.
template <int FMT>
__device__ __forceinline__ void emit_quantized(const Params &p, const uint32_t (&pk)[32], int g,
                                               int start, int row, int col) {
    constexpr int W = Fp4<FMT>::BLOCK / 2;            // words of a block
    uint32_t code[8], sc = 0;
#pragma unroll
    for (int b = 0; b < 32 / W; ++b) {
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint32_t w[4] = {pk[b * W + 4 * i], pk[b * W + 4 * i + 1], pk[b * W + 4 * i + 2],
                                   pk[b * W + 4 * i + 3]};
            am = max(am, amax8(w));
        }
        float factor;
        sc |= block_scale<FMT>(am, p.inv_unit, p.unit, factor) << (8 * b);
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint32_t w[4] = {pk[b * W + 4 * i], pk[b * W + 4 * i + 1], pk[b * W + 4 * i + 2],
                                   pk[b * W + 4 * i + 3]};
            code[b * (W / 4) + i] = quantize8<FMT>(w, factor);
        }
    }
    uint4 *q = reinterpret_cast<uint4 *>(p.q + static_cast<int64_t>(row) * (p.N / 2) + col / 2);
    q[0] = make_uint4(code[0], code[1], code[2], code[3]);
    q[1] = make_uint4(code[4], code[5], code[6], code[7]);
    const int64_t tiles = p.N / Fp4<FMT>::TILE_K;
    uint8_t *dst = p.sf +
                   (scale_row_block(g, start, row) * tiles + col / Fp4<FMT>::TILE_K) * kScaleTile +
                   scale_row_offset(row - start) + col / Fp4<FMT>::BLOCK % 4;
    if (FMT == MOE_FP4_MX)
        *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(sc);
    else
        *reinterpret_cast<uint32_t *>(dst) = sc;
}

// 128 bytes of each of an epilogue warp's 32 rows (lane i: row row0 + i, 64
// bf16 or 32 fp32 values from column col on).  With a box, rows all inside the
// group leave through it, in the 128-byte swizzle of the output map, as one TMA
// store; otherwise, and for a group's last rows, each lane stores its own.
template <typename T>
__device__ __forceinline__ void emit_words(const Params &p, uint8_t *box, int lane, bool boxed,
                                           bool ok, const uint32_t (&w)[32], int col, int row0) {
    if (boxed) {
        if (lane == 0) bulk_wait_read<0>();      // the last store has read the box
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((ch ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(&p.tmO, box, col, row0);
            bulk_commit();
        }
    } else if (ok) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) +
                                               static_cast<int64_t>(row0 + lane) * p.N + col);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
}

// Waits for half tile number u's accumulator (or, with `freed`, for it to be
// free again): number u takes accumulator u % NACC for the u / NACC-th time.
__device__ __forceinline__ bool wait_acc(uint64_t *bars, uint32_t u, bool freed,
                                         volatile int *abort, int32_t *dev_status) {
    return wait_phase(&bars[u % NACC], ((u / NACC) & 1u) ^ (freed ? 1u : 0u), abort, dev_status);
}

template <int FMT, int MODE, int CG>
__device__ __forceinline__ void fp4_gemm(const Params &p) {
    using C = Cfg<FMT, CG>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // a pair's MMAs are issued by its even CTA: full, tempty are used there
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;       // [NACC]
    uint64_t *tempty = tfull + NACC;        // [NACC]
    uint64_t *drain = tempty + NACC;        // [2], one per issuing thread
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    volatile int *s_bad = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 8);
    int *s_off = reinterpret_cast<int *>(smem + C::OFFS_OFF);
    int *s_prefix = s_off + p.G + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = rank == 0;
    const int first_tile = static_cast<int>(blockIdx.x) / CG;
    const int step = static_cast<int>(gridDim.x) / CG;

    // Barriers, tensor memory and descriptors are made ready.
    if (warp == 1) {
        if (CG == 1) {
            tmem_alloc(s_tmem, TMEM_COLS);
            tmem_relinquish();
        } else {
            tmem_alloc_pair(s_tmem, TMEM_COLS);
            tmem_relinquish_pair();
        }
    } else if (warp == 2 && elect_one()) {
        *s_abort = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);          // each producer arms its share
            mbar_init(&empty[s], 2);         // both issuers' MMAs have read it
        }
        for (int i = 0; i < NACC; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], CG * EPI_WARPS);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        fence_barrier_init();
    } else if (warp == 3 && elect_one()) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        tma_prefetch_desc(&p.tmSA);
        tma_prefetch_desc(&p.tmSB);
    }
    // Up to here nothing but shared and tensor memory is touched: launched as a
    // programmatic dependent, this part runs while the stream's last kernel ends.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Bad offsets leave no tiles; both CTAs of a pair read the same ones.
    const bool good = list_tiles<BM * CG>(p, s_off, s_prefix, s_bad);
    if (!good && tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
    const int total = good ? s_prefix[p.G] : 0;
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();         // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lead_full = mapa_shared(smem_u32(full), 0);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    const int kblocks = (p.K + BK - 1) / BK;
    const int ktiles = p.K / Fp4<FMT>::TILE_K;

    if (warp == 0 || warp == 3) {
        // ================= TMA producers: warp 0 A, warp 3 B, each with its scales
        if (elect_one()) {
            const bool is_a = warp == 0;
            int stage = 0;
            uint32_t phase = 0;
            int armed[STAGES];
            for (int s = 0; s < STAGES; ++s) armed[s] = -1;
            auto load2 = [&](void *dst, const CUtensorMap *m, int s, int c0, int c1) {
                if (CG == 1)
                    tma_load_2d(dst, m, &full[s], c0, c1);
                else
                    tma_load_2d_pair(dst, m, lead_full + 8u * static_cast<uint32_t>(s), c0, c1);
            };
            auto load3 = [&](void *dst, const CUtensorMap *m, int s, int c0, int c1, int c2) {
                if (CG == 1)
                    tma_load_3d(dst, m, &full[s], c0, c1, c2);
                else
                    tma_load_3d_pair(dst, m, lead_full + 8u * static_cast<uint32_t>(s), c0, c1, c2);
            };
            int g = 0;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<BM * CG>(p, tile, g, s_off, s_prefix);
                const int sa0 =
                    (static_cast<int>(scale_row_block(t.g, s_off[t.g], t.row0)) + rank) * ktiles;
                // the halves' first rows of B, and this CTA's
                const int b0 = MODE == MODE_STORE ? t.n_blk * BN : t.n_blk * HN;
                const int b1 = MODE == MODE_STORE ? b0 + HN : p.N + b0;
                const int br = rank * (HN / CG);
                const int64_t wblk = static_cast<int64_t>(t.g) * (p.wrows / 128);
                const int sb0 = static_cast<int>((wblk + b0 / 128) * ktiles);
                const int sb1 = static_cast<int>((wblk + b1 / 128) * ktiles);
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_phase(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    armed[stage] = static_cast<int>(phase);
                    uint8_t *a = smem + stage * C::STAGE;
                    uint8_t *b = a + A_BYTES;
                    uint8_t *sf = b + 2 * C::B_HALF;
                    const int k0 = kb * (BK / 2), t0 = kb * C::TILES;
                    if (leader)
                        mbar_arrive_expect_tx(&full[stage], CG * (is_a ? C::A_LOAD : C::B_LOAD));
                    if (is_a) {
                        load2(a, &p.tmA, stage, k0, t.row0 + BM * rank);
                        load2(sf, &p.tmSA, stage, 0, sa0 + t0);
                    } else {
                        load3(b, &p.tmB, stage, k0, b0 + br, t.g);
                        load3(b + C::B_HALF, &p.tmB, stage, k0, b1 + br, t.g);
                        load2(sf + C::SF_BYTES, &p.tmSB, stage, 0, sb0 + t0);
                        load2(sf + 2 * C::SF_BYTES, &p.tmSB, stage, 0, sb1 + t0);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
            if (*s_abort && leader) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(armed[s]));
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ================= MMA issuers: warp 1 half 0, warp 2 half 1 (even CTA only)
        if (leader && elect_one()) {
            const int h = warp - 1;
            int stage = 0;
            uint32_t phase = 0;
            uint32_t u = static_cast<uint32_t>(h);          // half tile number
            uint32_t set = 0;
            const uint32_t sf_col = tmem + SF_COL + static_cast<uint32_t>(h) * 2 * SF_SET;
            const bool tail = p.K % BK != 0;                // the last slice holds 128 columns
            // in units of 16 bytes
            const uint32_t base = smem_u32(smem) >> 4;
            const uint32_t b_off = (A_BYTES + static_cast<uint32_t>(h) * C::B_HALF) / 16;
            const uint32_t sa_off = (A_BYTES + 2 * C::B_HALF) / 16 + SCALES_LO;
            const uint32_t sb_off = (1 + static_cast<uint32_t>(h)) * C::SF_BYTES / 16;
            bool issued = false;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                if (!wait_acc(tempty, u, true, s_abort, p.dev_status)) break;
                tc_fence_after();
                const uint32_t d = tmem + (u % NACC) * HN;
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_phase(&full[stage], phase, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = base + static_cast<uint32_t>(stage) * (C::STAGE / 16);
                    const uint32_t a = at + OPERAND_LO, b = a + b_off;
                    const uint32_t sa = at + sa_off, sb = sa + sb_off;
                    if (kb + 1 < kblocks || !tail)
                        issue_slice<FMT, CG, 4>(d, a, b, sa, sb, sf_col, set, kb != 0);
                    else
                        issue_slice<FMT, CG, 2>(d, a, b, sa, sb, sf_col, set, kb != 0);
                    issued = true;
                    if (CG == 1)
                        tc_commit(&empty[stage]);
                    else
                        tc_commit_pair_mc(&empty[stage], 0x3);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (CG == 1)
                    tc_commit(&tfull[u % NACC]);
                else
                    tc_commit_pair_mc(&tfull[u % NACC], 0x3);
                u += 2;
            }
            if (*s_abort && issued) {
                // unwinding: every MMA issued so far ends before TMEM is freed
                if (CG == 1)
                    tc_commit(&drain[h]);
                else
                    tc_commit_pair_mc(&drain[h], 0x1);
                mbar_wait_drain(&drain[h], 0);
            }
        }
        __syncwarp();
    } else {
        // ================= epilogue (warps 4.. of every CTA)
        // Two warps share a TMEM lane quarter; each takes 64 columns of a half.
        const int quarter = warp & 3;
        const int c0 = 64 * ((warp - 4) >> 2);
        uint8_t *box = smem + C::EPI_OFF + (warp - 4) * EPI_BYTES;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t u = 0;
        // both 32-column parts of this warp's share of half tile u, and release it
        auto drain_half = [&](float (&x)[32], float (&y)[32]) -> bool {
            if (!wait_acc(tfull, u, false, s_abort, p.dev_status)) return false;
            tc_fence_after();
            const uint32_t taddr = tmem + lanes + (u % NACC) * HN + static_cast<uint32_t>(c0);
            __syncwarp();
            tmem_ld32(taddr, x);
            tmem_ld32(taddr + 32, y);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_drained(lead_tempty + 8u * (u % NACC));
            ++u;
            return true;
        };
        // act = SiLU(alpha g) (alpha u) = alpha^2 (g / (1 + e^(-alpha g))) u
        const float c = -1.4426950408889634f * p.alpha, a2 = p.alpha * p.alpha;
        const uint64_t gate_c = pair(c, c), alpha2 = pair(a2, a2);
        int g = 0;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<BM * CG>(p, tile, g, s_off, s_prefix);
            const int row0 = t.row0 + BM * rank + quarter * 32;
            const bool ok = row0 + lane < t.row_end;
            const bool boxed = C::BOXES > 0 && row0 + 32 <= t.row_end;
            if (MODE != MODE_STORE) {
                // half 0 is the gate, half 1 the same columns of up
                float x[32], y[32];
                uint64_t sg[32];
                if (!drain_half(x, y)) break;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sg[i] = silu2(x[2 * i], x[2 * i + 1], gate_c);
                    sg[16 + i] = silu2(y[2 * i], y[2 * i + 1], gate_c);
                }
                if (!drain_half(x, y)) break;
                const int col = t.n_blk * HN + c0;
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float *v = i < 16 ? x + 2 * i : y + 2 * (i - 16);
                    const float2 a = unpair(mul2(mul2(sg[i], pair(v[0], v[1])), alpha2));
                    w[i] = bf16x2(a.x, a.y);
                }
                if (MODE != MODE_SWIGLU_Q)
                    emit_words<uint16_t>(p, box, lane, boxed, ok, w, col, row0);
                else if (ok)
                    emit_quantized<FMT>(p, w, t.g, s_off[t.g], row0 + lane, col);
            } else {
                bool more = true;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float v[2][32];
                    more = drain_half(v[0], v[1]);
                    if (!more) break;
                    const int col = t.n_blk * BN + h * HN + c0;
                    if (col >= p.N) continue;                // N = 128 mod 256: no such columns
                    uint32_t w[32];
                    if (p.out_f32) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[i][j] * p.alpha);
                            emit_words<float>(p, box, lane, boxed, ok, w, col + 32 * i, row0);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            w[j] = bf16x2(v[j / 16][2 * (j % 16)] * p.alpha,
                                               v[j / 16][2 * (j % 16) + 1] * p.alpha);
                        emit_words<uint16_t>(p, box, lane, boxed, ok, w, col, row0);
                    }
                }
                if (!more) break;
            }
        }
        if (C::BOXES > 0 && lane == 0) bulk_wait<0>();   // every output box written
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();     // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        if (CG == 1)
            tmem_dealloc(tmem, TMEM_COLS);
        else
            tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(THREADS, 1) fp4_gemm_kernel(const __grid_constant__ Params p) {
    fp4_gemm<FMT, MODE, 1>(p);
}
template <int FMT, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ Params p) {
    fp4_gemm<FMT, MODE, 2>(p);
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// Codes [groups][rows][K / 2 bytes] as boxes of `box` rows x 128 bytes, swizzled.
bool code_map(CUtensorMap *m, const uint8_t *q, int rank, int64_t groups, int64_t rows, int K,
              int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row_bytes = static_cast<cuuint64_t>(K) / 2;
    cuuint64_t dim[3] = {row_bytes, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(groups)};
    cuuint64_t stride[2] = {row_bytes, row_bytes * static_cast<cuuint64_t>(rows)};
    cuuint32_t boxd[3] = {BK / 2, static_cast<cuuint32_t>(box), 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<uint8_t *>(q), dim, stride, boxd,
              es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 128 words, `box` of them at a time.
bool scale_map(CUtensorMap *m, const uint8_t *sf, int64_t tiles, int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dim[2] = {kScaleTile / 4, static_cast<cuuint64_t>(tiles)};
    cuuint64_t stride[1] = {kScaleTile};
    cuuint32_t boxd[2] = {kScaleTile / 4, static_cast<cuuint32_t>(box)}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(sf), dim, stride, boxd, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [rows, cols] as 32-row x 128-byte boxes, swizzled.
bool out_map(CUtensorMap *m, void *out, int64_t rows, int64_t cols, bool f32) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t stride[1] = {static_cast<cuuint64_t>(cols) * esz};
    cuuint32_t boxd[2] = {static_cast<cuuint32_t>(128 / esz), 32}, es[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out,
              dim, stride, boxd, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs take the products with more than one 128-row block per group on
// average.  Measured with 64 groups (us, pair against one CTA):
//   rows/group    128         160         192         256         512         1024
//   K=4096 SwiGLU 109 : 106   110 : 122   111 : 124   139 : 144   206 : 231   365 : 426
//   K=2048 matmul  68 : 68     70 : 85     71 : 85     85 : 96    128 : 160   223 : 303
// and below, where the weights' bytes decide, one CTA (32 rows: 103 : 92, 58 : 52).
bool use_pair(int n, int G) {
    return n > static_cast<int64_t>(BM) * G &&
           G <= std::min(Cfg<MOE_FP4_MX, 2>::MAX_G, Cfg<MOE_FP4_NV, 2>::MAX_G);
}

// Launched as a programmatic dependent of the stream's last kernel (the kernels
// wait for its end before they read or write memory): 62.2 -> 60.5 us for the
// weights of 41 experts, one product after another.
cudaError_t start(void (*kernel)(const Params), int grid, int smem, const Params &p,
                  cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int FMT, int MODE>
cudaError_t launch_pair(const Params &p, cudaStream_t stream) {
    using C = Cfg<FMT, 2>;
    static std::mutex mu;
    static int max_clusters[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    int limit = num_sms() / 2;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || max_clusters[dev] == 0) {
            const cudaError_t e =
                cudaFuncSetAttribute(fp4_gemm_pair_kernel<FMT, MODE>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            if (e != cudaSuccess) return e;
            // no more clusters than can be resident at once
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms()), 1, 1);
            cfg.blockDim = dim3(THREADS, 1, 1);
            cfg.dynamicSmemBytes = C::smem(C::MAX_G);
            cfg.stream = stream;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, fp4_gemm_pair_kernel<FMT, MODE>, &cfg) !=
                    cudaSuccess ||
                n <= 0) {
                cudaGetLastError();
                n = limit;
            }
            limit = std::min(n, limit);
            if (dev < 64) max_clusters[dev] = limit;
        } else {
            limit = max_clusters[dev];
        }
    }
    const int64_t tiles = (static_cast<int64_t>(p.n / (2 * BM)) + p.G) * p.nt;
    const int clusters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(limit, tiles)));
    return start(fp4_gemm_pair_kernel<FMT, MODE>, 2 * clusters, C::smem(p.G), p, stream);
}

template <int FMT, int MODE>
cudaError_t launch(Params &p, cudaStream_t stream) {
    using C = Cfg<FMT, 1>;
    if (use_pair(p.n, p.G)) {
        if (MODE != MODE_SWIGLU_Q && !out_map(&p.tmO, p.out, p.n, p.N, p.out_f32 != 0))
            return cudaErrorInvalidValue;
        return launch_pair<FMT, MODE>(p, stream);
    }
    static std::mutex mu;
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !attr_done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(
                fp4_gemm_kernel<FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            if (e != cudaSuccess) return e;
            if (dev < 64) attr_done[dev] = true;
        }
    }
    // at most this many tiles: ceil(rows / 128) summed over the groups
    const int64_t tiles = (static_cast<int64_t>(p.n / BM) + p.G) * p.nt;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms(), tiles)));
    return start(fp4_gemm_kernel<FMT, MODE>, grid, C::smem(p.G), p, stream);
}

struct Product {
    const moe_fp4_t *a, *w;
    const int32_t *offsets;
    int G, n, K, N;
};

template <int FMT>
bool make_maps(Params &p, const Product &d, int wrows, bool pair) {
    constexpr int TK = Fp4<FMT>::TILE_K;
    const int64_t ktiles = d.K / TK;
    return code_map(&p.tmA, d.a->q, 2, 1, d.n, d.K, BM) &&
           code_map(&p.tmB, d.w->q, 3, d.G, wrows, d.K, pair ? HN / 2 : HN) &&
           scale_map(&p.tmSA, d.a->sf, (d.n / 128 + d.G) * ktiles, BK / TK) &&
           scale_map(&p.tmSB, d.w->sf, static_cast<int64_t>(d.G) * (wrows / 128) * ktiles, BK / TK);
}

cudaError_t launch_product(const Product &d, int mode, void *out, bool out_f32,
                           const moe_fp4_t *act, int32_t *dev_status, cudaStream_t stream) {
    const bool mx = d.a->format == MOE_FP4_MX;
    const int wrows = mode == MODE_STORE ? d.N : 2 * d.N;
    Params p{};
    const bool pair = use_pair(d.n, d.G);
    if (!(mx ? make_maps<MOE_FP4_MX>(p, d, wrows, pair) : make_maps<MOE_FP4_NV>(p, d, wrows, pair)))
        return cudaErrorInvalidValue;
    p.offsets = d.offsets;
    p.G = d.G;
    p.n = d.n;
    p.K = d.K;
    p.N = d.N;
    p.nt = static_cast<int>(mode == MODE_STORE ? ceil_div(d.N, BN) : d.N / 128);
    p.wrows = wrows;
    p.alpha = pow2f(d.a->scale_exp + d.w->scale_exp);
    p.out = out;
    p.out_f32 = out_f32;
    if (act) {
        p.q = act->q;
        p.sf = act->sf;
        p.unit = pow2f(act->scale_exp);
        p.inv_unit = pow2f(-act->scale_exp);
    }
    p.dev_status = dev_status;
    if (mx) {
        if (mode == MODE_STORE) return launch<MOE_FP4_MX, MODE_STORE>(p, stream);
        if (mode == MODE_SWIGLU) return launch<MOE_FP4_MX, MODE_SWIGLU>(p, stream);
        return launch<MOE_FP4_MX, MODE_SWIGLU_Q>(p, stream);
    }
    if (mode == MODE_STORE) return launch<MOE_FP4_NV, MODE_STORE>(p, stream);
    if (mode == MODE_SWIGLU) return launch<MOE_FP4_NV, MODE_SWIGLU>(p, stream);
    return launch<MOE_FP4_NV, MODE_SWIGLU_Q>(p, stream);
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks common to the products, in the order of the other entry points.
moe_status_t check_product(const Product &d) {
    if (!d.a || !d.w || d.G <= 0 || d.n < 0 || d.K <= 0 || d.N <= 0) return MOE_ERR_INVALID_ARG;
    if (d.a->format != d.w->format) return MOE_ERR_INVALID_ARG;
    moe_status_t st = fp4_check(d.a->format, d.a->scale_exp);
    if (st == MOE_OK) st = fp4_check(d.w->format, d.w->scale_exp);
    if (st != MOE_OK) return st;
    if (d.G > MAX_GROUPS || d.K % 128 != 0 || d.N % 128 != 0 || d.K > (1 << 20) ||
        d.n > INT32_MAX - 1024)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    // tile coordinates and scale tiles are 32-bit
    const int64_t tile_rows = (static_cast<int64_t>(d.n) / 128 + d.G) * (d.K / 64);
    const int64_t w_tiles = static_cast<int64_t>(d.G) * (2 * static_cast<int64_t>(d.N) / 128) * (d.K / 64);
    const int64_t tiles = (static_cast<int64_t>(d.n) / 128 + d.G) * (d.N / 128);
    if (tile_rows >= (int64_t{1} << 31) || w_tiles >= (int64_t{1} << 31) ||
        tiles >= (int64_t{1} << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!d.offsets || !d.w->q || !d.w->sf) return MOE_ERR_INVALID_ARG;
    if (!a16(d.w->q) || !a16(d.w->sf)) return MOE_ERR_INVALID_ARG;
    if (d.n > 0 && (!d.a->q || !d.a->sf || !a16(d.a->q) || !a16(d.a->sf)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// The square of the matrices' common factor stays a normal fp32 number.
bool swiglu_range(const Product &d) {
    const int e = d.a->scale_exp + d.w->scale_exp;
    return e >= -60 && e <= 60;
}

moe_status_t run_product(const Product &d, int mode, void *out, bool out_f32, const moe_fp4_t *act,
                         int32_t *dev_status, moe_stream_t stream) {
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    if (!encode_fn()) return MOE_ERR_CUDA;
    return launch_product(d, mode, out, out_f32, act, dev_status,
                          reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_grouped_matmul(const moe_fp4_t *a, const int32_t *offsets, int32_t G,
                                               const moe_fp4_t *w, int32_t n, int32_t K, int32_t N,
                                               uint32_t flags, void *y, int32_t *dev_status,
                                               moe_stream_t stream) {
    const Product d{a, w, offsets, G, n, K, N};
    const moe_status_t st = check_product(d);
    if (st != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    if (!y || !a16(y)) return MOE_ERR_INVALID_ARG;
    return run_product(d, MODE_STORE, y, (flags & MOE_Y_F32) != 0, nullptr, dev_status, stream);
}

extern "C" moe_status_t moe_fp4_grouped_swiglu(const moe_fp4_t *a, const int32_t *offsets, int32_t G,
                                               const moe_fp4_t *w13, int32_t n, int32_t K, int32_t I,
                                               moe_bf16_t *act, const moe_fp4_t *act4,
                                               int32_t *dev_status, moe_stream_t stream) {
    const Product d{a, w13, offsets, G, n, K, I};
    moe_status_t st = check_product(d);
    if (st != MOE_OK) return st;
    if (!act == !act4) return MOE_ERR_INVALID_ARG;     // one form of the result
    if (!swiglu_range(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (act4) {
        st = fp4_check(act4->format, act4->scale_exp);
        if (st != MOE_OK) return st;
        if (act4->format != a->format) return MOE_ERR_INVALID_ARG;
    }
    if (n == 0) return MOE_OK;
    if (act ? !a16(act) : (!act4->q || !act4->sf || !a16(act4->q) || !a16(act4->sf)))
        return MOE_ERR_INVALID_ARG;
    return run_product(d, act ? MODE_SWIGLU : MODE_SWIGLU_Q, act, false, act4, dev_status, stream);
}

extern "C" moe_status_t moe_fp4_grouped_mlp(const moe_fp4_t *expanded_x, const int32_t *offsets,
                                            int32_t G, const moe_fp4_t *w13, const moe_fp4_t *w2,
                                            int32_t n, int32_t H, int32_t I, uint32_t flags,
                                            const moe_fp4_t *act, void *y, int32_t *dev_status,
                                            moe_stream_t stream) {
    const Product up{expanded_x, w13, offsets, G, n, H, I}, down{act, w2, offsets, G, n, I, H};
    moe_status_t st = check_product(up);
    if (st == MOE_OK) st = check_product(down);
    if (st != MOE_OK) return st;
    if (act->format != expanded_x->format) return MOE_ERR_INVALID_ARG;
    if (!swiglu_range(up)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (n == 0) return MOE_OK;
    if (!y || !a16(y)) return MOE_ERR_INVALID_ARG;
    st = run_product(up, MODE_SWIGLU_Q, nullptr, false, act, dev_status, stream);
    if (st != MOE_OK) return st;
    return run_product(down, MODE_STORE, y, (flags & MOE_Y_F32) != 0, nullptr, dev_status, stream);
}
