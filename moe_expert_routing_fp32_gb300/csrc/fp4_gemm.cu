// fp4_gemm.cu -- grouped expert matmuls on microscaled 4-bit operands.
//
// With A[r] = sum over blocks of scale * code along K and W[g] likewise,
//   STORE:   y[r, n] = A[r] . W[g, n]                      (bf16 or fp32)
//   SWIGLU:  act[r, n] = bf16(SiLU(A[r] . W[g, n]) * (A[r] . W[g, I + n]))
//   SWIGLU_Q: act quantised again (the next product's operand)
// for the rows r of group g, accumulated in fp32 by the block-scaled
// tcgen05.mma (kind::mxf4 for blocks of 32, kind::mxf4nvf4 for blocks of 16),
// which multiplies the scales in.
//
// One persistent CTA per SM takes 128-row x 256-column tiles in list order.
// A stage holds 256 columns of K: 16 KB of A and 32 KB of B as 128-byte rows
// (the same swizzled K-major tiles as a bf16 slice of 64), and the scale
// tiles, which one thread copies into tensor memory ahead of the stage's four
// MMAs (K = 64 each).  Tensor memory has 512 columns: two 256-column
// accumulators would leave none for the scales, so accumulator 1 starts at
// column 192 and shares 64 columns with accumulator 0; the epilogue drains
// the shared columns first and releases the next tile then, and only that
// part of a drain is not overlapped.
#include <cuda.h>
#include <cuda_runtime.h>

#include <stdlib.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

moe_status_t fp4_check(int format, int scale_exp);

namespace {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 256;                    // elements of K per stage: 128 bytes
constexpr int STAGES = 4;
constexpr int THREADS = 192;
constexpr int A_BYTES = BM * BK / 2;
constexpr int B_BYTES = BN * BK / 2;
constexpr int MAX_GROUPS = 1024;
constexpr int ACC1 = 192;                  // first column of accumulator 1
constexpr int SF_COL = 448;                // scales: columns 448..511
constexpr int TMEM_COLS = 512;

enum { MODE_STORE = 0, MODE_SWIGLU = 1, MODE_SWIGLU_Q = 2 };

struct Params {
    CUtensorMap tmA;        // codes of A: [n, K / 2] bytes, 128-row boxes of 128 bytes
    CUtensorMap tmB;        // codes of W: [G, rows, K / 2] bytes, likewise
    CUtensorMap tmSA;       // scale tiles of A and W: [tiles, 128] 32-bit words
    CUtensorMap tmSB;
    CUtensorMap tmO;        // output, 32-row x 64-byte boxes (pair kernel, not SWIGLU_Q)
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

template <int FMT>
struct Cfg {
    static constexpr int TILES = BK / Fp4<FMT>::TILE_K;        // scale tiles per stage along K
    static constexpr int SA_BYTES = TILES * kScaleTile;
    static constexpr int SB_BYTES = 2 * SA_BYTES;
    static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
    static constexpr int BAR_OFF = STAGES * STAGE;
    static constexpr int NBARS = 2 * STAGES + 4;               // full, empty, tfull[2], tempty, drain
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int OFFS_OFF = MISC_OFF + 16;
    static constexpr int PREFIX_OFF = OFFS_OFF + (MAX_GROUPS + 1) * 4;
    static constexpr int SMEM = 1024 + PREFIX_OFF + (MAX_GROUPS + 2) * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");
    static_assert(SF_COL + 4 * TILES + 8 * TILES <= TMEM_COLS, "scale columns");
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

// D (+)= A * B^T with the scales at sa (rows of A) and sb (rows of B).
// CG = 2: M = 256 over a CTA pair, each CTA holding its 128 rows of A (and
// their scales), half the rows of B and the scales of all of them.
#define MOE_MMA_FP4(GROUP, KIND)                                                              \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                     \
                 "setp.ne.b32 p, %6, 0;\n\t"                                                  \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND                               \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                           \
                 "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)                   \
                 : "memory")
template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
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
// its own shared memory).  Ordered before the MMAs this thread issues
// afterwards, and behind those it issued before.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128u >> 4) << 16;
    d |= static_cast<uint64_t>(128u >> 4) << 32;      // 8-row groups of 16-byte rows
    d |= static_cast<uint64_t>(1u) << 46;
    if (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d)
                     : "memory");
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
// other), columns fastest otherwise.
template <int BMT>
__device__ __forceinline__ Tile decode_tile(const Params &p, int tile, const int *s_off,
                                            const int *s_prefix) {
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    Tile t;
    const int cnt = s_off[lo + 1] - s_off[lo];
    const int mt = (cnt + BMT - 1) / BMT;
    const int local = tile - s_prefix[lo];
    const bool nfast = cnt > p.wrows;
    t.g = lo;
    t.n_blk = nfast ? local % p.nt : local / mt;
    t.row0 = s_off[lo] + (nfast ? local / p.nt : local % mt) * BMT;
    t.row_end = s_off[lo + 1];
    return t;
}

__device__ __forceinline__ float swiglu(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// 32 consecutive act columns of one row: codes and scale bytes.
template <int FMT>
__device__ __forceinline__ void emit_quantized(const Params &p, const uint32_t (&pk)[16], int g,
                                               int start, int row, int col) {
    uint32_t code[4], sc = 0;
    constexpr int W = Fp4<FMT>::BLOCK / 2;            // words of a block
#pragma unroll
    for (int b = 0; b < 16 / W; ++b) {
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
    *reinterpret_cast<uint4 *>(p.q + static_cast<int64_t>(row) * (p.N / 2) + col / 2) =
        make_uint4(code[0], code[1], code[2], code[3]);
    const int64_t tiles = p.N / Fp4<FMT>::TILE_K;
    uint8_t *dst = p.sf +
                   (scale_row_block(g, start, row) * tiles + col / Fp4<FMT>::TILE_K) * kScaleTile +
                   scale_row_offset(row - start) + col / Fp4<FMT>::BLOCK % 4;
    if (FMT == MOE_FP4_MX)
        *dst = static_cast<uint8_t>(sc);
    else
        *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(sc);
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(THREADS, 1) fp4_gemm_kernel(const __grid_constant__ Params p) {
    using C = Cfg<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;       // [2] accumulator complete
    uint64_t *tempty = tfull + 2;           // shared columns drained, once per tile
    uint64_t *drain = tempty + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    volatile int *s_bad = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 8);
    int *s_off = reinterpret_cast<int *>(smem + C::OFFS_OFF);
    int *s_prefix = reinterpret_cast<int *>(smem + C::PREFIX_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) *s_abort = 0;
    if (tid == 32) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&tfull[0], 1);
        mbar_init(&tfull[1], 1);
        mbar_init(tempty, 128);
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (!list_tiles<BM>(p, s_off, s_prefix, s_bad)) {
        if (tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
        return;
    }
    const int total = s_prefix[p.G];
    if (warp == 1) {
        tmem_alloc(s_tmem, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const int kblocks = (p.K + BK - 1) / BK;
    const int ktiles = p.K / Fp4<FMT>::TILE_K;

    if (warp == 0) {
        // ================= TMA producer
        if (elect_one()) {
            tma_prefetch_desc(&p.tmA);
            tma_prefetch_desc(&p.tmB);
            tma_prefetch_desc(&p.tmSA);
            tma_prefetch_desc(&p.tmSB);
            int stage = 0;
            uint32_t phase = 0;
            int armed[STAGES];
            for (int s = 0; s < STAGES; ++s) armed[s] = -1;
            for (int tile = blockIdx.x; tile < total && !*s_abort; tile += gridDim.x) {
                const Tile t = decode_tile<BM>(p, tile, s_off, s_prefix);
                const int sa_blk = static_cast<int>(scale_row_block(t.g, s_off[t.g], t.row0));
                const int b0 = MODE == MODE_STORE ? t.n_blk * BN : t.n_blk * 128;
                const int b1 = MODE == MODE_STORE ? b0 + 128 : p.N + b0;
                const int64_t wblk = static_cast<int64_t>(t.g) * (p.wrows / 128);
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    armed[stage] = static_cast<int>(phase);
                    uint8_t *a = smem + stage * C::STAGE;
                    uint8_t *b = a + A_BYTES;
                    uint8_t *sa = b + B_BYTES;
                    uint8_t *sb = sa + C::SA_BYTES;
                    mbar_arrive_expect_tx(&full[stage], C::STAGE);
                    const int k0 = kb * (BK / 2), t0 = kb * C::TILES;
                    tma_load_2d(a, &p.tmA, &full[stage], k0, t.row0);
                    tma_load_3d(b, &p.tmB, &full[stage], k0, b0, t.g);
                    tma_load_3d(b + B_BYTES / 2, &p.tmB, &full[stage], k0, b1, t.g);
                    tma_load_2d(sa, &p.tmSA, &full[stage], 0, sa_blk * ktiles + t0);
                    tma_load_2d(sb, &p.tmSB, &full[stage], 0,
                                static_cast<int>((wblk + b0 / 128) * ktiles) + t0);
                    tma_load_2d(sb + C::SA_BYTES, &p.tmSB, &full[stage], 0,
                                static_cast<int>((wblk + b1 / 128) * ktiles) + t0);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
            if (*s_abort) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(armed[s]));
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer
        if (elect_one()) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t free_phase = 1;        // the first tile finds both accumulators free
            bool issued = false;
            const uint32_t sa_t = tmem + SF_COL, sb_t = sa_t + 4 * C::TILES;
            for (int tile = blockIdx.x; tile < total && !*s_abort; tile += gridDim.x) {
                if (!mbar_wait_bounded(tempty, free_phase, s_abort, p.dev_status)) break;
                free_phase ^= 1;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(acc * ACC1);
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&full[stage], phase, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + stage * C::STAGE);
                    const uint32_t b = a + A_BYTES;
                    const uint32_t sa = b + B_BYTES;
                    const uint32_t sb = sa + C::SA_BYTES;
#pragma unroll
                    for (int i = 0; i < C::TILES; ++i) {
                        copy_scales<1>(sa_t + 4 * i, sa + i * kScaleTile);
                        copy_scales<1>(sb_t + 8 * i, sb + i * kScaleTile);
                        copy_scales<1>(sb_t + 8 * i + 4, sb + C::SA_BYTES + i * kScaleTile);
                    }
                    // the last slice may hold 128 columns only
                    const int steps = min(BK, p.K - kb * BK) / 64;
                    for (int kk = 0; kk < steps; ++kk) {
                        const int i = FMT == MOE_FP4_MX ? kk / 2 : kk;
                        const uint32_t id = FMT == MOE_FP4_MX && (kk & 1) ? idesc<FMT>(BM, BN, 2)
                                                                          : idesc<FMT>(BM, BN, 0);
                        mma_fp4<FMT, 1>(d, sdesc_kmajor_sw128(a + kk * 32),
                                     sdesc_kmajor_sw128(b + kk * 32), id, sa_t + 4 * i,
                                     sb_t + 8 * i, (kb | kk) != 0 ? 1u : 0u);
                    }
                    issued = true;
                    tc_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit(&tfull[acc]);
                acc ^= 1;
            }
            if (*s_abort && issued) {
                tc_commit(drain);
                mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ================= epilogue (warps 2..5)
        const int quarter = warp & 3;               // TMEM lane quarter of this warp
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
            const Tile t = decode_tile<BM>(p, tile, s_off, s_prefix);
            if (!mbar_wait_bounded(&tfull[acc], acc_phase, s_abort, p.dev_status)) break;
            tc_fence_after();
            const int row = t.row0 + quarter * 32 + lane;
            const bool ok = row < t.row_end;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * ACC1);
            if (MODE != MODE_STORE) {
                // the shared 64 columns hold up columns 64.. of accumulator 0
                // and gate columns ..63 of accumulator 1: that half goes first
                const int first = acc == 0 ? 64 : 0;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int c = (first + 32 * i) & 127;
                    if (i == 2) {
                        __syncwarp();
                        tc_fence_before();
                        mbar_arrive(tempty);
                    }
                    float g[32], u[32];
                    __syncwarp();
                    tmem_ld32(taddr + c, g);
                    tmem_ld32(taddr + 128 + c, u);
                    tmem_ld_wait();
                    uint32_t pk[16];
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        pk[v] = pack_bf16x2(swiglu(g[2 * v] * p.alpha, u[2 * v] * p.alpha),
                                            swiglu(g[2 * v + 1] * p.alpha, u[2 * v + 1] * p.alpha));
                    if (!ok) continue;
                    const int col = t.n_blk * 128 + c;
                    if (MODE == MODE_SWIGLU_Q) {
                        emit_quantized<FMT>(p, pk, t.g, s_off[t.g], row, col);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                                               static_cast<int64_t>(row) * p.N + col);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2],
                                                pk[4 * v + 3]);
                    }
                }
            } else {
                const int first = acc == 0 ? BN - 64 : 0;
#pragma unroll 1
                for (int i = 0; i < BN / 32; ++i) {
                    const int c = (first + 32 * i) & (BN - 1);
                    if (i == 2) {
                        __syncwarp();
                        tc_fence_before();
                        mbar_arrive(tempty);
                    }
                    float v[32];
                    __syncwarp();
                    tmem_ld32(taddr + c, v);
                    tmem_ld_wait();
                    const int col = t.n_blk * BN + c;
                    if (!ok || col >= p.N) continue;
                    const int64_t off = static_cast<int64_t>(row) * p.N + col;
                    if (p.out_f32) {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_float4(v[4 * j] * p.alpha, v[4 * j + 1] * p.alpha,
                                                 v[4 * j + 2] * p.alpha, v[4 * j + 3] * p.alpha);
                    } else {
                        uint4 *dst =
                            reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + off);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                w[x] = pack_bf16x2(v[8 * j + 2 * x] * p.alpha,
                                                   v[8 * j + 2 * x + 1] * p.alpha);
                            dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ CTA pairs
// The same product on 256 x 256 tiles of a cluster of two CTAs
// (tcgen05.mma.cta_group::2).  A one-CTA tile needs 12 KB of operands for an
// MMA of 128 cycles, more than an SM takes in (64 bytes a cycle); a pair
// stages 8 KB per CTA for the same time, half of B each.
//   SWIGLU: the even CTA stages the 128 gate rows, the odd CTA the up rows.
// The scales of B are needed whole in both CTAs' tensor memory.  Scale copies
// go to two sets of columns in turn, two scale tiles at a time, so that a set
// is not rewritten while the MMAs in front still read it.
// Two producer threads per CTA, one for A and one for B, halve the issue time
// of a stage.  Output leaves through TMA stores of 32-row boxes.
constexpr int BM2 = 256;
constexpr int STAGES2 = 5;
constexpr int THREADS2 = 224;              // A producer, MMA, 4 epilogue warps, B producer
constexpr int EPI_BYTES = 32 * 64;         // one output box: 32 rows of 64 bytes

template <int FMT>
struct Cfg2 {
    static constexpr int TILES = Cfg<FMT>::TILES;
    static constexpr int SA_BYTES = TILES * kScaleTile;
    static constexpr int SB_BYTES = 2 * SA_BYTES;
    static constexpr int A_LOAD = A_BYTES + SA_BYTES;             // per CTA
    static constexpr int B_LOAD = B_BYTES / 2 + SB_BYTES;
    static constexpr int STAGE = A_LOAD + B_LOAD;
    static constexpr int EPI_OFF = STAGES2 * STAGE;
    static constexpr int BAR_OFF = EPI_OFF + 4 * 2 * EPI_BYTES;
    static constexpr int NBARS = 2 * STAGES2 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int OFFS_OFF = MISC_OFF + 16;
    static constexpr int PREFIX_OFF = OFFS_OFF + (MAX_GROUPS + 1) * 4;
    static constexpr int SMEM = 1024 + PREFIX_OFF + (MAX_GROUPS + 2) * 4;
    static constexpr int SETS = TILES / 2;                        // scale sets per stage
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGE % 1024 == 0, "swizzled tiles need 1 KB alignment");
    static_assert(SF_COL + 2 * 24 <= TMEM_COLS, "scale columns");
};

// One 32-row x 64-byte output box (lane i holds row row0 + i as 16 words from
// column col on) through one of the warp's two staging boxes, in the 64-byte
// swizzle of the output map, and out as a TMA store.
__device__ __forceinline__ void emit_box(uint8_t *ebox, int &eb, int lane, const uint32_t (&w)[16],
                                         const CUtensorMap *map, int col, int row0) {
    uint8_t *box = ebox + eb * EPI_BYTES;
    if (lane == 0) bulk_wait_read<1>();      // the store that last used this box has read it
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
        *reinterpret_cast<uint4 *>(box + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, box, col, row0);
        bulk_commit();
    }
    eb ^= 1;
}

template <int FMT, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS2, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ Params p) {
    using C = Cfg2<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);   // even CTA's are used
    uint64_t *empty = full + STAGES2;
    uint64_t *tfull = empty + STAGES2;      // [2]
    uint64_t *tempty = tfull + 2;           // even CTA's is used
    uint64_t *drain = tempty + 1;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    volatile int *s_bad = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 8);
    int *s_off = reinterpret_cast<int *>(smem + C::OFFS_OFF);
    int *s_prefix = reinterpret_cast<int *>(smem + C::PREFIX_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int first_tile = static_cast<int>(cluster_id_x());
    const int step = static_cast<int>(gridDim.x) / 2;

    if (tid == 0) *s_abort = 0;
    if (tid == 32) {
        for (int s = 0; s < STAGES2; ++s) {
            mbar_init(&full[s], 2);          // the even CTA's two producers arm their shares
            mbar_init(&empty[s], 1);
        }
        mbar_init(&tfull[0], 1);
        mbar_init(&tfull[1], 1);
        mbar_init(tempty, 8);                // four epilogue warps of both CTAs
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    // both CTAs read the same offsets, so both leave here together
    if (!list_tiles<BM2>(p, s_off, s_prefix, s_bad)) {
        if (tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
        return;
    }
    const int total = s_prefix[p.G];
    if (warp == 1) {
        tmem_alloc_pair(s_tmem, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                      // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lead_full = mapa_shared(smem_u32(full), 0);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    const int kblocks = (p.K + BK - 1) / BK;
    const int ktiles = p.K / Fp4<FMT>::TILE_K;

    if (warp == 0 || warp == 6) {
        // ================= TMA producers: warp 0 A, warp 6 B, each with its scales
        if (elect_one()) {
            const bool is_a = warp == 0;
            tma_prefetch_desc(is_a ? &p.tmA : &p.tmB);
            tma_prefetch_desc(is_a ? &p.tmSA : &p.tmSB);
            int stage = 0;
            uint32_t phase = 0;
            int armed[STAGES2];
            for (int s = 0; s < STAGES2; ++s) armed[s] = -1;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<BM2>(p, tile, s_off, s_prefix);
                const int sa_blk =
                    static_cast<int>(scale_row_block(t.g, s_off[t.g], t.row0)) + rank;
                const int b0 = MODE == MODE_STORE ? t.n_blk * BN : t.n_blk * 128;
                const int b1 = MODE == MODE_STORE ? b0 + 128 : p.N + b0;
                const int64_t wblk = static_cast<int64_t>(t.g) * (p.wrows / 128);
                const int sa0 = sa_blk * ktiles;
                const int sb0 = static_cast<int>((wblk + b0 / 128) * ktiles);
                const int sb1 = static_cast<int>((wblk + b1 / 128) * ktiles);
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    armed[stage] = static_cast<int>(phase);
                    uint8_t *a = smem + stage * C::STAGE;
                    uint8_t *b = a + A_BYTES;
                    uint8_t *sa = b + B_BYTES / 2;
                    uint8_t *sb = sa + C::SA_BYTES;
                    const uint32_t fb = lead_full + 8u * static_cast<uint32_t>(stage);
                    const int k0 = kb * (BK / 2), t0 = kb * C::TILES;
                    if (leader)
                        mbar_arrive_expect_tx(&full[stage], 2u * (is_a ? C::A_LOAD : C::B_LOAD));
                    if (is_a) {
                        tma_load_2d_pair(a, &p.tmA, fb, k0, t.row0 + 128 * rank);
                        tma_load_2d_pair(sa, &p.tmSA, fb, 0, sa0 + t0);
                    } else {
                        tma_load_3d_pair(b, &p.tmB, fb, k0, rank == 0 ? b0 : b1, t.g);
                        tma_load_2d_pair(sb, &p.tmSB, fb, 0, sb0 + t0);
                        tma_load_2d_pair(sb + C::SA_BYTES, &p.tmSB, fb, 0, sb1 + t0);
                    }
                    if (++stage == STAGES2) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
            if (*s_abort && leader) {
                for (int s = 0; s < STAGES2; ++s)
                    if (armed[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(armed[s]));
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer (even CTA only)
        if (leader && elect_one()) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t free_phase = 1;
            uint32_t set = 0;
            bool issued = false;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                if (!mbar_wait_bounded_cluster(tempty, free_phase, s_abort, p.dev_status)) break;
                free_phase ^= 1;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(acc * ACC1);
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded(&full[stage], phase, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + stage * C::STAGE);
                    const uint32_t b = a + A_BYTES;
                    const uint32_t sa = b + B_BYTES / 2;
                    const uint32_t sb = sa + C::SA_BYTES;
                    const int steps = min(BK, p.K - kb * BK) / 64;
                    constexpr int PER = 4 / C::SETS;              // MMAs per scale set
#pragma unroll
                    for (int h = 0; h < C::SETS; ++h) {
                        const uint32_t sa_t = tmem + SF_COL + set * 24u, sb_t = sa_t + 8;
                        if (h * PER >= steps) break;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t o = (2 * h + i) * kScaleTile;
                            copy_scales<2>(sa_t + 4 * i, sa + o);
                            copy_scales<2>(sb_t + 8 * i, sb + o);
                            copy_scales<2>(sb_t + 8 * i + 4, sb + C::SA_BYTES + o);
                        }
                        set ^= 1;
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const int kk = h * PER + j;
                            if (kk >= steps) break;
                            const int i = FMT == MOE_FP4_MX ? j / 2 : j;
                            const uint32_t id = FMT == MOE_FP4_MX && (j & 1)
                                                    ? idesc<FMT>(BM2, BN, 2)
                                                    : idesc<FMT>(BM2, BN, 0);
                            mma_fp4<FMT, 2>(d, sdesc_kmajor_sw128(a + kk * 32),
                                            sdesc_kmajor_sw128(b + kk * 32), id, sa_t + 4 * i,
                                            sb_t + 8 * i, (kb | kk) != 0 ? 1u : 0u);
                        }
                    }
                    issued = true;
                    tc_commit_pair_mc(&empty[stage], 0x3);
                    if (++stage == STAGES2) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair_mc(&tfull[acc], 0x3);
                acc ^= 1;
            }
            if (*s_abort && issued) {
                tc_commit_pair_mc(drain, 0x1);
                mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ================= epilogue (warps 2..5 of both CTAs)
        const int quarter = warp & 3;
        uint8_t *ebox = smem + C::EPI_OFF + (warp - 2) * 2 * EPI_BYTES;
        int eb = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<BM2>(p, tile, s_off, s_prefix);
            if (!mbar_wait_bounded(&tfull[acc], acc_phase, s_abort, p.dev_status)) break;
            tc_fence_after();
            const int row_base = t.row0 + 128 * rank + quarter * 32;
            const int row = row_base + lane;
            const bool ok = row < t.row_end;
            const bool boxed = row_base + 32 <= t.row_end;   // else a group's last rows: by lane
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(acc * ACC1);
            if (MODE != MODE_STORE) {
                const int first = acc == 0 ? 64 : 0;         // the shared columns' half first
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int c = (first + 32 * i) & 127;
                    float g[32], u[32];
                    __syncwarp();
                    tmem_ld32(taddr + c, g);
                    tmem_ld32(taddr + 128 + c, u);
                    tmem_ld_wait();
                    if (i == 1) {
                        __syncwarp();
                        tc_fence_before();
                        if (lane == 0) mbar_arrive_cluster(lead_tempty);
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        pk[v] = pack_bf16x2(swiglu(g[2 * v] * p.alpha, u[2 * v] * p.alpha),
                                            swiglu(g[2 * v + 1] * p.alpha, u[2 * v + 1] * p.alpha));
                    const int col = t.n_blk * 128 + c;
                    if (MODE == MODE_SWIGLU_Q) {
                        if (ok) emit_quantized<FMT>(p, pk, t.g, s_off[t.g], row, col);
                    } else if (boxed) {
                        emit_box(ebox, eb, lane, pk, &p.tmO, col, row_base);
                    } else if (ok) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                                               static_cast<int64_t>(row) * p.N + col);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2],
                                                pk[4 * v + 3]);
                    }
                }
            } else {
                const int first = acc == 0 ? BN - 64 : 0;
#pragma unroll 1
                for (int i = 0; i < BN / 32; ++i) {
                    const int c = (first + 32 * i) & (BN - 1);
                    float v[32];
                    __syncwarp();
                    tmem_ld32(taddr + c, v);
                    tmem_ld_wait();
                    if (i == 1) {
                        __syncwarp();
                        tc_fence_before();
                        if (lane == 0) mbar_arrive_cluster(lead_tempty);
                    }
                    const int col = t.n_blk * BN + c;
                    if (col >= p.N) continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= p.alpha;
                    uint32_t w[16];
                    if (p.out_f32) {
                        float *dst = static_cast<float *>(p.out) + static_cast<int64_t>(row) * p.N + col;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[16 * h + j]);
                            if (boxed) {
                                emit_box(ebox, eb, lane, w, &p.tmO, col + 16 * h, row_base);
                            } else if (ok) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    reinterpret_cast<uint4 *>(dst + 16 * h)[j] = make_uint4(
                                        w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                        if (boxed) {
                            emit_box(ebox, eb, lane, w, &p.tmO, col, row_base);
                        } else if (ok) {
                            uint4 *dst = reinterpret_cast<uint4 *>(
                                static_cast<uint16_t *>(p.out) + static_cast<int64_t>(row) * p.N + col);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2],
                                                    w[4 * j + 3]);
                        }
                    }
                }
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
        if (lane == 0) bulk_wait<0>();       // every output box written
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();      // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
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

// Output [rows, cols] as 32-row x 64-byte boxes, 64-byte swizzled.
bool out_map(CUtensorMap *m, void *out, int64_t rows, int64_t cols, bool f32) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t stride[1] = {static_cast<cuuint64_t>(cols) * esz};
    cuuint32_t boxd[2] = {static_cast<cuuint32_t>(64 / esz), 32}, es[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out,
              dim, stride, boxd, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs take the products with many rows per group.
bool use_pair(int n, int G) {
    static const int64_t least = [] {
        const char *v = getenv("MOE_FP4_PAIR_ROWS");
        return v ? atoll(v) : 256ll;
    }();
    return n / G >= least;
}

template <int FMT, int MODE>
cudaError_t launch_pair(const Params &p, cudaStream_t stream) {
    using C = Cfg2<FMT>;
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
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e != cudaSuccess) return e;
            // no more clusters than can be resident at once
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms()), 1, 1);
            cfg.blockDim = dim3(THREADS2, 1, 1);
            cfg.dynamicSmemBytes = C::SMEM;
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
    const int64_t tiles = (static_cast<int64_t>(p.n / BM2) + p.G) * p.nt;
    const int clusters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(limit, tiles)));
    fp4_gemm_pair_kernel<FMT, MODE><<<2 * clusters, THREADS2, C::SMEM, stream>>>(p);
    return cudaGetLastError();
}

template <int FMT, int MODE>
cudaError_t launch(Params &p, cudaStream_t stream) {
    using C = Cfg<FMT>;
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
                fp4_gemm_kernel<FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
            if (e != cudaSuccess) return e;
            if (dev < 64) attr_done[dev] = true;
        }
    }
    // at most this many tiles: ceil(rows / 128) summed over the groups
    const int64_t tiles = (static_cast<int64_t>(p.n / BM) + p.G) * p.nt;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms(), tiles)));
    fp4_gemm_kernel<FMT, MODE><<<grid, THREADS, C::SMEM, stream>>>(p);
    return cudaGetLastError();
}

struct Product {
    const moe_fp4_t *a, *w;
    const int32_t *offsets;
    int G, n, K, N;
};

template <int FMT>
bool make_maps(Params &p, const Product &d, int wrows) {
    constexpr int TK = Fp4<FMT>::TILE_K;
    const int64_t ktiles = d.K / TK;
    return code_map(&p.tmA, d.a->q, 2, 1, d.n, d.K, BM) &&
           code_map(&p.tmB, d.w->q, 3, d.G, wrows, d.K, 128) &&
           scale_map(&p.tmSA, d.a->sf, (d.n / 128 + d.G) * ktiles, BK / TK) &&
           scale_map(&p.tmSB, d.w->sf, static_cast<int64_t>(d.G) * (wrows / 128) * ktiles, BK / TK);
}

cudaError_t launch_product(const Product &d, int mode, void *out, bool out_f32,
                           const moe_fp4_t *act, int32_t *dev_status, cudaStream_t stream) {
    const bool mx = d.a->format == MOE_FP4_MX;
    const int wrows = mode == MODE_STORE ? d.N : 2 * d.N;
    Params p{};
    if (!(mx ? make_maps<MOE_FP4_MX>(p, d, wrows) : make_maps<MOE_FP4_NV>(p, d, wrows)))
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
    if (d.G > MAX_GROUPS || d.K % 128 != 0 || d.N % 128 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
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
    if (n == 0) return MOE_OK;
    if (!y || !a16(y)) return MOE_ERR_INVALID_ARG;
    st = run_product(up, MODE_SWIGLU_Q, nullptr, false, act, dev_status, stream);
    if (st != MOE_OK) return st;
    return run_product(down, MODE_STORE, y, (flags & MOE_Y_F32) != 0, nullptr, dev_status, stream);
}
