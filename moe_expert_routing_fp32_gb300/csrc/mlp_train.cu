// mlp_train.cu -- the expert FFN's training passes on the tensor cores.
//
// For the rows r of group g, [gate up] = x[r] W13[g]^T, act = SiLU(gate) up,
// y = act W2[g]^T.  With s = sigmoid(gate) the gradients are
//   d_act = d_y W2[g],  d_up = d_act gate s,  d_gate = d_act up s (1 + gate (1 - s)),
//   d_x = [d_gate d_up] W13[g],  d_W13[g] = [d_gate d_up]^T x,  d_W2[g] = d_y^T act.
// Five products on one kernel body:
//   FWD   x W13^T, epilogue: h = [gate up] and act, rounded to bf16 once each
//         (act from the fp32 sums, as the forward pass without gradients has it)
//   DOWN  act W2^T = y
//   DACT  d_y W2, epilogue: reads h, writes d_h = [d_gate d_up] and act again
//         (from h: keeping act for the backward pass would cost half of h's
//         memory more, making it again costs n I stores beside a product)
//   DX    d_h W13
//   DW    d_h^T x and d_y^T act over each group's rows, one launch for both
// d_h and act are operands of the next products, hence bf16; everything is
// accumulated in fp32 by the MMAs.
//
// Operand layouts.  Nothing is transposed in memory: the tensor cores take an
// operand whose rows run along K (K-major, as x, act, d_y, d_h and, in the forward
// pass, the weights) or across it (MN-major: the weights in DACT and DX, both
// operands of DW).  A K-major slice is 128-byte rows of 64 K values, an MN-major
// one 128-byte rows of 64 M or N values, one row per K; both in the 128-byte
// swizzle TMA writes.
//
// Ragged groups.  A row tile may read rows of the next group; only the group's
// own are stored.  In DW the rows are the contraction, 16 to an MMA: those of the
// group's last step that belong to the next group (and may hold anything) are
// zeroed in shared memory, of both operands, before the MMA.  Such a slice is
// announced on a barrier of each CTA; the CTA's spare warp zeroes the rows and
// arrives in the producers' place on the barrier that the MMA waits for.
//
// Roles (12 warps): 0 TMA of A, 3 TMA of B, 1 MMA, 2 setup (DW: the zeroes),
// 4-11 epilogue.  Tiles are 256 rows x 256 columns on a pair of CTAs (tcgen05
// cta_group::2, half of B in each CTA), two accumulators in turn; a group's last rows,
// if they are at most 128, are a tile of half the MMA time.
//
// What bounds it.  Many rows a group: the MMAs.  A pair's 256 x 256 tile needs 64 bytes
// a cycle of each multiprocessor for them, all that one gets from L2, so depth of
// the operands' ring and little else on that way decide.  131072 rows of 64 groups, H = 4096,
// I = 2048: forward 3.5-3.9 ms (0.94-0.96 of the MMAs' rate), backward 7.2-8.2 (DX 0.96,
// DW 0.89, DACT 0.83); in a loop under the power cap 4.25-4.45 and 8.5-8.9; the flops' floors are
// 3.5 and 7.0.  Few rows: the weights and their gradients; 509 rows, H = 2048, I = 1024: backward
// 253 us, the bytes' floor 218.  Between, both at once: 32768 rows 650-664 us, floors 311 and
// 438.  Gradients in fp32 cost 1.13 (32768 rows) to 1.54 (509) of the bf16 pass, added to
// what their buffers hold 1.56 to 2.64; their bytes alone say 1.0-1.5 and 1.5-2.5.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BM = 256, BN = 256;           // rows and columns of a tile
constexpr int MAX_GROUPS = 1024;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int EPI_BYTES = 32 * 64;          // an output box: 32 rows of 64 bytes
constexpr int SLICE = 128 * 128;            // bytes of 128 rows (K-major) x 64 K

enum { FWD = 0, DACT = 1, DX = 2, DW = 3, DOWN = 4 };

struct Params {
    CUtensorMap tmA, tmB;      // operands (not DW)
    CUtensorMap tmO0, tmO1;    // FWD: h, act; DACT: d_h, act; DX: d_x; DOWN: y; DW: d_W13, d_W2
    CUtensorMap tmAh, tmBh;    // a pair's tiles of at most 128 rows: 64-row boxes of A (FWD: and B)
    CUtensorMap tmG[4];        // DW's operands: d_h and x, d_y and act
    CUtensorMap tmH;           // DACT: h
    const int32_t *offsets;
    int32_t G, n;
    int32_t K;                 // contraction (not DW)
    int32_t N;                 // FWD, DACT: I; DX, DOWN: H
    int32_t nt;                // column tiles of a row block
    int32_t wrows;             // rows a group's weights would have as an operand like A
    uint16_t *out0, *out1;
    int32_t ld0, ld1;
    // DW: product 0 is d_W13 (M = 2I, N = H), 1 is d_W2 (M = H, N = I)
    int32_t mt0, nt0, mt1, nt1;
    int32_t H, I;
    int32_t w_f32, accumulate;
    int32_t *dev_status;
};

template <int MODE>
struct Cfg {
    // 64-wide slices of K per stage: two at a time load a little faster, one wastes
    // less of a group's last rows (DW, 32768 rows of 64 groups: 645 us a pass, 666 with two)
    // and lets the ring shrink by half as much (DACT)
    static constexpr int KSUB = MODE != DW && MODE != DACT ? 2 : 1;
    // DACT: h comes by TMA, too, into boxes that take a stage's place
    static constexpr int STAGES = MODE == DACT ? 5 : 6 / KSUB;
    static constexpr int A_STAGE = SLICE * KSUB;
    static constexpr int B_SLICE = BN / 2 * 128;
    static constexpr int B_STAGE = B_SLICE * KSUB;
    static constexpr int STAGE = A_STAGE + B_STAGE;
    // behind the stages: an output box per epilogue warp (a second one, filled while the
    // first one's store still reads it, is worth nothing: 655 us a pass of those 32768 rows
    // against 645 with one), and what follows them, counted from there
    static constexpr int EPI_OFF = STAGES * STAGE;
    static constexpr int BOX_BYTES = EPI_WARPS * EPI_BYTES;
    static constexpr int H_BYTES = MODE == DACT ? 2 * BOX_BYTES : 0;     // gate and up of each warp
    static constexpr int BAR_OFF = 0;
    // full, empty, tail, tfull, tempty, drain, h
    static constexpr int NBARS = 3 * STAGES + 5 + (MODE == DACT ? EPI_WARPS : 0);
    static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
    static constexpr int OFFS_OFF = MISC_OFF + 16;
    static constexpr int smem(int G) {
        return 1024 + EPI_OFF + BOX_BYTES + H_BYTES + OFFS_OFF + (MODE == DW ? G + 1 : 2 * G + 2) * 4;
    }
    static constexpr bool A_MN = MODE == DW, B_MN = MODE != FWD && MODE != DOWN;
    // shared-memory descriptors: the high word is the same for both layouts (1 KB
    // between groups of eight 128-byte rows, 128-byte swizzle); the low word's
    // leading offset, between 64-element blocks of M or N, is used by MN-major ones
    static constexpr uint32_t MN_LO = static_cast<uint32_t>(64 * KSUB * 128 / 16) << 16;
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (A_MN ? 1u << 15 : 0u) |
                                      (B_MN ? 1u << 16 : 0u) |
                                      (static_cast<uint32_t>(BN >> 3) << 17) |
                                      (static_cast<uint32_t>(256 >> 4) << 24);
    static_assert(smem(MAX_GROUPS) <= 227 * 1024, "shared memory");
    static_assert(STAGE % 1024 == 0 && BOX_BYTES % 1024 == 0, "alignment");
};

// D (+)= A B^T with the descriptors' low words a and b.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                    uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
                 "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(0x40004040u)
                 : "memory");
}

__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1,
                                             int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
        : "memory");
}
__device__ __forceinline__ void tma_add_3d(const void *tmap, const void *src, int c0, int c1,
                                           int c2) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], "
        "[%4];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
        "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
        : "memory");
}

struct Tile {
    int g;
    int row0, row_end;     // row modes: rows of the tile; DW: rows of the group (the contraction)
    int n_blk;             // row modes: column tile
    int prod, m0, n0;      // DW
};

// Row modes: the group offsets and the tiles of the groups before each;
// returns the number of tiles, -1 for bad offsets.  All threads.
__device__ int list_tiles(const Params &p, int *s_off, int *s_prefix, volatile int *s_bad) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int g = tid; g <= p.G; g += THREADS) s_off[g] = p.offsets[g];
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
                tiles = b > a ? ((b - a + BM - 1) / BM) * p.nt : 0;
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
    return *s_bad ? -1 : s_prefix[p.G];
}

// Tiles of a group: rows fastest while the group has fewer rows than its
// weights, columns fastest otherwise (what is shared is read from L2).  DW: the
// rows of the gradient fastest, both products of a group one after the other.
template <int MODE, int BNT = BN>
__device__ __forceinline__ Tile decode_tile(const Params &p, int tile, int &g, const int *s_off,
                                            const int *s_prefix) {
    Tile t;
    if (MODE == DW) {
        const int t0 = p.mt0 * p.nt0, per = t0 + p.mt1 * p.nt1;
        t.g = tile / per;
        int local = tile - t.g * per;
        t.prod = local >= t0;
        if (t.prod) local -= t0;
        const int mt = t.prod ? p.mt1 : p.mt0;
        const int n = local / mt;
        t.m0 = (local - n * mt) * 256;
        t.n0 = n * BNT;
        t.row0 = s_off[t.g];
        t.row_end = s_off[t.g + 1];
        t.n_blk = 0;
    } else {
        while (s_prefix[g + 1] <= tile) ++g;
        const int start = s_off[g], end = s_off[g + 1], cnt = end - start;
        const int local = tile - s_prefix[g];
        const bool nfast = cnt > p.wrows;
        const int inner = nfast ? p.nt : (cnt + BM - 1) / BM;
        const int hi = static_cast<int>(static_cast<unsigned>(local) / static_cast<unsigned>(inner));
        const int lo = local - hi * inner;
        t.g = g;
        t.n_blk = nfast ? lo : hi;
        t.row0 = start + (nfast ? hi : lo) * BM;
        t.row_end = end;
        t.prod = t.m0 = t.n0 = 0;
    }
    return t;
}

// An epilogue warp's output box.
struct Box {
    uint8_t *at;
    int lane;
    // 64 bytes of each of the warp's 32 rows (lane i: row row0 + i), in the 64-byte
    // swizzle of the output maps; the caller stores it.
    __device__ __forceinline__ void fill(const uint32_t *w) const {
        if (lane == 0) bulk_wait_read<0>();          // the last store has read it
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
            *reinterpret_cast<uint4 *>(at + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        fence_proxy_async();
        __syncwarp();
    }
    // 32 bf16 columns of the rows: through a box where all 32 rows belong to the
    // group, else each lane its own row.
    __device__ __forceinline__ void emit(bool boxed, bool ok, const uint32_t (&w)[16],
                                         const CUtensorMap *map, uint16_t *out, int ld, int row0,
                                         int col) const {
        if (boxed) {
            fill(w);
            if (lane == 0) {
                tma_store_2d(map, at, col, row0);
                bulk_commit();
            }
        } else if (ok) {
            uint4 *dst = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(row0 + lane) * ld + col);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
    }
};

// FWD: 32 columns of gate (x) and up (y) sums to h and act.
__device__ __forceinline__ void emit_forward(const Params &p, const Box &box, bool boxed, bool ok,
                                             const float (&x)[32], const float (&y)[32], int row0,
                                             int col) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2(x[2 * i], x[2 * i + 1]);
    box.emit(boxed, ok, w, &p.tmO0, p.out0, p.ld0, row0, col);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2(y[2 * i], y[2 * i + 1]);
    box.emit(boxed, ok, w, &p.tmO0, p.out0, p.ld0, row0, p.N + col);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float v = x[2 * i + j];
            a[j] = __fdividef(v, 1.0f + __expf(-v)) * y[2 * i + j];
        }
        w[i] = bf16x2(a[0], a[1]);
    }
    box.emit(boxed, ok, w, &p.tmO1, p.out1, p.ld1, row0, col);
}

// DW: 64 columns of a gradient from tensor memory at `taddr`; false where they and
// all further ones are off the gradient (sizes of 128 mod the tile) or nothing has to
// be written (an idle expert's zeros, added).
__device__ __forceinline__ bool emit_gradient(const Params &p, const Box &box, const Tile &t,
                                              uint32_t taddr, int row0, int col) {
    const CUtensorMap *om = t.prod ? &p.tmO1 : &p.tmO0;
    const int M = t.prod ? p.H : 2 * p.I, N = t.prod ? p.I : p.H;
    const bool none = t.row_end == t.row0;
    if (row0 >= M || col >= N || (none && p.accumulate)) return false;
    auto store = [&](const uint32_t *w, int c) {
        box.fill(w);
        if (box.lane == 0) {
            if (p.accumulate)
                tma_add_3d(om, box.at, c, row0, t.g);
            else
                tma_store_3d(om, box.at, c, row0, t.g);
            bulk_commit();
        }
    };
    float v[2][32];
    if (none) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[0][i] = v[1][i] = 0.0f;
    } else {
        __syncwarp();
        tmem_read32(taddr, v[0]);
        tmem_read32(taddr + 32, v[1]);
    }
    uint32_t w[16];
    if (p.w_f32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[k / 2][16 * (k % 2) + i]);
            store(w, col + 16 * k);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = bf16x2(v[k][2 * i], v[k][2 * i + 1]);
            store(w, col + 32 * k);
        }
    }
    return true;
}

// DW: the group offsets, and whether they ascend inside the rows.  All threads.
__device__ __forceinline__ bool load_groups(const Params &p, int *s_off) {
    int bad = 0;
    for (int g = threadIdx.x; g <= p.G; g += THREADS) {
        const int a = p.offsets[g], b = p.offsets[min(g + 1, p.G)];
        s_off[g] = a;
        bad |= a < 0 || b < a || b > p.n;
    }
    return !__syncthreads_or(bad);
}

// wait_phase with an acquire that reaches the other CTA of the pair.
__device__ __forceinline__ bool wait_zeroed(uint64_t *bar, uint32_t parity, volatile int *abort,
                                            int32_t *dev_status) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)                       // no timer is read at first
        if (mbar_try_wait_cluster(bar, parity)) return true;
    return mbar_wait_bounded_cluster(bar, parity, abort, dev_status);
}

// DW: whether the group's last 16-row step has rows of the next group in it.
__device__ __forceinline__ bool has_tail(const Tile &t) { return ((t.row_end - t.row0) & 15) != 0; }
// The parities of the stages' tail barriers, which complete a phase per use.
struct Tails {
    uint32_t used = 0, parity = 0;      // by stage
    __device__ __forceinline__ void arm(int s) {
        used |= 1u << s;
        parity ^= 1u << s;
    }
    __device__ __forceinline__ uint32_t take(int s) {
        const uint32_t p = (parity >> s) & 1u;
        parity ^= 1u << s;
        return p;
    }
    // the last loads announced on each barrier land before the CTA leaves
    __device__ __forceinline__ void drain(uint64_t *tail, int stages) const {
        for (int s = 0; s < stages; ++s)
            if ((used >> s) & 1u) mbar_wait_drain(&tail[s], ((parity >> s) & 1u) ^ 1u);
    }
};
// Rows `from` .. the end of its step of 16 in each of a stage's blocks of 64 rows x
// 128 bytes (a row is 128 bytes in the swizzle, too).  One warp.
__device__ __forceinline__ void zero_rows(uint8_t *stage, int blocks, int from, int lane) {
    const int to = (from + 15) & ~15;
    for (int b = 0; b < blocks; ++b)
        for (int r = from + (lane >> 3); r < to; r += 4)     // eight lanes a row
            *reinterpret_cast<uint4 *>(stage + b * (64 * 128) + r * 128 + (lane & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    __syncwarp();
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    train_gemm_kernel(const __grid_constant__ Params p) {
    using C = Cfg<MODE>;
    constexpr int STAGES = C::STAGES, KSUB = C::KSUB, BK = 64 * KSUB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // a pair's MMAs are issued by its even CTA: full, tempty are used there
    uint8_t *h_boxes = smem + C::EPI_OFF + C::BOX_BYTES;
    uint8_t *rest = h_boxes + C::H_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(rest + C::BAR_OFF);
    uint64_t *empty = full + STAGES;
    uint64_t *tail = empty + STAGES;        // DW: a stage that needs zeroes has landed here
    uint64_t *tfull = tail + STAGES;        // [2]
    uint64_t *tempty = tfull + 2;           // [2]
    uint64_t *drain = tempty + 2;
    uint64_t *h_full = drain + 1;           // an epilogue warp's boxes of h have landed
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(rest + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(rest + C::MISC_OFF + 4);
    volatile int *s_bad = reinterpret_cast<volatile int *>(rest + C::MISC_OFF + 8);
    int *s_off = reinterpret_cast<int *>(rest + C::OFFS_OFF);
    int *s_prefix = s_off + p.G + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int first_tile = static_cast<int>(blockIdx.x) / 2, step = static_cast<int>(gridDim.x) / 2;

    if (warp == 1) {
        tmem_alloc_pair(s_tmem, 512);
        tmem_relinquish_pair();
    } else if (warp == 2 && elect_one()) {
        *s_abort = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);          // each producer arms its share
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        if (MODE == DACT)
            for (int i = 0; i < EPI_WARPS; ++i) mbar_init(&h_full[i], 1);
        fence_barrier_init();
    } else if (warp == 3 && MODE != DW && elect_one()) {
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
    }
    int total;
    if (MODE == DW) {
        total = load_groups(p, s_off) ? p.G * (p.mt0 * p.nt0 + p.mt1 * p.nt1) : -1;
    } else {
        total = list_tiles(p, s_off, s_prefix, s_bad);
    }
    if (total < 0) {                         // both CTAs of a pair read the same offsets
        if (tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
        total = 0;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                      // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lead_full = mapa_shared(smem_u32(full), 0);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    // a pair's tile of at most 128 rows (256 rows a group: forward 204 -> 197 us, backward
    // 455 -> 449, 512: 319 -> 307 and no change)
    auto is_half = [&](const Tile &t) { return MODE != DW && t.row_end - t.row0 <= 128; };
    auto kblocks = [&](const Tile &t) {
        return MODE == DW ? (t.row_end - t.row0 + BK - 1) / BK : (p.K + BK - 1) / BK;
    };

    if (warp == 0 || warp == 3) {
        // ================= TMA producers: warp 0 A, warp 3 B
        if (elect_one()) {
            const bool is_a = warp == 0;
            int stage = 0;
            uint32_t phase = 0;
            int armed[STAGES];
            for (int s = 0; s < STAGES; ++s) armed[s] = -1;
            Tails tails;
            auto load2 = [&](void *dst, const CUtensorMap *m, int s, int c0, int c1) {
                tma_load_2d_pair(dst, m, lead_full + 8u * static_cast<uint32_t>(s), c0, c1);
            };
            auto load3 = [&](void *dst, const CUtensorMap *m, int s, int c0, int c1, int c2) {
                tma_load_3d_pair(dst, m, lead_full + 8u * static_cast<uint32_t>(s), c0, c1, c2);
            };
            int g = 0;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<MODE>(p, tile, g, s_off, s_prefix);
                const bool half = is_half(t);
                const CUtensorMap *m = MODE == DW ? &p.tmG[2 * t.prod + (is_a ? 0 : 1)]
                                       : is_a     ? (half ? &p.tmAh : &p.tmA)
                                                  : (half && MODE == FWD ? &p.tmBh : &p.tmB);
                const int nkb = kblocks(t);
                const uint32_t tx = 2 * (is_a ? C::A_STAGE / (half ? 2 : 1) : C::B_STAGE);
                bool ok = true;
                for (int i = 0; i < nkb; ++i) {
                    const int kb = MODE == DW && has_tail(t) ? (i == 0 ? nkb - 1 : i - 1) : i;
                    if (!wait_phase(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = smem + stage * C::STAGE + (is_a ? 0 : C::A_STAGE);
                    const int k0 = kb * BK;
                    if (MODE == DW && kb + 1 == nkb && has_tail(t)) {
                        // to this CTA's own barrier, for the warp that zeroes
                        const int c = (is_a ? t.m0 : t.n0) + 128 * rank;
                        mbar_arrive_expect_tx(&tail[stage], is_a ? C::A_STAGE : C::B_STAGE);
                        tails.arm(stage);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            tma_load_2d(dst + j * (64 * BK * 2), m, &tail[stage], c + 64 * j, t.row0 + k0);
                        armed[stage] = -1;
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                        continue;
                    }
                    armed[stage] = static_cast<int>(phase);
                    if (leader)
                        mbar_arrive_expect_tx(&full[stage], tx);
                    if (MODE == DW) {
                        const int c = (is_a ? t.m0 : t.n0) + 128 * rank;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            load2(dst + j * (64 * BK * 2), m, stage, c + 64 * j, t.row0 + k0);
                    } else if (is_a) {
#pragma unroll
                        for (int s = 0; s < KSUB; ++s)
                            load2(dst + s * SLICE, m, stage, k0 + 64 * s, t.row0 + (half ? 64 : 128) * rank);
                    } else if (MODE == FWD && half) {
                        // 64 gate rows and the same of up in each CTA
#pragma unroll
                        for (int s = 0; s < KSUB; ++s)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                load3(dst + s * C::B_SLICE + j * (SLICE / 2), m, stage, k0 + 64 * s,
                                      j * p.N + t.n_blk * 128 + 64 * rank, t.g);
                    } else if (MODE == FWD) {
                        // gate rows in the even CTA, up's in the odd one
#pragma unroll
                        for (int s = 0; s < KSUB; ++s)
                            load3(dst + s * C::B_SLICE, m, stage, k0 + 64 * s, rank * p.N + t.n_blk * 128,
                                  t.g);
                    } else if (MODE == DOWN) {
#pragma unroll
                        for (int s = 0; s < KSUB; ++s)
                            load3(dst + s * C::B_SLICE, m, stage, k0 + 64 * s, t.n_blk * BN + 128 * rank,
                                  t.g);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            load3(dst + j * (64 * BK * 2), m, stage, t.n_blk * BN + 128 * rank + 64 * j, k0,
                                  t.g);
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
            if (MODE == DW && *s_abort) tails.drain(tail, STAGES);
        }
        __syncwarp();
    } else if (MODE == DW && warp == 2) {
        // ================= zeroes: the rows behind a group in its last step
        int stage = 0, g = 0;
        Tails tails;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<MODE>(p, tile, g, s_off, s_prefix);
            const int nkb = kblocks(t);
            if (has_tail(t)) {                       // a tile's first stage
                if (!whole_warp(wait_phase(&tail[stage], tails.take(stage), s_abort, p.dev_status))) break;
                zero_rows(smem + stage * C::STAGE, C::STAGE / (64 * 128), t.row_end - t.row0 - (nkb - 1) * BK, lane);
                if (lane == 0) mbar_arrive_cluster(lead_full + 8u * static_cast<uint32_t>(stage));
            }
            stage = (stage + nkb) % STAGES;
        }
    } else if (warp == 1) {
        // ================= MMA issuer (even CTA only)
        if (leader && elect_one()) {
            int stage = 0;
            uint32_t phase = 0, u = 0;              // u: tile count, accumulator u & 1
            const uint32_t base = smem_u32(smem) >> 4;
            bool issued = false;
            int g = 0;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<MODE>(p, tile, g, s_off, s_prefix);
                const int nkb = kblocks(t);
                // DW: the 16-row steps of the last slice that hold rows of the group
                const int last =
                    MODE == DW ? (t.row_end - t.row0 - (nkb - 1) * BK + 15) / 16 : BK / 16;
                if (!wait_phase(&tempty[u & 1], ((u >> 1) & 1) ^ 1, s_abort, p.dev_status)) break;
                tc_fence_after();
                const uint32_t d = tmem + (u & 1) * BN;
                const uint32_t idesc = is_half(t) ? C::IDESC - (8u << 24) : C::IDESC;    // M = 128
                bool ok = true;
                // DW's slice with zeroes is loaded first and taken some slices later (as many as
                // the ring allows), so that nobody waits for its zeroes
                const bool early = MODE == DW && nkb > 0 && has_tail(t);
                const int taken = early ? min(nkb - 1, STAGES - 2) : 0;
                for (int i = 0; i < nkb; ++i) {
                    // place in the order of loading, slice, stage
                    const int at = !early || i > taken ? i : i == taken ? 0 : i + 1;
                    const int kb = !early ? at : at == 0 ? nkb - 1 : at - 1;
                    const int ring = stage + at, st = ring % STAGES;
                    const uint32_t ph = phase ^ (static_cast<uint32_t>(ring / STAGES) & 1u);
                    // (zeroes are written by the warps of both CTAs, through the generic proxy)
                    const bool zeroed = early && at == 0;
                    if (zeroed ? !wait_zeroed(&full[st], ph, s_abort, p.dev_status)
                               : !wait_phase(&full[st], ph, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    if (zeroed) fence_proxy_async();
                    tc_fence_after();
                    const uint32_t addr = base + static_cast<uint32_t>(st) * (C::STAGE / 16);
                    const uint32_t a = addr + (C::A_MN ? C::MN_LO : 1u << 16);
                    const uint32_t b = addr + C::A_STAGE / 16 + (C::B_MN ? C::MN_LO : 1u << 16);
                    const int steps = kb + 1 < nkb ? BK / 16 : last;
#pragma unroll
                    for (int s = 0; s < BK / 16; ++s) {
                        if (MODE == DW && s >= steps) break;
                        // 16 K further: 32 bytes of each row, or 16 rows of 128 bytes
                        const uint32_t ka = C::A_MN ? s * 128 : s / 4 * (SLICE / 16) + s % 4 * 2;
                        const uint32_t kbb =
                            C::B_MN ? s * 128 : s / 4 * (C::B_SLICE / 16) + s % 4 * 2;
                        mma(d, a + ka, b + kbb, idesc, (i | s) != 0 ? 1u : 0u);
                    }
                    issued = true;
                    tc_commit_pair_mc(&empty[st], 0x3);
                }
                if (!ok) break;
                stage += nkb;
                phase ^= static_cast<uint32_t>(stage / STAGES) & 1u;
                stage %= STAGES;
                tc_commit_pair_mc(&tfull[u & 1], 0x3);
                ++u;
            }
            if (*s_abort && issued) {
                // unwinding: every MMA issued so far ends before TMEM is freed
                tc_commit_pair_mc(drain, 0x1);
                mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ================= epilogue: two warps share a TMEM lane quarter
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const Box box{smem + C::EPI_OFF + (warp - 4) * EPI_BYTES, lane};
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t *h_box = h_boxes + (warp - 4) * (2 * EPI_BYTES);
        uint32_t h_phase = 0;
        bool h_pending = false, lost = false;
        int g = 0;
        uint32_t u = 0;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<MODE>(p, tile, g, s_off, s_prefix);
            // half tiles: 64 rows a CTA, N's lower 128 columns in lanes 0-63 and its upper
            // ones, of the same rows, in lanes 64-127
            const bool half = is_half(t);
            const int hq = half ? quarter >> 1 : 0;
            const int row0 = (MODE == DW ? t.m0 : t.row0) + (half ? 64 : 128) * rank +
                             32 * (half ? quarter & 1 : quarter);
            const int span = half ? 64 : 128;       // columns of this warp (FWD: of gate and up)
            const bool ok = row0 + lane < t.row_end;
            const bool boxed = row0 + 32 <= t.row_end;
            const uint32_t acc = tmem + lanes + (u & 1) * BN;
            // DACT: 32 columns of gate and up of h, fetched one step ahead (the first while the
            // tile is still computed) by TMA into the warp's own boxes.  Loads of a row per
            // lane keep the other roles' instructions waiting: 1,364 cycles a slice of 128
            // against 1,238 (131072 rows of H = 4096, I = 2048).
            auto fetch_h = [&](int c) {
                const int col = t.n_blk * BN + 128 * hq + c;
                if (col >= p.N) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&h_full[warp - 4], 2 * EPI_BYTES);
                    tma_load_2d(h_box, &p.tmH, &h_full[warp - 4], col, row0);
                    tma_load_2d(h_box + EPI_BYTES, &p.tmH, &h_full[warp - 4], p.N + col, row0);
                }
                h_pending = true;
            };
            if (MODE == DACT) fetch_h(span * part);
            if (!whole_warp(wait_phase(&tfull[u & 1], (u >> 1) & 1, s_abort, p.dev_status))) break;
            tc_fence_after();
            if (MODE == FWD) {
                // columns [0, span) gate, [span, 2 span) up; this warp takes half of each
#pragma unroll 1
                for (int c = span / 2 * part; c < span / 2 * (part + 1); c += 32) {
                    float x[32], y[32];
                    __syncwarp();
                    tmem_read32(acc + c, x);
                    tmem_read32(acc + span + c, y);
                    emit_forward(p, box, boxed, ok, x, y, row0, t.n_blk * 128 + 64 * hq + c);
                }
            } else if (MODE == DACT) {
#pragma unroll 1
                for (int c = span * part; c < span * (part + 1); c += 32) {
                    const int col = t.n_blk * BN + 128 * hq + c;
                    if (col >= p.N) break;               // N = 128 mod 256: no such columns
                    if (!whole_warp(wait_phase(&h_full[warp - 4], h_phase, s_abort, p.dev_status))) {
                        lost = true;
                        break;
                    }
                    h_phase ^= 1;
                    h_pending = false;
                    uint32_t hg[16], hu[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);
                        const uint4 g4 = *reinterpret_cast<const uint4 *>(h_box + at);
                        const uint4 u4 = *reinterpret_cast<const uint4 *>(h_box + EPI_BYTES + at);
                        hg[4 * j] = g4.x, hg[4 * j + 1] = g4.y, hg[4 * j + 2] = g4.z, hg[4 * j + 3] = g4.w;
                        hu[4 * j] = u4.x, hu[4 * j + 1] = u4.y, hu[4 * j + 2] = u4.z, hu[4 * j + 3] = u4.w;
                    }
                    // the reads are over before the next ones land there (a barrier of the
                    // warp alone lets them wait in line behind its stores of single rows)
                    fence_proxy_async();
                    __syncwarp();
                    if (c + 32 < span * (part + 1)) fetch_h(c + 32);
                    float d[32];
                    __syncwarp();
                    tmem_read32(acc + c, d);
                    uint32_t wg[16], wu[16], wa[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const f2 gt = from_bf16x2(hg[i]), up = from_bf16x2(hu[i]);
                        const f2 dd = pack2(d[2 * i], d[2 * i + 1]);
                        // s = 1 / (1 + 2^(-gate log2 e))
                        const float2 e = unpack2(mul2(gt, splat(-1.4426950408889634f)));
                        const float2 q = unpack2(add2(pack2(ex2(e.x), ex2(e.y)), splat(1.0f)));
                        const f2 s = pack2(rcp(q.x), rcp(q.y));
                        const f2 gs = mul2(gt, s);                  // SiLU(gate)
                        wa[i] = to_bf16x2(mul2(gs, up));
                        wu[i] = to_bf16x2(mul2(dd, gs));
                        // s (1 + gate (1 - s)) = s + gs (1 - s)
                        const f2 t = fma2(gs, fma2(s, splat(-1.0f), splat(1.0f)), s);
                        wg[i] = to_bf16x2(mul2(mul2(dd, up), t));
                    }
                    box.emit(boxed, ok, wg, &p.tmO0, p.out0, p.ld0, row0, col);
                    box.emit(boxed, ok, wu, &p.tmO0, p.out0, p.ld0, row0,
                              p.N + col);
                    box.emit(boxed, ok, wa, &p.tmO1, p.out1, p.ld1, row0, col);
                }
                if (lost) break;
            } else if (MODE == DX || MODE == DOWN) {
#pragma unroll 1
                for (int c = span * part; c < span * (part + 1); c += 32) {
                    const int col = t.n_blk * BN + 128 * hq + c;
                    if (col >= p.N) break;
                    float v[32];
                    __syncwarp();
                    tmem_read32(acc + c, v);
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
                    box.emit(boxed, ok, w, &p.tmO0, p.out0, p.ld0, row0, col);
                }
            } else {
#pragma unroll 1
                for (int c = 128 * part; c < 128 * part + 128; c += 64)
                    if (!emit_gradient(p, box, t, acc + c, row0, t.n0 + c)) break;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_drained(lead_tempty + 8u * (u & 1));
            ++u;
        }
        if (MODE == DACT && h_pending) mbar_wait_drain(&h_full[warp - 4], h_phase);    // unwinding
        if (lane == 0) bulk_wait<0>();       // every output box written
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                  // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    __syncwarp();
    cluster_sync_all();                  // nor before both have given their tensor memory back
}

// ------------------------------------------------------------------ wide tiles
// DW in tiles of 256 rows x 512 columns per CTA pair: half as many hand-overs
// between the roles, and 48 KB of operands for the MMAs that take 64 KB in 256 x 256
// tiles.  The accumulator fills tensor memory, so tiles overlap by halves of 256
// columns: the epilogue drains half 0 and then half 1; the next tile's MMAs start on
// half 0 as soon as that is free and run ahead on it over the staged slices until
// half 1 is free, too; and a tile's last W_TAIL slices issue their half-1 MMAs after
// all of half 0, which is then drained while they run.  CTA r stages columns
// [256 r, 256 r + 256); column j of half h is column 128 h + j (j < 128) or
// 256 + 128 h + (j - 128).
constexpr int BW = 512;
constexpr int W_STAGES = 4;
constexpr int W_TAIL = 3;
constexpr int W_B = 2 * SLICE;                       // 256 columns (or rows) x 64 K
constexpr int W_STAGE = SLICE + W_B;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gradient_wide_kernel(const __grid_constant__ Params p) {
    using C = Cfg<DW>;
    static_assert(W_STAGES * W_STAGE == C::EPI_OFF && W_STAGES <= C::STAGES, "shared memory");
    constexpr int BK = 64;
    constexpr uint32_t MN_LO = static_cast<uint32_t>(64 * 128 / 16) << 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *rest = smem + C::EPI_OFF + C::BOX_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(rest + C::BAR_OFF);    // used in the even CTA
    uint64_t *empty = full + W_STAGES;
    uint64_t *tail = empty + W_STAGES;      // a stage that needs zeroes has landed here
    uint64_t *tfull = tail + W_STAGES;      // [2]: half h is complete
    uint64_t *tempty = tfull + 2;           // [2], used in the even CTA
    uint64_t *drain = tempty + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(rest + C::MISC_OFF);
    volatile int *s_abort = reinterpret_cast<volatile int *>(rest + C::MISC_OFF + 4);
    int *s_off = reinterpret_cast<int *>(rest + C::OFFS_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int first_tile = static_cast<int>(blockIdx.x) / 2, step = static_cast<int>(gridDim.x) / 2;

    if (warp == 1) {
        tmem_alloc_pair(s_tmem, 512);
        tmem_relinquish_pair();
    } else if (warp == 2 && elect_one()) {
        *s_abort = 0;
        for (int s = 0; s < W_STAGES; ++s) {
            mbar_init(&full[s], 2);          // each producer arms its share
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    int total = load_groups(p, s_off) ? p.G * (p.mt0 * p.nt0 + p.mt1 * p.nt1) : -1;
    if (total < 0) {                         // both CTAs of a pair read the same offsets
        if (tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
        total = 0;
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                      // barriers and TMEM of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lead_full = mapa_shared(smem_u32(full), 0);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    auto slices = [&](const Tile &t) { return (t.row_end - t.row0 + BK - 1) / BK; };

    if (warp == 0 || warp == 3) {
        // ================= TMA producers: warp 0 A, warp 3 B
        if (elect_one()) {
            const bool is_a = warp == 0;
            int stage = 0;
            uint32_t phase = 0;
            int armed[W_STAGES];
            for (int s = 0; s < W_STAGES; ++s) armed[s] = -1;
            Tails tails;
            int g = 0;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<DW, BW>(p, tile, g, s_off, nullptr);
                const int nkb = slices(t);
                const CUtensorMap *m = &p.tmG[2 * t.prod + (is_a ? 0 : 1)];
                bool ok = true;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait_phase(&empty[stage], phase ^ 1, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = smem + stage * W_STAGE + (is_a ? 0 : SLICE);
                    const uint32_t fb = lead_full + 8u * static_cast<uint32_t>(stage);
                    // with zeroes to come: to this CTA's own barrier
                    const bool last = kb + 1 == nkb && has_tail(t);
                    if (last) {
                        mbar_arrive_expect_tx(&tail[stage], is_a ? SLICE : W_B);
                        tails.arm(stage);
                    } else if (leader) {
                        mbar_arrive_expect_tx(&full[stage], 2 * (is_a ? SLICE : W_B));
                    }
                    armed[stage] = last ? -1 : static_cast<int>(phase);
                    const int c = is_a ? t.m0 + 128 * rank : t.n0 + 256 * rank;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (is_a && j >= 2) break;
                        if (last)
                            tma_load_2d(dst + j * (SLICE / 2), m, &tail[stage], c + 64 * j, t.row0 + kb * BK);
                        else
                            tma_load_2d_pair(dst + j * (SLICE / 2), m, fb, c + 64 * j, t.row0 + kb * BK);
                    }
                    if (++stage == W_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
            if (*s_abort && leader) {
                for (int s = 0; s < W_STAGES; ++s)
                    if (armed[s] >= 0) mbar_wait_drain(&full[s], static_cast<uint32_t>(armed[s]));
            }
            if (*s_abort) tails.drain(tail, W_STAGES);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ================= zeroes: the rows behind a group in its last step
        int stage = 0, g = 0;
        Tails tails;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<DW, BW>(p, tile, g, s_off, nullptr);
            const int nkb = slices(t);
            if (nkb == 0) continue;
            stage = (stage + nkb - 1) % W_STAGES;
            if (has_tail(t)) {
                if (!whole_warp(wait_phase(&tail[stage], tails.take(stage), s_abort, p.dev_status))) break;
                zero_rows(smem + stage * W_STAGE, W_STAGE / (64 * 128), t.row_end - t.row0 - (nkb - 1) * BK, lane);
                if (lane == 0) mbar_arrive_cluster(lead_full + 8u * static_cast<uint32_t>(stage));
            }
            if (++stage == W_STAGES) stage = 0;
        }
    } else if (warp == 1) {
        // ================= MMA issuer (even CTA only)
        if (leader && elect_one()) {
            int stage = 0, g = 0;
            uint32_t phase = 0, tph = 0;
            const uint32_t base = smem_u32(smem) >> 4;
            bool issued = false;
            for (int tile = first_tile; tile < total && !*s_abort; tile += step) {
                const Tile t = decode_tile<DW, BW>(p, tile, g, s_off, nullptr);
                const int nkb = slices(t);
                // the 16-row steps of the last slice that hold rows of the group
                const int last = (t.row_end - t.row0 - (nkb - 1) * BK + 15) / 16;
                // half h of slice kb, staged in st
                auto mma_half = [&](int st, int kb, int h) {
                    const uint32_t at = base + static_cast<uint32_t>(st) * (W_STAGE / 16);
                    const uint32_t a = at + MN_LO;
                    const uint32_t b = a + (1 + static_cast<uint32_t>(h)) * (SLICE / 16);
                    const int steps = kb + 1 < nkb ? 4 : last;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        mma(tmem + 256u * static_cast<uint32_t>(h), a + k * 128, b + k * 128, C::IDESC,
                               (kb | k) != 0 ? 1u : 0u);
                    }
                };
                if (!wait_phase(&tempty[0], tph ^ 1, s_abort, p.dev_status)) break;
                tc_fence_after();
                bool h1 = false, ok = true;              // half 1 is free
                int pend[W_STAGES], npend = 0, pend_kb = 0;
                auto flush = [&]() {
                    for (int i = 0; i < npend; ++i) {
                        mma_half(pend[i], pend_kb + i, 1);
                        tc_commit_pair_mc(&empty[pend[i]], 0x3);
                    }
                    npend = 0;
                };
                auto wait_h1 = [&]() {
                    if (!h1) {
                        h1 = wait_phase(&tempty[1], tph ^ 1, s_abort, p.dev_status);
                        tc_fence_after();
                    }
                    return h1;
                };
                for (int kb = 0; kb < nkb; ++kb) {
                    const bool zeroed = kb + 1 == nkb && has_tail(t);
                    if (zeroed ? !wait_zeroed(&full[stage], phase, s_abort, p.dev_status)
                               : !wait_phase(&full[stage], phase, s_abort, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    if (zeroed) fence_proxy_async();
                    tc_fence_after();
                    mma_half(stage, kb, 0);
                    issued = true;
                    const bool tail = kb >= nkb - W_TAIL;
                    if (!tail && !h1 && mbar_test_wait_cluster(&tempty[1], tph ^ 1)) {
                        tc_fence_after();
                        h1 = true;
                    }
                    if (h1 && !tail) {
                        flush();
                        mma_half(stage, kb, 1);
                        tc_commit_pair_mc(&empty[stage], 0x3);
                    } else {
                        if (npend == 0) pend_kb = kb;
                        pend[npend++] = stage;
                        if (npend == W_STAGES) {         // every stage waits for half 1
                            if (!wait_h1()) {
                                ok = false;
                                break;
                            }
                            flush();
                        }
                    }
                    if (++stage == W_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair_mc(&tfull[0], 0x3);
                if (!wait_h1()) break;
                flush();
                tc_commit_pair_mc(&tfull[1], 0x3);
                tph ^= 1;
            }
            if (*s_abort && issued) {
                // unwinding: every MMA issued so far ends before TMEM is freed
                tc_commit_pair_mc(drain, 0x1);
                mbar_wait_drain(drain, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ================= epilogue: two warps share a TMEM lane quarter
        const int quarter = warp & 3, part = (warp - 4) >> 2;
        const Box box{smem + C::EPI_OFF + (warp - 4) * EPI_BYTES, lane};
        int g = 0;
        uint32_t tph = 0;
        for (int tile = first_tile; tile < total; tile += step) {
            const Tile t = decode_tile<DW, BW>(p, tile, g, s_off, nullptr);
            const int row0 = t.m0 + 128 * rank + 32 * quarter;
            const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            bool stop = false;
            for (int h = 0; h < 2; ++h) {
                if (!whole_warp(wait_phase(&tfull[h], tph, s_abort, p.dev_status))) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tq + 256u * static_cast<uint32_t>(h) + 128u * static_cast<uint32_t>(part);
#pragma unroll 1
                for (int c = 0; c < 128; c += 64)
                    if (!emit_gradient(p, box, t, acc + c, row0, t.n0 + 128 * h + 256 * part + c)) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_drained(lead_tempty + 8u * static_cast<uint32_t>(h));
            }
            if (stop) break;
            tph ^= 1;
        }
        if (lane == 0) bulk_wait<0>();       // every output box written
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                  // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    __syncwarp();
    cluster_sync_all();                  // nor before both have given their tensor memory back
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

// bf16 [groups][rows][cols] as boxes of 64 columns x box_rows rows, 128-byte
// swizzle: K-major operands (columns are K) and MN-major ones (rows are K).
bool operand_map(CUtensorMap *m, const void *ptr, int groups, int64_t rows, int64_t cols,
                 int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dim[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                         static_cast<cuuint64_t>(std::max(groups, 1))};
    cuuint64_t stride[2] = {dim[0] * 2, dim[0] * dim[1] * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups > 0 ? 3 : 2, const_cast<void *>(ptr), dim,
              stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output [groups][rows][cols] (and h) as boxes of 32 rows x 64 bytes, swizzled over as many.
bool out_map(CUtensorMap *m, void *ptr, int groups, int64_t rows, int64_t cols, bool f32) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dim[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                         static_cast<cuuint64_t>(std::max(groups, 1))};
    cuuint64_t stride[2] = {dim[0] * esz, dim[0] * dim[1] * esz};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(64 / esz), 32, 1}, es[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              groups > 0 ? 3 : 2, ptr, dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// DW in wide tiles: with few rows a group, where the gradients' stores decide and
// fewer hand-overs help, and with very many.  Measured with H = 2048, I = 1024 and 64
// groups (whole backward pass, us, 256 against 512 columns): 16 rows a group 296 : 280,
// 64 330 : 295, 128 373 : 360, 256 450 : 456, 512 683 : 713, 1024 1210 : 1245, 2048
// 2252 : 2278; 16384 rows of H = 4096, I = 2048: one group 1030 : 1006, two 1028 : 1022.
// The rule takes the mean over all groups, which the host knows; the figures are of groups
// that all have rows.  A few large ones among many idle get the tiles of few rows.
bool wide_gradient(int n, int G) { return n < 192ll * G || n >= 8192ll * G; }

template <int MODE, bool WIDE = false>
cudaError_t launch(const Params &p, int64_t tiles, cudaStream_t stream) {
    void (*kernel)(const Params) = train_gemm_kernel<MODE>;
    if (WIDE) kernel = gradient_wide_kernel;                 // DW only
    static std::mutex mu;
    static int resident[64] = {};        // pairs that can run at once, by device
    int dev = 0;
    cudaGetDevice(&dev);
    int limit = num_sms() / 2;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || resident[dev] == 0) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms()), 1, 1);
            cfg.blockDim = dim3(THREADS, 1, 1);
            cfg.dynamicSmemBytes = 227 * 1024;
            cfg.stream = stream;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
                cudaGetLastError();
                n = limit;
            }
            limit = std::min(n, limit);
            if (dev < 64) resident[dev] = limit;
        } else {
            limit = resident[dev];
        }
    }
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(limit, tiles));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * units), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(Cfg<MODE>::smem(p.G));
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// All but DW: A [n, K], B as the mode's weights.
template <int MODE>
cudaError_t launch_rows(Params &p, const void *a, const void *w, cudaStream_t stream) {
    constexpr bool K_MAJOR = MODE == FWD || MODE == DOWN;                           // the weights
    const int64_t brows = MODE == FWD ? 2 * static_cast<int64_t>(p.N) : K_MAJOR ? p.N : p.K;
    const int bcols = K_MAJOR ? p.K : p.N;
    // rows of B's box: 128 weight rows, or a stage's K
    const int box = K_MAJOR ? 128 : 64 * Cfg<MODE>::KSUB;
    if (!operand_map(&p.tmA, a, 0, p.n, p.K, 128) || !operand_map(&p.tmB, w, p.G, brows, bcols, box) ||
        !operand_map(&p.tmAh, a, 0, p.n, p.K, 64) ||
        (MODE == FWD && !operand_map(&p.tmBh, w, p.G, brows, bcols, 64)))
        return cudaErrorInvalidValue;
    p.nt = static_cast<int>(ceil_div(p.N, MODE == FWD ? 128 : 256));
    const int64_t tiles = (static_cast<int64_t>(p.n / BM) + std::min(p.G, p.n)) * p.nt;
    return launch<MODE>(p, tiles, stream);
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct BwdWs {
    size_t d_h, act, total;
};
BwdWs bwd_layout(int n, int I) {
    BwdWs w;
    auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    w.d_h = 0;
    w.act = up(static_cast<size_t>(n) * 2 * I * 2);
    w.total = w.act + up(static_cast<size_t>(n) * I * 2);
    return w;
}

moe_status_t check_sizes(int32_t G, int32_t n, int32_t H, int32_t I) {
    if (G <= 0 || n < 0 || H <= 0 || I <= 0) return MOE_ERR_INVALID_ARG;
    if (G > MAX_GROUPS || H % 128 != 0 || I % 128 != 0 || H > (1 << 20) || I > (1 << 19) ||
        n > INT32_MAX - 1024)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    // tile numbers are 32-bit
    const int64_t w = std::max(2 * static_cast<int64_t>(I), static_cast<int64_t>(H)) / 128;
    const int64_t row_tiles = (n / 128 + static_cast<int64_t>(G)) * w;
    const int64_t w_tiles = static_cast<int64_t>(G) * 2 * ceil_div(2 * static_cast<int64_t>(I), 256) *
                            ceil_div(H, 256);
    if (row_tiles >= (int64_t{1} << 31) || w_tiles >= (int64_t{1} << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

#define TRY_CUDA(x)                                     \
    do {                                                \
        if ((x) != cudaSuccess) return MOE_ERR_CUDA;    \
    } while (0)

extern "C" moe_status_t moe_grouped_mlp_train(const moe_bf16_t *expanded_x, const int32_t *offsets,
                                              int32_t G, const moe_bf16_t *w13, const moe_bf16_t *w2,
                                              int32_t n, int32_t H, int32_t I, moe_bf16_t *h,
                                              moe_bf16_t *act, moe_bf16_t *y, int32_t *dev_status,
                                              moe_stream_t stream) {
    const moe_status_t st = check_sizes(G, n, H, I);
    if (st != MOE_OK) return st;
    if (!offsets || !w13 || !w2) return MOE_ERR_INVALID_ARG;
    if (n == 0) return MOE_OK;
    if (!expanded_x || !h || !act || !y) return MOE_ERR_INVALID_ARG;
    if (!a16(expanded_x) || !a16(w13) || !a16(w2) || !a16(h) || !a16(act) || !a16(y))
        return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    if (!encode_fn()) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Params p{};
    if (!out_map(&p.tmO0, h, 0, n, 2 * static_cast<int64_t>(I), false) ||
        !out_map(&p.tmO1, act, 0, n, I, false))
        return MOE_ERR_CUDA;
    p.offsets = offsets;
    p.G = G;
    p.n = n;
    p.K = H;
    p.N = I;
    p.wrows = 2 * I;
    p.out0 = h;
    p.ld0 = 2 * I;
    p.out1 = act;
    p.ld1 = I;
    p.dev_status = dev_status;
    TRY_CUDA(launch_rows<FWD>(p, expanded_x, w13, s));
    if (!out_map(&p.tmO0, y, 0, n, H, false)) return MOE_ERR_CUDA;
    p.K = I;
    p.N = H;
    p.wrows = H;
    p.out0 = y;
    p.ld0 = H;
    TRY_CUDA(launch_rows<DOWN>(p, act, w2, s));
    return MOE_OK;
}

extern "C" moe_status_t moe_grouped_mlp_backward_workspace_size(int32_t n, int32_t I, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_sizes(1, n, 128, I);
    if (st != MOE_OK) return st;
    *bytes = bwd_layout(n, I).total;
    return MOE_OK;
}

extern "C" moe_status_t moe_grouped_mlp_backward(
    const moe_bf16_t *d_y, const moe_bf16_t *expanded_x, const int32_t *offsets, int32_t G,
    const moe_bf16_t *h, const moe_bf16_t *w13, const moe_bf16_t *w2, int32_t n, int32_t H,
    int32_t I, uint32_t flags, moe_bf16_t *d_x, void *d_w13, void *d_w2, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, moe_stream_t stream) {
    const moe_status_t st = check_sizes(G, n, H, I);
    if (st != MOE_OK) return st;
    const bool f32 = (flags & MOE_DW_F32) != 0, add = (flags & MOE_DW_ACCUMULATE) != 0;
    if (add && !f32) return MOE_ERR_INVALID_ARG;
    if (!offsets || !w13 || !w2) return MOE_ERR_INVALID_ARG;
    if ((d_x && !a16(d_x)) || (d_w13 && !a16(d_w13)) || (d_w2 && !a16(d_w2)))
        return MOE_ERR_INVALID_ARG;
    if (!d_x && !d_w13 && !d_w2) return MOE_OK;
    if (n > 0) {
        if (!d_y || !expanded_x || !h) return MOE_ERR_INVALID_ARG;
        if (!a16(d_y) || !a16(expanded_x) || !a16(h) || !a16(w13) || !a16(w2))
            return MOE_ERR_INVALID_ARG;
        if (!workspace || workspace_bytes < bwd_layout(n, I).total ||
            (reinterpret_cast<uintptr_t>(workspace) & 255))
            return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t I2 = 2 * static_cast<int64_t>(I);
    if (n == 0) {
        const size_t bytes = static_cast<size_t>(G) * I * H * (f32 ? 4 : 2);
        if (!add && d_w13) TRY_CUDA(cudaMemsetAsync(d_w13, 0, 2 * bytes, s));
        if (!add && d_w2) TRY_CUDA(cudaMemsetAsync(d_w2, 0, bytes, s));
        return MOE_OK;
    }
    if (!encode_fn()) return MOE_ERR_CUDA;
    const BwdWs L = bwd_layout(n, I);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *d_h = reinterpret_cast<uint16_t *>(ws + L.d_h);
    uint16_t *act = reinterpret_cast<uint16_t *>(ws + L.act);
    Params p{};
    p.offsets = offsets;
    p.G = G;
    p.n = n;
    p.dev_status = dev_status;
    // d_act and what follows from it
    if (!out_map(&p.tmO0, d_h, 0, n, I2, false) || !out_map(&p.tmO1, act, 0, n, I, false) ||
        !out_map(&p.tmH, const_cast<uint16_t *>(h), 0, n, I2, false) ||
        !operand_map(&p.tmG[0], d_h, 0, n, I2, 64) ||
        !operand_map(&p.tmG[1], expanded_x, 0, n, H, 64) ||
        !operand_map(&p.tmG[2], d_y, 0, n, H, 64) || !operand_map(&p.tmG[3], act, 0, n, I, 64))
        return MOE_ERR_CUDA;
    p.K = H;
    p.N = I;
    p.wrows = I;
    p.out0 = d_h;
    p.ld0 = 2 * I;
    p.out1 = act;
    p.ld1 = I;
    TRY_CUDA(launch_rows<DACT>(p, d_y, w2, s));
    if (d_x) {
        if (!out_map(&p.tmO0, d_x, 0, n, H, false)) return MOE_ERR_CUDA;
        p.K = 2 * I;
        p.N = H;
        p.wrows = H;
        p.out0 = d_x;
        p.ld0 = H;
        TRY_CUDA(launch_rows<DX>(p, d_h, w13, s));
    }
    if (d_w13 || d_w2) {
        if ((d_w13 && !out_map(&p.tmO0, d_w13, G, I2, H, f32)) ||
            (d_w2 && !out_map(&p.tmO1, d_w2, G, H, I, f32)))
            return MOE_ERR_CUDA;
        p.mt0 = d_w13 ? static_cast<int>(ceil_div(I2, 256)) : 0;
        const int bn = wide_gradient(n, G) ? BW : BN;
        p.nt0 = d_w13 ? static_cast<int>(ceil_div(H, bn)) : 0;
        p.mt1 = d_w2 ? static_cast<int>(ceil_div(H, 256)) : 0;
        p.nt1 = d_w2 ? static_cast<int>(ceil_div(I, bn)) : 0;
        p.H = H;
        p.I = I;
        p.w_f32 = f32;
        p.accumulate = add;
        const int64_t tiles =
            static_cast<int64_t>(G) * (p.mt0 * p.nt0 + static_cast<int64_t>(p.mt1) * p.nt1);
        TRY_CUDA((bn == BW ? launch<DW, true>(p, tiles, s) : launch<DW>(p, tiles, s)));
    }
    return MOE_OK;
}
