// fp4_weight.cu -- bf16 rows times 4-bit weights, for the few rows per expert
// of a decoding step.
//
//   STORE:   y[r, n] = x[r] . W[g, n]
//   SWIGLU:  act[r, n] = SiLU(x[r] . W[g, n]) (x[r] . W[g, I + n])
// for the rows r of group g, W[g, n, k] = e2m1 code * block scale.
//
// What bounds it is reading the weights: K (1/2 + 1/block) bytes a weight row,
// each used for a handful of rows.  So the weights stream through shared memory
// in 16-byte asynchronous copies (two CTAs a multiprocessor, 3 or 4 stages of 128
// rows x 256 columns each), and what is done with them has to fit beside: at
// full bandwidth a multiprocessor has about three issue slots a weight.
//
// The arithmetic.  The weights are the 16-row operand of mma.sync m16n8k16, the
// rows the 8-column one, so one instruction multiplies 256 weights with up to 8
// rows.  In f16 a pair of codes takes one conversion (cvt.f16x2.e2m1x2, exact;
// there is none to bf16, and picking the bits apart takes 4 to 5 instructions a
// pair).  So the rows go to f16, too, after a scaling by a power of two that puts
// a row's largest finite magnitude into [2^15, 2^16): a bf16 value fits f16's 11
// bits and is exact down to 2^-30 of that maximum; below it is rounded by at
// most 2^-40 of the maximum.  The scaling comes off the fp32 sums at the end.
//   MX: the sum over a block of 32 columns is made apart and added to the fp32
//       total times the block's power of two.
//   NV: code * e4m3 scale has at most 6 significant bits and lies within
//       [2^-10, 2688], exact in f16, so the scale goes onto the weight and the
//       MMAs accumulate throughout (post-scaling would cost 4 FMAs per 16 columns).
// Lane (g, t) of an MMA takes, of each 32 columns, columns 8t .. 8t + 7 of its
// rows: 4 bytes of codes and 16 bytes of a token, in an order of K of its own
// that both operands share.
//
// A cluster of CTAs may share a tile along K (few tiles, long K); their sums meet
// through distributed shared memory in a fixed order.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "internal.h"

namespace moe {

moe_status_t fp4_check(int format, int scale_exp);

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int THREADS = 256;
constexpr int ROWS = 128;                    // weight rows of a tile
constexpr int KC = 256;                      // columns of a stage
constexpr int W_BYTES = ROWS * KC / 2;
constexpr int P_LD = ROWS + 4;               // row stride of the partial sums, in floats

struct Params {
    const uint8_t *q, *sf;
    const uint16_t *xh;                      // f16 rows [n, K]
    const float *xscale;                     // what takes their scaling off again
    const int32_t *offsets;
    int32_t G, n, K, N;                      // N: output columns
    int32_t wrows;                           // rows of a group's weights
    int32_t split;                           // CTAs that share a tile along K
    float alpha;                             // 2^scale_exp
    void *out;
    int32_t out_f32;
    int32_t *dev_status;
};

template <int FMT, bool SWIGLU, int MAXT>
struct Cfg {
    static constexpr int STAGES = MAXT == 8 ? 4 : 3;
    static constexpr int KTILES = KC / Fp4<FMT>::TILE_K;              // scale tiles along K
    static constexpr int S_TILES = KTILES * (SWIGLU ? 2 : 1);
    static constexpr int S_BYTES = S_TILES * kScaleTile;
    static constexpr int X_BYTES = MAXT * KC * 2;
    static constexpr int STAGE = W_BYTES + S_BYTES + X_BYTES;
    static constexpr int P_OFF = STAGES * STAGE;
    static constexpr int P_BYTES = MAXT * P_LD * 4;                   // one of two buffers
    static constexpr int OFFS_OFF = P_OFF + 2 * P_BYTES;
    static constexpr int smem(int G) { return OFFS_OFF + (2 * G + 3) * 4; }
    // two CTAs a multiprocessor, 1 KB of each taken by the system
    static_assert(2 * (smem(MAX_GROUPS) + 1024) <= 228 * 1024, "shared memory");
};

// 16 bytes, or zeros.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(read ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes to four pairs of f16 values.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Byte `i` of w as an e4m3 value, twice.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t w, uint32_t i) {
    uint32_t r;
    const uint16_t b = static_cast<uint16_t>(__byte_perm(w, 0, i * 0x11u));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
    return r;
}
// Four scale bytes 2^(b - 127) as fp32 (255: NaN).
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&s)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xFFFF0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xFFFF0000u);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Rows to f16 under a power of two of their own; one CTA per row.
constexpr int PREP_THREADS = 256;
__global__ void __launch_bounds__(PREP_THREADS)
    prep_kernel(const uint16_t *__restrict__ x, int K, uint16_t *__restrict__ xh,
                float *__restrict__ xscale) {
    __shared__ uint32_t s_max[PREP_THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // from here on everything before this call has ended: the products may start
    // on the weights and the offsets, and wait for the rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t base = static_cast<int64_t>(blockIdx.x) * K;
    const uint4 *row = reinterpret_cast<const uint4 *>(x + base);
    const int nv = K / 8;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < nv; i += PREP_THREADS) {
        const uint4 v = row[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = w[j] & 0x7FFFu, b = (w[j] >> 16) & 0x7FFFu;
            if (a < 0x7F80u) m = max(m, a);
            if (b < 0x7F80u) m = max(m, b);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PREP_THREADS / 32; ++i) m = max(m, s_max[i]);
    // 2^(142 - e) of the maximum's exponent field e, at most 2^127
    const int e = max(static_cast<int>(m >> 7), 15);
    const float up = pow2f(142 - e);
    if (threadIdx.x == 0)   // 2^(e - 142), which may be subnormal
        xscale[blockIdx.x] = e >= 16 ? pow2f(e - 142) : __uint_as_float(1u << 22);
    uint4 *dst = reinterpret_cast<uint4 *>(xh + base);
    for (int i = threadIdx.x; i < nv; i += PREP_THREADS) {
        const uint4 v = row[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * up,
                                                __uint_as_float(w[j] & 0xFFFF0000u) * up);
            o[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

struct Item {
    int g, tok0, cnt, n0;      // group, first row and number of rows, first output column
};

template <int FMT, bool SWIGLU, int MAXT>
__global__ void __launch_bounds__(THREADS, 2) weight_kernel(const Params p) {
    using C = Cfg<FMT, SWIGLU, MAXT>;
    constexpr int STAGES = C::STAGES, NT = MAXT / 8, OUT = SWIGLU ? ROWS / 2 : ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    int *s_off = reinterpret_cast<int *>(smem + C::OFFS_OFF);
    int *s_prefix = s_off + p.G + 1;
    int *s_bad = s_prefix + p.G + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(blockIdx.x) % p.split;
    const int unit = static_cast<int>(blockIdx.x) / p.split;
    const int units = static_cast<int>(gridDim.x) / p.split;
    const int rtiles = p.N / OUT;

    // items of the groups before each
    for (int g = tid; g <= p.G; g += THREADS) s_off[g] = p.offsets[g];
    if (tid == 0) *s_bad = 0;
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        bool bad = false;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int items = 0;
            if (g < p.G) {
                const int a = s_off[g], b = s_off[g + 1];
                if (a < 0 || b < a || b > p.n) bad = true;
                items = b > a ? ((b - a + MAXT - 1) / MAXT) * rtiles : 0;
            }
            int inc = items;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += o;
            }
            if (g < p.G) s_prefix[g] = run + inc - items;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) s_prefix[p.G] = run;
        if (__any_sync(0xffffffffu, bad) && lane == 0) *s_bad = 1;
    }
    __syncthreads();
    if (*s_bad && tid == 0 && blockIdx.x == 0) report(p.dev_status, MOE_DEV_BAD_OFFSETS);
    const int total = *s_bad ? 0 : s_prefix[p.G];

    auto decode = [&](int item, int &g) {
        while (s_prefix[g + 1] <= item) ++g;
        const int start = s_off[g], cnt = s_off[g + 1] - start;
        const int local = item - s_prefix[g];
        const int chunks = (cnt + MAXT - 1) / MAXT;      // next to each other: they share weights
        const int tile = local / chunks, c = local - tile * chunks;
        return Item{g, start + c * MAXT, min(MAXT, cnt - c * MAXT), tile * OUT};
    };
    const int stages_k = (p.K + KC - 1) / KC;
    const int k_begin = rank * stages_k / p.split, k_end = (rank + 1) * stages_k / p.split;
    const int64_t ktiles = p.K / Fp4<FMT>::TILE_K;       // scale tiles along K

    // The copies run ahead of the products by STAGES - 1 stages, across items.
    int ld_item = unit, ld_k = k_begin, ld_slot = 0, ld_g = 0;
    Item ld{};
    if (ld_item < total) ld = decode(ld_item, ld_g);
    auto copy_weights = [&](int slot, const Item &it, int ks) {
        uint8_t *w = smem + slot * C::STAGE, *s = w + W_BYTES;
        const int64_t half = p.K / 2;
        // row r's 16-byte piece c lies at c ^ (r & 7)
#pragma unroll
        for (int i = 0; i < W_BYTES / 16 / THREADS; ++i) {
            const int e = i * THREADS + tid, r = e >> 3, c = e & 7;
            const int64_t wr = static_cast<int64_t>(it.g) * p.wrows + it.n0 +
                               (SWIGLU && r >= 64 ? p.N + r - 64 : r);
            const int col = ks * (KC / 2) + c * 16;
            const bool in = col < half;
            copy16(w + r * (KC / 2) + ((c ^ (r & 7)) << 4), p.q + wr * half + (in ? col : 0), in);
        }
        for (int e = tid; e < C::S_BYTES / 16; e += THREADS) {
            const int t = e >> 5, c = e & 31;            // scale tile, 16-byte piece
            const int part = t / C::KTILES, kt = ks * C::KTILES + t % C::KTILES;
            const int64_t blk = (static_cast<int64_t>(it.g) * p.wrows + it.n0 +
                                 (part ? p.N : 0)) / 128;
            const bool in = kt < ktiles;
            copy16(s + t * kScaleTile + c * 16,
                   p.sf + (blk * ktiles + (in ? kt : 0)) * kScaleTile + c * 16, in);
        }
    };
    auto copy_rows = [&](int slot, const Item &it, int ks) {
        uint8_t *x = smem + slot * C::STAGE + W_BYTES + C::S_BYTES;
        // token j's 16-byte piece c lies at c ^ (4 (j & 1))
#pragma unroll
        for (int i = 0; i < C::X_BYTES / 16 / THREADS; ++i) {
            const int e = i * THREADS + tid, j = e >> 5, c = e & 31;
            const int col = ks * KC + c * 8;
            const bool in = j < it.cnt && col < p.K;
            copy16(x + j * (KC * 2) + ((c ^ ((j & 1) << 2)) << 4),
                   p.xh + (in ? static_cast<int64_t>(it.tok0 + j) * p.K + col : 0), in);
        }
    };
    auto advance = [&]() {
        if (++ld_slot == STAGES) ld_slot = 0;
        if (++ld_k == k_end) {
            ld_k = k_begin;
            ld_item += units;
            if (ld_item < total) ld = decode(ld_item, ld_g);
        }
    };
    {
        // weights first: they do not wait for the rows' conversion
        const int item0 = ld_item, k0 = ld_k, g0 = ld_g;
        const Item it0 = ld;
        for (int s = 0; s < STAGES - 1; ++s) {
            if (ld_item < total) copy_weights(s, ld, ld_k);
            advance();
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        ld_item = item0;
        ld_k = k0;
        ld_g = g0;
        ld = it0;
        ld_slot = 0;
        for (int s = 0; s < STAGES - 1; ++s) {
            if (ld_item < total) copy_rows(s, ld, ld_k);
            copy_commit();
            advance();
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int wr = (warp & 3) * 32, khalf = warp >> 2;   // this warp's rows, and its half of a stage
    const int g8 = lane >> 2, t4 = lane & 3;
    int slot = 0, g = 0, parity = 0;
    for (int item = unit; item < total; item += units) {
        const Item it = decode(item, g);
        const int nt = (it.cnt + 7) >> 3;
        // where this warp's rows have their scales: tile part and row in it
        const int s_part = SWIGLU && wr >= 64 ? 1 : 0;
        const int s_row = (SWIGLU ? it.n0 & 64 : 0) + (SWIGLU ? wr & 63 : wr);
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
        for (int ks = k_begin; ks < k_end; ++ks) {
            copy_wait<STAGES - 2>();
            __syncthreads();
            if (ld_item < total) {
                copy_weights(ld_slot, ld, ld_k);
                copy_rows(ld_slot, ld, ld_k);
            }
            copy_commit();
            advance();
            const uint8_t *w = smem + slot * C::STAGE;
            const uint8_t *s = w + W_BYTES + s_part * C::KTILES * kScaleTile;
            const uint8_t *x = w + W_BYTES + C::S_BYTES;
            if (++slot == STAGES) slot = 0;
            // scales of rows g8 and g8 + 8 of both 16-row parts
            uint32_t sw[2][2][C::KTILES / 2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < C::KTILES / 2; ++k)
                        sw[m][h][k] = *reinterpret_cast<const uint32_t *>(
                            s + (khalf * (C::KTILES / 2) + k) * kScaleTile +
                            scale_row_offset(s_row + 16 * m + 8 * h + g8)) &
                            (FMT == MOE_FP4_NV ? 0x7F7F7F7Fu : 0xFFFFFFFFu);
            float sc[2][2][4];
            if (FMT == MOE_FP4_MX) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) e8m0x4(sw[m][h][0], sc[m][h]);
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {                 // 32 columns at a time
                const int kb = khalf * 4 + b;
                uint4 xb[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt)
                        xb[j] = *reinterpret_cast<const uint4 *>(
                            x + (8 * j + g8) * (KC * 2) +
                            (((kb * 4 + t4) ^ ((g8 & 1) << 2)) << 4));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = wr + 16 * m + 8 * h + g8;
                        decode8(*reinterpret_cast<const uint32_t *>(
                                    w + r * (KC / 2) + ((kb ^ (r & 7)) << 4) + t4 * 4),
                                a[h]);
                        if (FMT == MOE_FP4_NV) {
                            // blocks 2b and 2b + 1: this lane's bytes lie in one of them
                            const uint32_t f = e4m3_f16x2(sw[m][h][b / 2],
                                                          (2 * b & 3) + (t4 >> 1));
#pragma unroll
                            for (int i = 0; i < 4; ++i) a[h][i] = mul_f16x2(a[h][i], f);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (j >= nt) break;
                        if (FMT == MOE_FP4_NV) {
                            mma16816(acc[m][j], a[0][0], a[1][0], a[0][1], a[1][1], xb[j].x, xb[j].y);
                            mma16816(acc[m][j], a[0][2], a[1][2], a[0][3], a[1][3], xb[j].z, xb[j].w);
                        } else {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(d, a[0][0], a[1][0], a[0][1], a[1][1], xb[j].x, xb[j].y);
                            mma16816(d, a[0][2], a[1][2], a[0][3], a[1][3], xb[j].z, xb[j].w);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[m][j][i] = fmaf(d[i], sc[m][i >> 1][b], acc[m][j][i]);
                        }
                    }
                }
            }
        }
        // The halves of the stages are added, then the CTAs' sums: [token][row].
        float *P = reinterpret_cast<float *>(smem + C::P_OFF + parity * C::P_BYTES);
        auto at = [&](int m, int j, int i) -> float & {
            return P[(8 * j + 2 * t4 + (i & 1)) * P_LD + wr + 16 * m + g8 + 8 * (i >> 1)];
        };
        if (khalf == 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) at(m, j, i) = acc[m][j][i];
        }
        __syncthreads();
        if (khalf == 0) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) at(m, j, i) += acc[m][j][i];
        }
        if (p.split > 1)
            cluster_sync_all();      // two buffers: the next but one item's sync is behind every read
        else
            __syncthreads();
        const uint32_t mine = smem_u32(P);
        auto sum = [&](int tok, int row) {
            const uint32_t off = static_cast<uint32_t>(tok * P_LD + row) * 4;
            if (p.split == 1) return P[tok * P_LD + row];
            float v = 0.0f;
            for (int c = 0; c < p.split; ++c)
                v += ld_cluster_f32(mapa_shared(mine, static_cast<uint32_t>(c)) + off);
            return v;
        };
        for (int e = rank * THREADS + tid; e < it.cnt * OUT; e += p.split * THREADS) {
            const int tok = e / OUT, row = e % OUT;
            const float f = __ldg(p.xscale + it.tok0 + tok);
            float v = sum(tok, row) * f * p.alpha;
            if (SWIGLU) {
                const float u = sum(tok, 64 + row) * f * p.alpha;
                v = __fdividef(v, 1.0f + __expf(-v)) * u;
            }
            const int64_t o = static_cast<int64_t>(it.tok0 + tok) * p.N + it.n0 + row;
            if (p.out_f32)
                static_cast<float *>(p.out)[o] = v;
            else
                static_cast<uint16_t *>(p.out)[o] = float_to_bf16_bits(v);
        }
        parity ^= 1;
    }
    copy_wait<0>();
    if (p.split > 1) cluster_sync_all();     // no CTA leaves while its sums may be read
}

// ------------------------------------------------------------------ host side
template <int FMT, bool SWIGLU, int MAXT>
cudaError_t launch(Params &p, cudaStream_t stream) {
    using C = Cfg<FMT, SWIGLU, MAXT>;
    auto kernel = weight_kernel<FMT, SWIGLU, MAXT>;
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
    // As many groups as may have rows decide how far a tile is split along K: the
    // split with the least time on the fullest multiprocessor.
    const int slots = 2 * num_sms();
    const int64_t groups = std::min(p.n, p.G);
    const int64_t chunks = std::max<int64_t>(groups, ceil_div(p.n, MAXT));
    const int64_t tiles = chunks * (p.N / (SWIGLU ? ROWS / 2 : ROWS));
    const int stages_k = static_cast<int>(ceil_div(p.K, KC));
    double best = 1e30;
    p.split = 1;
    for (int s = 1; s <= 8 && s <= stages_k; s *= 2) {
        const int64_t rounds = ceil_div(tiles, slots / s);
        // a tile's own time in stages: its share of K, and 1 for the join
        const double t = static_cast<double>(rounds) * (static_cast<double>(ceil_div(stages_k, s)) + (s > 1 ? 1.0 : 0.5));
        if (t < best) {
            best = t;
            p.split = s;
        }
    }
    const int64_t units = std::max<int64_t>(1, std::min<int64_t>(slots / p.split, tiles));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * p.split), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(C::smem(p.G));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int FMT, bool SWIGLU>
cudaError_t launch_rows(Params &p, cudaStream_t stream) {
    // rows per pass over a group's weights: a group with more reads them again
    // (from L2, its passes run side by side)
    return p.n <= std::max(8, 2 * p.G) ? launch<FMT, SWIGLU, 8>(p, stream)
                                       : launch<FMT, SWIGLU, 16>(p, stream);
}

cudaError_t launch_prep(const uint16_t *x, int n, int K, uint16_t *xh, float *xscale,
                        cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n), 1, 1);
    cfg.blockDim = dim3(PREP_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prep_kernel, x, K, xh, xscale);
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t workspace_bytes_of(int n, int K) {
    return ((static_cast<size_t>(n) * K * 2 + 255) & ~static_cast<size_t>(255)) +
           static_cast<size_t>(n) * 4;
}

struct Product {
    const moe_bf16_t *x;
    const int32_t *offsets;
    int G;
    const moe_fp4_t *w;
    int n, K, N;
    bool swiglu;
};

moe_status_t check(const Product &d) {
    if (!d.w || d.G <= 0 || d.n < 0 || d.K <= 0 || d.N <= 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = fp4_check(d.w->format, d.w->scale_exp);
    if (st != MOE_OK) return st;
    if (d.G > MAX_GROUPS || d.K % 128 != 0 || d.N % 128 != 0 || d.K > (1 << 20) || d.N > (1 << 24) ||
        (static_cast<int64_t>(d.n) / 8 + d.G) * (d.N / 64) >= (int64_t{1} << 30))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!d.offsets || !d.w->q || !d.w->sf || !a16(d.w->q) || !a16(d.w->sf))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t run(const Product &d, uint32_t flags, void *out, void *workspace, int32_t *dev_status,
                 cudaStream_t s) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint16_t *xh = reinterpret_cast<uint16_t *>(ws);
    float *xscale = reinterpret_cast<float *>(
        ws + ((static_cast<size_t>(d.n) * d.K * 2 + 255) & ~static_cast<size_t>(255)));
    if (launch_prep(d.x, d.n, d.K, xh, xscale, s) != cudaSuccess) return MOE_ERR_CUDA;
    Params p{};
    p.q = d.w->q;
    p.sf = d.w->sf;
    p.xh = xh;
    p.xscale = xscale;
    p.offsets = d.offsets;
    p.G = d.G;
    p.n = d.n;
    p.K = d.K;
    p.N = d.N;
    p.wrows = d.swiglu ? 2 * d.N : d.N;
    p.alpha = pow2f(d.w->scale_exp);
    p.out = out;
    p.out_f32 = (flags & MOE_Y_F32) != 0;
    p.dev_status = dev_status;
    const bool mx = d.w->format == MOE_FP4_MX;
    cudaError_t e;
    if (d.swiglu)
        e = mx ? launch_rows<MOE_FP4_MX, true>(p, s) : launch_rows<MOE_FP4_NV, true>(p, s);
    else
        e = mx ? launch_rows<MOE_FP4_MX, false>(p, s) : launch_rows<MOE_FP4_NV, false>(p, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool bad_workspace(void *ws, size_t have, size_t need) {
    return !ws || have < need || (reinterpret_cast<uintptr_t>(ws) & 255);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_weight_workspace_size(int32_t n, int32_t K, size_t *bytes) {
    if (!bytes || n < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > (1 << 20)) return MOE_ERR_UNSUPPORTED_SHAPE;
    *bytes = workspace_bytes_of(n, K);
    return MOE_OK;
}

static moe_status_t product(const Product &d, uint32_t flags, void *out, void *workspace,
                            size_t workspace_bytes, int32_t *dev_status, moe_stream_t stream) {
    const moe_status_t st = check(d);
    if (st != MOE_OK) return st;
    if (d.n == 0) return MOE_OK;
    if (!d.x || !a16(d.x) || !out || !a16(out)) return MOE_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes, workspace_bytes_of(d.n, d.K)))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
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
    return product(Product{x, offsets, G, w13, n, K, I, true}, flags, act, workspace,
                   workspace_bytes, dev_status, stream);
}

extern "C" moe_status_t moe_fp4_weight_mlp(const moe_bf16_t *expanded_x, const int32_t *offsets,
                                           int32_t G, const moe_fp4_t *w13, const moe_fp4_t *w2,
                                           int32_t n, int32_t H, int32_t I, uint32_t flags,
                                           moe_bf16_t *act, void *y, void *workspace,
                                           size_t workspace_bytes, int32_t *dev_status,
                                           moe_stream_t stream) {
    const Product up{expanded_x, offsets, G, w13, n, H, I, true}, down{act, offsets, G, w2, n, I, H,
                                                                       false};
    moe_status_t st = check(up);
    if (st == MOE_OK) st = check(down);
    if (st != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    if (!expanded_x || !a16(expanded_x) || !act || !a16(act) || !y || !a16(y))
        return MOE_ERR_INVALID_ARG;
    if (bad_workspace(workspace, workspace_bytes, workspace_bytes_of(n, std::max(H, I))))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = run(up, 0, act, workspace, dev_status, s);
    if (st != MOE_OK) return st;
    return run(down, flags, y, workspace, dev_status, s);
}
