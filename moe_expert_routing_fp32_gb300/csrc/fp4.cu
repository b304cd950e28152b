// fp4.cu -- rows to microscaled 4-bit floating point and back.
//
// Both kernels are copies with arithmetic on the way and bound by HBM: per
// element 2 bytes in and 1/2 + 1/block bytes out for every row written, or
// the reverse.  A warp takes 1024 columns of a row, a lane 32 of them: whole
// blocks, so a block's largest magnitude is found without another lane, and 16
// bytes of codes to a store.  With `row_idx` a token's row is read and
// quantised once and written to each of its k rows in expert order, the
// permute of the bf16 path at a quarter of its bytes.
//
// Measured at 16384 tokens x 4096 into 8 rows each (MX): quantise 73 us, 5.7 TB/s
// of the 419 MB it cannot do without; dequantise the 131072 rows 200 us, 6.8 TB/s.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_COLS = 1024;      // columns of one warp's piece of a row
constexpr int kMaxGroups = 1024;

__device__ __forceinline__ void load_offsets(int *s_off, const int32_t *offsets, int G) {
    if (offsets) {
        for (int g = threadIdx.x; g <= G; g += blockDim.x) s_off[g] = offsets[g];
    } else if (threadIdx.x == 0) {
        s_off[0] = 0;
        s_off[1] = 0x7fffffff;
    }
    __syncthreads();
}

// Byte offset of row r's scales (of its first tile), or -1 where no group
// holds the row.
__device__ __forceinline__ int64_t row_scales(const int *s_off, int G, int r, int64_t row_bytes) {
    const int g = find_group(s_off, G, r);
    if (g < 0) return -1;
    return scale_row_block(g, s_off[g], r) * row_bytes + scale_row_offset(r - s_off[g]);
}

template <int FMT>
__global__ void __launch_bounds__(Q_THREADS)
fp4_quantize_kernel(const uint16_t *__restrict__ x, const int32_t *__restrict__ row_idx, int T,
                    int K, int k, int n, const int32_t *__restrict__ offsets, int G,
                    float inv_unit, float unit, uint8_t *__restrict__ q, uint8_t *__restrict__ sf,
                    int32_t *dev_status) {
    constexpr int BLOCKS = 32 / Fp4<FMT>::BLOCK;     // scale blocks of a lane's 32 columns
    constexpr int LPT = 4 / BLOCKS;                  // lanes sharing a tile's four blocks
    __shared__ int s_off[kMaxGroups + 1];
    load_offsets(s_off, offsets, G);
    const int lane = threadIdx.x & 31;
    const int pieces = (K + Q_COLS - 1) / Q_COLS;
    const int64_t units = static_cast<int64_t>(T) * pieces;
    const int64_t tile_row = static_cast<int64_t>(K / Fp4<FMT>::TILE_K) * kScaleTile;
    const int per_cta = blockDim.x / 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * per_cta;
    for (int64_t u = blockIdx.x * static_cast<int64_t>(per_cta) + (threadIdx.x >> 5); u < units;
         u += warps) {
        const int t = static_cast<int>(u / pieces);
        const int c = static_cast<int>(u % pieces) * Q_COLS + lane * 32;
        // lane j holds destination j: its row and where its scales go
        int my_row = -1;
        if (lane < k) my_row = row_idx ? row_idx[static_cast<int64_t>(t) * k + lane] : t;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < K)
                v[i] = __ldg(reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(t) * K + c) + i);
        }
        int64_t my_sf = -1;
        if (my_row >= n) report(dev_status, MOE_DEV_BAD_OFFSETS);
        if (my_row >= 0 && my_row < n) my_sf = row_scales(s_off, G, my_row, tile_row);
        if (my_sf < 0) my_row = -1;                  // behind the last group: left as it was
        uint32_t am[4], code[4], sc = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            am[i] = amax8(w);
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            float factor;
            uint32_t m = 0;
#pragma unroll
            for (int i = b * 4 / BLOCKS; i < (b + 1) * 4 / BLOCKS; ++i) m = max(m, am[i]);
            sc |= block_scale<FMT>(m, inv_unit, unit, factor) << (8 * b);
#pragma unroll
            for (int i = b * 4 / BLOCKS; i < (b + 1) * 4 / BLOCKS; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                code[i] = quantize8<FMT>(w, factor);
            }
        }
        // the four scale bytes of a tile's row end up in its first lane
#pragma unroll
        for (int o = 1; o < LPT; o <<= 1)
            sc |= __shfl_down_sync(0xffffffffu, sc, o) << (8 * BLOCKS * o);
        for (int j = 0; j < k; ++j) {
            const int row = __shfl_sync(0xffffffffu, my_row, j);
            const int64_t so = __shfl_sync(0xffffffffu, my_sf, j);
            if (row < 0 || c >= K) continue;
            *reinterpret_cast<uint4 *>(q + static_cast<int64_t>(row) * (K / 2) + c / 2) =
                make_uint4(code[0], code[1], code[2], code[3]);
            if (lane % LPT == 0)
                *reinterpret_cast<uint32_t *>(sf + so + static_cast<int64_t>(c / Fp4<FMT>::TILE_K) *
                                                            kScaleTile) = sc;
        }
    }
}

// Two e2m1 codes (a byte) to fp32, times s, as packed bf16; the products have
// at most six significant bits, so nothing is rounded.
__device__ __forceinline__ uint32_t dequantize2(uint32_t byte, float s) {
    uint32_t h;
    asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(h)
        : "r"(byte));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return bf16x2(lo * s, hi * s);
}

// What a scale byte stands for.  The formats' NaN bytes are NaN here as they
// are to the tensor cores.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t b, float unit) {
    if ((FMT == MOE_FP4_MX ? b : b & 0x7Fu) == kScaleNaN<FMT>) return __uint_as_float(0x7FFFFFFFu);
    if (FMT == MOE_FP4_MX) return __uint_as_float(b == 0 ? 1u << 22 : b << 23);
    return e4m3_value(b) * unit;
}

// A warp takes 1024 columns of the rows r, r + 32, r + 64 and r + 96 of a
// 128-row scale block: their scale bytes share 16 bytes of every tile, loaded
// once.  A row's eight passes of 128 columns write 8 bytes a lane.
template <int FMT>
__global__ void __launch_bounds__(Q_THREADS)
fp4_dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ sf,
                      const int32_t *__restrict__ offsets, int G, int n, int K, float unit,
                      uint16_t *__restrict__ out) {
    constexpr int TK = Fp4<FMT>::TILE_K;
    __shared__ int s_off[kMaxGroups + 1];
    load_offsets(s_off, offsets, G);
    const int lane = threadIdx.x & 31;
    const int pieces = (K + Q_COLS - 1) / Q_COLS;
    const int64_t blocks = offsets ? static_cast<int64_t>(n / 128) + G : (static_cast<int64_t>(n) + 127) / 128;
    const int64_t units = blocks * 32 * pieces;
    const int ktiles = K / TK;
    const int per_cta = blockDim.x / 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * per_cta;
    for (int64_t u = blockIdx.x * static_cast<int64_t>(per_cta) + (threadIdx.x >> 5); u < units;
         u += warps) {
        const int c0 = static_cast<int>(u % pieces) * Q_COLS;
        const int64_t rb = u / pieces;
        const int r32 = static_cast<int>(rb & 31);
        const int64_t blk = rb >> 5;
        // the last group whose blocks begin at or before this one
        int g = 0;
        if (offsets) {
            int hi = G - 1;
            while (g < hi) {
                const int mid = (g + hi + 1) >> 1;
                if (scale_row_block(mid, s_off[mid], s_off[mid]) <= blk)
                    g = mid;
                else
                    hi = mid - 1;
            }
        }
        const int start = s_off[g], end = offsets ? min(s_off[g + 1], n) : n;
        const int64_t first = start + (blk - scale_row_block(g, start, start)) * 128 + r32;
        if (start < 0 || blk < scale_row_block(g, start, start) || first >= end) continue;
        // lane i < tiles of the piece: 16 scale bytes of tile i, one word per row
        const int t0 = c0 / TK;
        uint4 sc = make_uint4(0u, 0u, 0u, 0u);
        if (lane < Q_COLS / TK && t0 + lane < ktiles)
            sc = __ldg(reinterpret_cast<const uint4 *>(
                sf + (blk * ktiles + t0 + lane) * kScaleTile + r32 * 16));
        const uint32_t words[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = first + 32 * j;
            if (row >= end) break;
            const uint8_t *src = q + row * (K / 2);
            uint16_t *dst = out + row * K;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i * 256 + lane * 8;
                w[i] = c < K ? __ldg(reinterpret_cast<const uint32_t *>(src + c / 2)) : 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int cl = i * 256 + lane * 8;
                const uint32_t b = __shfl_sync(0xffffffffu, words[j], cl / TK) >>
                                       (8 * (cl / Fp4<FMT>::BLOCK % 4)) & 0xFFu;
                const float s = scale_value<FMT>(b, unit);
                if (c0 + cl < K)
                    *reinterpret_cast<uint4 *>(dst + c0 + cl) =
                        make_uint4(dequantize2(w[i] & 0xFFu, s), dequantize2(w[i] >> 8 & 0xFFu, s),
                                   dequantize2(w[i] >> 16 & 0xFFu, s), dequantize2(w[i] >> 24, s));
            }
        }
    }
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Warps for `units` pieces: eight to a CTA, and a CTA for every eight pieces up
// to 64 an SM (with 8 an SM, each looping, the last round leaves SMs idle:
// dequantising 131072 x 4096 takes 228 us instead of 200).  Few units spread over
// the SMs in smaller CTAs (64 rows of 4096 columns: 256 units on 128 CTAs
// instead of 32).
struct QShape {
    int grid, threads;
};
QShape q_shape(int64_t units) {
    const int64_t sms = num_sms();
    int per = Q_THREADS / 32;
    while (per > 1 && ceil_div(units, per) < 2 * sms) per /= 2;
    return {static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(units, per), sms * 64))),
            per * 32};
}

}  // namespace

// Shared by the entry points that take 4-bit matrices: format and factor.
moe_status_t fp4_check(int format, int scale_exp) {
    if (format != MOE_FP4_MX && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    if (format == MOE_FP4_MX ? scale_exp != 0 : (scale_exp < -60 || scale_exp > 60))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_scales_size(int32_t rows, int32_t K, int32_t G, int32_t format,
                                            size_t *bytes) {
    if (!bytes || rows < 0 || K <= 0 || G < 0) return MOE_ERR_INVALID_ARG;
    if (format != MOE_FP4_MX && format != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > (1 << 20) || G > kMaxGroups) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int64_t blocks = G > 0 ? static_cast<int64_t>(rows / 128) + G : ceil_div(rows, 128);
    const int tile_k = format == MOE_FP4_MX ? Fp4<MOE_FP4_MX>::TILE_K : Fp4<MOE_FP4_NV>::TILE_K;
    *bytes = static_cast<size_t>(blocks) * (K / tile_k) * kScaleTile;
    return MOE_OK;
}

extern "C" moe_status_t moe_fp4_quantize(const moe_bf16_t *x, int32_t T, int32_t K,
                                         const int32_t *expanded_row_idx, int32_t k,
                                         const int32_t *offsets, int32_t G, const moe_fp4_t *out,
                                         int32_t *dev_status, moe_stream_t stream) {
    if (T < 0 || K <= 0 || k <= 0 || !out) return MOE_ERR_INVALID_ARG;
    if (offsets ? G <= 0 : G != 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = fp4_check(out->format, out->scale_exp);
    if (st != MOE_OK) return st;
    if (K % 128 != 0 || K > (1 << 20) || k > 32 || G > kMaxGroups || (!expanded_row_idx && k != 1))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(T) * k >= (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !out->q || !out->sf || !a16(x) || !a16(out->q) || !a16(out->sf))
        return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const QShape qs = q_shape(static_cast<int64_t>(T) * ceil_div(K, Q_COLS));
    const int groups = offsets ? G : 1;
    const float unit = pow2f(out->scale_exp), inv = pow2f(-out->scale_exp);
    if (out->format == MOE_FP4_MX)
        fp4_quantize_kernel<MOE_FP4_MX><<<qs.grid, qs.threads, 0, s>>>(
            x, expanded_row_idx, T, K, k, T * k, offsets, groups, inv, unit, out->q, out->sf,
            dev_status);
    else
        fp4_quantize_kernel<MOE_FP4_NV><<<qs.grid, qs.threads, 0, s>>>(
            x, expanded_row_idx, T, K, k, T * k, offsets, groups, inv, unit, out->q, out->sf,
            dev_status);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_fp4_dequantize(const moe_fp4_t *m, int32_t n, int32_t K,
                                           const int32_t *offsets, int32_t G, moe_bf16_t *x,
                                           moe_stream_t stream) {
    if (n < 0 || K <= 0 || !m) return MOE_ERR_INVALID_ARG;
    if (offsets ? G <= 0 : G != 0) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = fp4_check(m->format, m->scale_exp);
    if (st != MOE_OK) return st;
    if (K % 128 != 0 || K > (1 << 20) || G > kMaxGroups) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (n == 0) return MOE_OK;
    if (!x || !m->q || !m->sf || !a16(x) || !a16(m->q) || !a16(m->sf)) return MOE_ERR_INVALID_ARG;
    if (!current_device_ok()) return MOE_ERR_NO_DEVICE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const QShape qs = q_shape((offsets ? n / 128 + static_cast<int64_t>(G) : ceil_div(n, 128)) * 32 *
                              ceil_div(K, Q_COLS));
    const int groups = offsets ? G : 1;
    const float unit = pow2f(m->scale_exp);
    if (m->format == MOE_FP4_MX)
        fp4_dequantize_kernel<MOE_FP4_MX><<<qs.grid, qs.threads, 0, s>>>(m->q, m->sf, offsets, groups, n,
                                                                    K, unit, x);
    else
        fp4_dequantize_kernel<MOE_FP4_NV><<<qs.grid, qs.threads, 0, s>>>(m->q, m->sf, offsets, groups, n,
                                                                    K, unit, x);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
