// fp4.cu -- rows to microscaled 4-bit floating point and back.
//
// Both kernels are copies with arithmetic on the way and bound by HBM: per
// element 2 bytes in and 1/2 + 1/block bytes out for every row written, or
// the reverse.  A warp takes 1024 columns of one row: four passes of 256
// columns, a lane holding 8 of them (16 bytes), so loads and stores are whole
// 512- and 128-byte lines and a block's largest magnitude needs two shuffles
// (32 columns) or one (16).  With `row_idx` a token's row is read and
// quantised once and written to each of its k rows in expert order, the
// permute of the bf16 path at a quarter of its bytes.
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
    constexpr int LPB = Fp4<FMT>::BLOCK / 8;         // lanes sharing a block
    __shared__ int s_off[kMaxGroups + 1];
    load_offsets(s_off, offsets, G);
    const int lane = threadIdx.x & 31;
    const int pieces = (K + Q_COLS - 1) / Q_COLS;
    const int64_t units = static_cast<int64_t>(T) * pieces;
    const int64_t tile_row = static_cast<int64_t>(K / Fp4<FMT>::TILE_K) * kScaleTile;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (Q_THREADS / 32);
    for (int64_t u = blockIdx.x * static_cast<int64_t>(Q_THREADS / 32) + (threadIdx.x >> 5);
         u < units; u += warps) {
        const int t = static_cast<int>(u / pieces);
        const int c0 = static_cast<int>(u % pieces) * Q_COLS;
        // lane j holds destination j: its row and where its scales go
        int my_row = -1;
        int64_t my_sf = -1;
        if (lane < k) {
            my_row = row_idx ? row_idx[static_cast<int64_t>(t) * k + lane] : t;
            if (my_row >= n) {
                report(dev_status, MOE_DEV_BAD_OFFSETS);
                my_row = -1;
            }
            if (my_row >= 0) my_sf = row_scales(s_off, G, my_row, tile_row);
            if (my_sf < 0) my_row = -1;              // behind the last group: left as it was
        }
        const uint4 *src = reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(t) * K);
        uint32_t code[Q_COLS / 256];
        uint32_t sc[Q_COLS / 256];
#pragma unroll
        for (int i = 0; i < Q_COLS / 256; ++i) {
            const int c = c0 + i * 256 + lane * 8;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (c < K) v = __ldg(src + c / 8);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t am = amax8(w);
#pragma unroll
            for (int o = 1; o < LPB; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
            float factor;
            uint32_t b = block_scale<FMT>(am, inv_unit, unit, factor);
            code[i] = quantize8<FMT>(w, factor);
            // the four scale bytes of a tile's row end up in its first lane
            b |= __shfl_down_sync(0xffffffffu, b, LPB) << 8;
            b |= __shfl_down_sync(0xffffffffu, b, 2 * LPB) << 16;
            sc[i] = b;
        }
        for (int j = 0; j < k; ++j) {
            const int row = __shfl_sync(0xffffffffu, my_row, j);
            const int64_t so = __shfl_sync(0xffffffffu, my_sf, j);
            if (row < 0) continue;
            uint32_t *dst = reinterpret_cast<uint32_t *>(q + static_cast<int64_t>(row) * (K / 2));
#pragma unroll
            for (int i = 0; i < Q_COLS / 256; ++i) {
                const int c = c0 + i * 256 + lane * 8;
                if (c >= K) break;
                dst[c / 8] = code[i];
                if (lane % (4 * LPB) == 0)
                    *reinterpret_cast<uint32_t *>(sf + so + c / Fp4<FMT>::TILE_K * kScaleTile) =
                        sc[i];
            }
        }
    }
}

// e2m1 code -> value, exactly.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float v = e == 0 ? 0.5f * static_cast<float>(m)
                           : __uint_as_float(((e + 126u) << 23) | (m << 22));
    return (c & 8u) ? -v : v;
}

template <int FMT>
__global__ void __launch_bounds__(Q_THREADS)
fp4_dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ sf,
                      const int32_t *__restrict__ offsets, int G, int n, int K, float unit,
                      uint16_t *__restrict__ out) {
    __shared__ int s_off[kMaxGroups + 1];
    load_offsets(s_off, offsets, G);
    const int lane = threadIdx.x & 31;
    const int pieces = (K + Q_COLS - 1) / Q_COLS;
    const int64_t units = static_cast<int64_t>(n) * pieces;
    const int64_t tile_row = static_cast<int64_t>(K / Fp4<FMT>::TILE_K) * kScaleTile;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (Q_THREADS / 32);
    for (int64_t u = blockIdx.x * static_cast<int64_t>(Q_THREADS / 32) + (threadIdx.x >> 5);
         u < units; u += warps) {
        const int r = static_cast<int>(u / pieces);
        const int c0 = static_cast<int>(u % pieces) * Q_COLS;
        const int64_t so = row_scales(s_off, G, r, tile_row);
        if (so < 0) continue;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(q + static_cast<int64_t>(r) * (K / 2));
        uint4 *dst = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(r) * K);
#pragma unroll
        for (int i = 0; i < Q_COLS / 256; ++i) {
            const int c = c0 + i * 256 + lane * 8;
            if (c >= K) break;
            const uint32_t w = __ldg(src + c / 8);
            const uint32_t b = sf[so + static_cast<int64_t>(c / Fp4<FMT>::TILE_K) * kScaleTile +
                                  c / Fp4<FMT>::BLOCK % 4];
            float s;
            if (FMT == MOE_FP4_MX)
                s = b == 0 ? __uint_as_float(1u << 22) : __uint_as_float(b << 23);
            else
                s = e4m3_value(b) * unit;
            uint32_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
                o[p] = bf16x2(e2m1_value(w >> (8 * p)) * s, e2m1_value(w >> (8 * p + 4)) * s);
            dst[c / 8] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

inline bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int q_grid(int64_t units) {
    return static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(ceil_div(units, Q_THREADS / 32), static_cast<int64_t>(num_sms()) * 8)));
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
    const int grid = q_grid(static_cast<int64_t>(T) * ceil_div(K, Q_COLS));
    const int groups = offsets ? G : 1;
    const float unit = pow2f(out->scale_exp), inv = pow2f(-out->scale_exp);
    if (out->format == MOE_FP4_MX)
        fp4_quantize_kernel<MOE_FP4_MX><<<grid, Q_THREADS, 0, s>>>(
            x, expanded_row_idx, T, K, k, T * k, offsets, groups, inv, unit, out->q, out->sf,
            dev_status);
    else
        fp4_quantize_kernel<MOE_FP4_NV><<<grid, Q_THREADS, 0, s>>>(
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
    const int grid = q_grid(static_cast<int64_t>(n) * ceil_div(K, Q_COLS));
    const int groups = offsets ? G : 1;
    const float unit = pow2f(m->scale_exp);
    if (m->format == MOE_FP4_MX)
        fp4_dequantize_kernel<MOE_FP4_MX><<<grid, Q_THREADS, 0, s>>>(m->q, m->sf, offsets, groups, n,
                                                                    K, unit, x);
    else
        fp4_dequantize_kernel<MOE_FP4_NV><<<grid, Q_THREADS, 0, s>>>(m->q, m->sf, offsets, groups, n,
                                                                    K, unit, x);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
