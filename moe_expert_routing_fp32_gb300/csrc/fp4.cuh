// fp4.cuh -- microscaled 4-bit floating point: formats, scale layout and the
// device helpers shared by the quantisation and the matmul kernels.
//
// A value is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times its
// block's scale, one byte per block along K:
//   MOE_FP4_MX  blocks of 32, scale 2^(byte - 127);
//   MOE_FP4_NV  blocks of 16, scale e4m3(byte) * 2^scale_exp.
// Two elements share a byte, the lower column in its low four bits.
//
// Scale layout.  The tensor cores take the scales of 128 rows x 4 blocks as
// one 512-byte tile: the byte of row r, block b (r < 128, b < 4) lies at
// (r % 32) * 16 + (r / 32) * 4 + b, so that a 32-lane x 16-byte copy into
// tensor memory puts rows 32c.. into column c.  Tiles of one 128-row block
// follow each other along K, then come the next 128 rows.  A grouped matrix
// starts every group on a tile of its own without a scan over the groups:
// group g's row blocks begin at offsets[g] / 128 + g.  They do not overlap:
// floor((a + c) / 128) + 1 >= floor(a / 128) + ceil(c / 128).
#pragma once

#include "common.cuh"

namespace moe {

template <int FMT>
struct Fp4 {
    static constexpr int BLOCK = FMT == MOE_FP4_MX ? 32 : 16;   // elements per scale
    static constexpr int TILE_K = 4 * BLOCK;                    // columns of a scale tile
};

constexpr int kScaleTile = 512;   // bytes: 128 rows x 4 blocks

// The scale byte that makes its block NaN.
template <int FMT>
constexpr uint32_t kScaleNaN = FMT == MOE_FP4_MX ? 255u : 127u;

// Row block (128 rows) of row `r` of a matrix whose group g starts at `start`.
__host__ __device__ __forceinline__ int64_t scale_row_block(int g, int start, int r) {
    return static_cast<int64_t>(start / 128) + g + (r - start) / 128;
}
__host__ __device__ __forceinline__ int scale_row_offset(int local_row) {
    const int r = local_row & 127;
    return (r & 31) * 16 + (r >> 5) * 4;
}

// Group of row r (the last g with off[g] <= r); -1 if no group holds it.
__device__ __forceinline__ int find_group(const int *off, int G, int r) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return (off[lo] >= 0 && off[lo] <= r && r < off[lo + 1]) ? lo : -1;
}

// Two fp32 values to packed bf16 (nearest even) in one conversion; two single
// conversions and a merge take four times as long in a kernel's epilogue.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four packed e2m1 pairs: the eight values' codes, value i in bits [4i, 4i+4)
// (nearest, ties to even, magnitudes beyond 6 to 6).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// e4m3 byte of f >= 0 (nearest even, beyond 448 to 448) and back (not of NaN).
__device__ __forceinline__ uint32_t e4m3_bits(float f) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(f));
    return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const uint32_t e = (b >> 3) & 15u, m = b & 7u;
    return e == 0 ? static_cast<float>(m) * 0.001953125f          // m 2^-9
                  : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// The scale byte of a block whose largest magnitude has the bf16 bits `amax`,
// and the factor that brings the block's elements onto the e2m1 grid.
//   MX: 2^(floor(log2 amax) - 2), exact; below 2^-125 the byte is 0.
//   NV: e4m3(amax / 6) in units of 2^scale_exp; a block whose scale rounds to
//       zero is held as zeros (factor 0).
// A block with an infinity or a NaN gets the NaN byte: its codes, which know
// neither, would make them 6 times a finite scale.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, float inv_unit, float unit,
                                                float &factor) {
    if (amax >= 0x7F80u) {
        factor = 0.0f;
        return kScaleNaN<FMT>;
    }
    if (FMT == MOE_FP4_MX) {
        const int e = static_cast<int>(amax >> 7);
        const uint32_t b = static_cast<uint32_t>(e > 2 ? e - 2 : 0);
        factor = __uint_as_float((254u - b) << 23);
        return b;
    }
    const uint32_t b = e4m3_bits(__fdiv_rn(__uint_as_float(amax << 16), 6.0f) * inv_unit);
    factor = b == 0 ? 0.0f : __frcp_rn(e4m3_value(b) * unit);
    return b;
}

// Codes of eight bf16 values (packed in pairs) under a block's factor.
//   MX: value * factor is exact, so the conversion's one rounding is that of
//       the definition.
//   NV: the quotient value / scale has at most 8 over 4 significant bits.  It
//       is either exactly a midpoint of the e2m1 grid or 2^-8 and more away
//       from one (relative), so rounding value * (1 / scale), which is off by
//       2^-22, to 13 significant bits first restores the exact midpoints and
//       moves nothing else across one.
template <int FMT>
__device__ __forceinline__ uint32_t quantize8(const uint32_t (&w)[4], float factor) {
    if (FMT == MOE_FP4_NV && factor == 0.0f) return 0u;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16) * factor;
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * factor;
    }
    if (FMT == MOE_FP4_NV) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float((__float_as_uint(v[i]) + 0x400u) & 0xFFFFF800u);
    }
    return e2m1x8(v);
}

// Largest magnitude (bf16 bits) of eight packed bf16 values.
__device__ __forceinline__ uint32_t amax8(const uint32_t (&w)[4]) {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
}

// 2^e for -126 <= e <= 127.
__host__ __device__ __forceinline__ float pow2f(int e) {
    union {
        uint32_t u;
        float f;
    } c;
    c.u = static_cast<uint32_t>(e + 127) << 23;
    return c.f;
}

}  // namespace moe
