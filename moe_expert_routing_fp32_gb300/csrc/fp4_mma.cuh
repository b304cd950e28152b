// fp4_mma.cuh -- the block-scaled tensor-core instructions of 4-bit operands and
// the tensor maps they are fed by, shared by the matmul kernels.
#pragma once

#include <cuda.h>

#include <mutex>

#include "fp4.cuh"

namespace moe {

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

// ------------------------------------------------------------------ host side
constexpr int kCodeBox = 128;     // bytes of a row in a box of codes: 256 columns

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
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
inline bool code_map(CUtensorMap *m, const uint8_t *q, int rank, int64_t groups, int64_t rows, int K,
              int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t row_bytes = static_cast<cuuint64_t>(K) / 2;
    cuuint64_t dim[3] = {row_bytes, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(groups)};
    cuuint64_t stride[2] = {row_bytes, row_bytes * static_cast<cuuint64_t>(rows)};
    cuuint32_t boxd[3] = {kCodeBox, static_cast<cuuint32_t>(box), 1}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<uint8_t *>(q), dim, stride, boxd,
              es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 128 words, `box` of them at a time.
inline bool scale_map(CUtensorMap *m, const uint8_t *sf, int64_t tiles, int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dim[2] = {kScaleTile / 4, static_cast<cuuint64_t>(tiles)};
    cuuint64_t stride[1] = {kScaleTile};
    cuuint32_t boxd[2] = {kScaleTile / 4, static_cast<cuuint32_t>(box)}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(sf), dim, stride, boxd, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
