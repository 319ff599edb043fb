// attn_tc.cuh -- pieces shared by the two tensor-core attention kernels: 8-bit
// tcgen05 products, the page-by-page tile copies of the cache, and the cut of a
// ragged batch into equal shares.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace gdn {
namespace attn {

constexpr int kTile = 128;                    // keys per tile
constexpr uint32_t kTileBytes = kTile * kHd;  // one tile of K or V codes
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kNoWindow = 1 << 30;            // positions are below this

// D[tmem] (+)= A[smem] * B[smem]^T with e4m3 operands and 32-bit sums (a K step is 32).
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// Instruction descriptor of an e4m3 x e4m3 product: as idesc_f16 (both formats 0).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) { return tc::idesc_f16(M, N); }
constexpr uint32_t kIdescTransA = 1u << 15;   // A is MN-major

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// One box (one page of one head: P rows of 128 bytes) into shared memory.
__device__ __forceinline__ void copy_page(const CUtensorMap *map, uint32_t dst, uint32_t mbar, int head)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(head), "r"(mbar)
                 : "memory");
}

// tanh for the score cap. The quotient form loses small arguments to cancellation, so below 0.25
// the odd series to x^7 stands in (next term 62/2835 x^9, 3e-7 relative there).
__device__ __forceinline__ float tanh_cap(float x)
{
    const float x2 = x * x;
    const float small = x * fmaf(x2, fmaf(x2, fmaf(x2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
    const float big = 1.0f - __fdividef(2.0f, 1.0f + ex2(2.0f * kLog2e * x));
    return fabsf(x) < 0.25f ? small : big;
}

// The tensor map of a cache array: [n_pages * Hkv][P][128] codes in boxes of one page of one head, the
// 16-byte pieces of a row exchanged by the 128-byte swizzle that the tensor core reads.
inline bool encode_cache_map(CUtensorMap *map, const Batch &b, const uint8_t *codes)
{
    const EncodeTiledFn enc = tensor_map_encoder();
    const int64_t heads = (int64_t)b.n_pages * b.Hkv;
    if (!enc || heads > 0x7fffffff)
        return false;
    const cuuint64_t dims[3] = {kHd, (cuuint64_t)b.P, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {kHd, (cuuint64_t)b.P * kHd};
    const cuuint32_t box[3] = {kHd, (cuuint32_t)b.P, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace gdn
