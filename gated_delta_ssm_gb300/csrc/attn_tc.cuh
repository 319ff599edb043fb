// attn_tc.cuh -- pieces shared by the two tensor-core attention kernels: 8-bit
// tcgen05 products, the split of q and of weights into two e4m3 numbers, the score
// cap, bounded waits and the page-by-page tile copies of the cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "attn_share.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace gdn {
namespace attn {

constexpr uint32_t kTileBytes = kTile * kHd;  // one tile of K or V codes
constexpr float kLog2e = 1.4426950408889634f;

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

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How scores are capped: not, so low that weights need no reference, or anyhow.
enum { kNoCap = 0, kLowCap = 1, kAnyCap = 2 };
// In base 2: sums of 2^30 weights stay below 2^110; and the factor 2 log2 e / cap stays finite.
constexpr float kMostCap = 80.0f, kLeastCap = 1e-6f;
__host__ __device__ inline int cap_mode(float softcap)
{
    return softcap == 0.0f ? kNoCap : softcap * kLog2e <= kMostCap && softcap >= kLeastCap ? kLowCap : kAnyCap;
}

// a * b + c and a + b of two packed floats.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The smaller of the two; NaN where either is (fminf would give the other).
__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t a)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ float redux_max(float x)
{
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Two e4m3 numbers whose sum is (x, y), to within 2^-8 of each and 2^-10, for magnitudes up to 448 (callers stay at 256
// and below): the low byte of each result is x's. By way of fp16, which both conversions and the difference between
// them take two at a time; its rounding, 2^-11, is an eighth of the sum's.
__device__ __forceinline__ void split_e4m3(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 v = __floats2half2_rn(x, y);
    hi = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    const __half2 back(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3));
    lo = __nv_cvt_halfraw2_to_fp8x2(__hsub2(v, back), __NV_SATFINITE, __NV_E4M3);
}

// 16 bf16 elements as floats.
__device__ __forceinline__ void unpack_q16(uint4 a, uint4 b, float (&v)[16])
{
    const uint32_t y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[2 * e] = __uint_as_float(y[e] << 16);
        v[2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u);
    }
}

// 16 elements of a q row (16-byte aligned).
__device__ __forceinline__ void load_q16(const __nv_bfloat16 *p, float (&v)[16])
{
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    unpack_q16(a, b, v);
}

// x with 2^x top in [128, 256) (1 for top = 0: the factor of its scores, 0.72 scale, is finite for any scale); at
// most 126, so that 2^x stays finite.
__device__ __forceinline__ int q_exponent(float top)
{
    return top > 0.0f ? min(126, 134 - (int)(__float_as_uint(top) >> 23)) : 1;
}
__device__ __forceinline__ float pow2i(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

// The factor of a q row whose largest magnitude is top: 2^q_exponent, or NaN for a row that holds an infinity:
// its scores, and with them its output, are NaN, capped or not, as are those of a row that holds a NaN.
__device__ __forceinline__ float q_factor(float top)
{
    return top < CUDART_INF_F ? pow2i(q_exponent(top)) : CUDART_NAN_F;
}

// The 16 elements times `up` as hi + lo, at dst and dst + lo_at.
__device__ __forceinline__ void store_q16(uint8_t *dst, uint32_t lo_at, const float (&v)[16], float up)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t h0, l0, h1, l1;
        split_e4m3(v[4 * c] * up, v[4 * c + 1] * up, h0, l0);
        split_e4m3(v[4 * c + 2] * up, v[4 * c + 3] * up, h1, l1);
        hi[c] = h0 | h1 << 16;
        lo[c] = l0 | l1 << 16;
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(dst + lo_at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// Wait for a phase, at most limit_ns of the global timer, or until *abort. A try sleeps for as long as the
// hardware sees fit. The timer is read once in 256 tries. A limit under 1 us gives up at once, without a
// try: a test hook takes that path.
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity, uint64_t limit_ns,
                                           const volatile int *abort)
{
    if (limit_ns < 1000)
        return false;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
        if (done)
            return true;
        if (*abort != 0)
            return false;
        if (i % 256 == 0) {
            const uint64_t now = tc::global_ns();
            if (t0 == 0)
                t0 = now;
            else if (now - t0 > limit_ns)
                return false;
        }
    }
}

// Whether any of the threads that meet at a named barrier says so.
__device__ __forceinline__ bool named_any(int id, int threads, bool mine)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(id), "r"(threads), "r"((uint32_t)mine) : "memory");
    return any != 0;
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
