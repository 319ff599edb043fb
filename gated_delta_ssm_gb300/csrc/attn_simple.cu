// attn_simple.cu -- attention over the paged 8-bit cache, one warp per (token,
// q head): each lane holds 4 of the 128 dimensions, the score of a key is a
// warp reduction, and the softmax runs online over the keys.
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_attn_error;

__device__ __forceinline__ float4 code_values(uint32_t w)
{
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffff), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    return make_float4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(256) attn_simple_kernel(const __grid_constant__ AttnArgs A)
{
    const Batch &B = A.b;
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const Seq s = load_seq(B, b);
    if (!s.ok) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            atomicOr(&g_attn_error, kErrMeta);
        return;
    }
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int tok = (int)(item / B.Hq), h = (int)(item - (int64_t)tok * B.Hq), hk = h / B.G;
    if (tok >= s.n)
        return;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(A.q) +
                             (int64_t)(s.row0 + tok) * A.q_stride + h * kHd + lane * 4;
    float qv[4];
    for (int i = 0; i < 4; ++i)
        qv[i] = __bfloat162float(q[i]) * A.scale;
    const int p = s.L - s.n + tok;
    const int lo = A.window > 0 ? max(0, p - A.window + 1) : 0;
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    int page = -1, blk = -1;
    float ks = 0, vs = 0;
    for (int j = lo; j <= p; ++j) {
        if (j / B.P != blk) {
            blk = j / B.P;
            page = __ldg(B.page_table + (int64_t)b * B.max_pages + blk);
            if (page < 0 || page >= B.n_pages) {
                if (lane == 0)
                    atomicOr(&g_attn_error, kErrMeta);
                page = -1;
            } else {
                ks = B.k_scale[(int64_t)page * B.Hkv + hk];
                vs = B.v_scale[(int64_t)page * B.Hkv + hk];
            }
        }
        if (page < 0)
            continue;
        const int64_t at = (((int64_t)page * B.Hkv + hk) * B.P + j - blk * B.P) * kHd + lane * 4;
        const float4 k = code_values(*reinterpret_cast<const uint32_t *>(B.k + at));
        float d = qv[0] * k.x + qv[1] * k.y + qv[2] * k.z + qv[3] * k.w;
        for (int x = 16; x > 0; x >>= 1)
            d += __shfl_xor_sync(0xffffffffu, d, x);
        d *= ks;
        if (A.softcap > 0)
            d = A.softcap * tanhf(d / A.softcap);
        const float mn = fmaxf(m, d), al = expf(m - mn), w = expf(d - mn);
        const float4 v = code_values(*reinterpret_cast<const uint32_t *>(B.v + at));
        l = l * al + w;
        o[0] = o[0] * al + w * vs * v.x;
        o[1] = o[1] * al + w * vs * v.y;
        o[2] = o[2] * al + w * vs * v.z;
        o[3] = o[3] * al + w * vs * v.w;
        m = mn;
    }
    const float inv = l > 0 ? 1.0f / l : 0.0f;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(A.out) +
                         ((int64_t)(s.row0 + tok) * B.Hq + h) * kHd + lane * 4;
    for (int i = 0; i < 4; ++i)
        out[i] = __float2bfloat16_rn(o[i] * inv);
}

static cudaError_t launch_simple(const AttnArgs &a, cudaStream_t s)
{
    const int64_t rows = (int64_t)a.b.max_q * a.b.Hq;
    attn_simple_kernel<<<dim3((unsigned)((rows + 7) / 8), a.b.n_seq), 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_prefill(const AttnArgs &a, cudaStream_t s) { return launch_simple(a, s); }
size_t prefill_workspace_bytes(int) { return 16; }

cudaError_t take_prefill_error(int *code)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(int));
    if (e == cudaSuccess && v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(int));
    }
    *code = v;
    return e;
}
}  // namespace attn
}  // namespace gdn
