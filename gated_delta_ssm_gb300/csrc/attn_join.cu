// attn_join.cu -- joins the partial results of the attention kernels: a block of
// q rows whose keys were shared out over several CTAs.
#include "attn_device.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace attn {

// CTA x joins the block that begins in share x: its own part (slot 2 x + 1) and the parts that the shares
// after it began with (slots 2 c). A warp per row, four dimensions per lane. A part's row holds the 128
// unnormalised sums, the sum of weights l and their reference m: the true values are 2^m times these.
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs A, int rows)
{
    const Batch &B = A.b;
    wait_previous_grid();
    allow_next_grid();
    const PartMeta m = reinterpret_cast<const PartMeta *>(A.ws)[blockIdx.x];
    if (!m.owner)
        return;
    const Seq s = load_seq(B, m.b);
    const int i = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int r = m.row0 + i;
    if (i >= rows || r >= s.n * B.G)
        return;
    const float *parts = part_slots(A.ws, gridDim.x);
    const size_t size = (size_t)rows * kPartRow;
    float big = -INFINITY, l = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int c = blockIdx.x; c <= m.last_cta; ++c) {
        const float *p = parts + (size_t)(2 * c + (c == (int)blockIdx.x ? 1 : 0)) * size + (size_t)i * kPartRow;
        const float2 lm = *reinterpret_cast<const float2 *>(p + kHd);
        const float4 x = *reinterpret_cast<const float4 *>(p + 4 * lane);
        const float grown = fmaxf(big, lm.y);
        const float a = grown == -INFINITY ? 1.0f : exp2f(big - grown);
        const float b = grown == -INFINITY ? 0.0f : exp2f(lm.y - grown);
        l = fmaf(l, a, lm.x * b);
        o.x = fmaf(o.x, a, x.x * b);
        o.y = fmaf(o.y, a, x.y * b);
        o.z = fmaf(o.z, a, x.z * b);
        o.w = fmaf(o.w, a, x.w * b);
        big = grown;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    const int tok = r / B.G, g = r - tok * B.G;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(A.out) +
                              ((int64_t)(s.row0 + tok) * B.Hq + m.h * B.G + g) * kHd)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

cudaError_t launch_join(const AttnArgs &a, int grid, int rows, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, (rows + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel, a, rows);
}

}  // namespace attn
}  // namespace gdn
