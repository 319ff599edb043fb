// attn_join.cu -- joins the partial results of the attention kernels: a block of
// q rows whose keys were shared out over several CTAs. Bound by latency: about
// 5 us behind a decode of one long sequence.

#include "attn_device.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace attn {

// CTA x joins the block that begins in share x: its own part (slot 2 x + 1) and the parts that the shares
// after it began with (slots 2 c). A part's row holds the 128 unnormalised sums, the sum of weights l and their
// reference m: the true values are 2^m times these. SPLIT warps take a row's parts in turn, four dimensions per
// lane: all maxima are read first (a lane per part), so the sums' loads do not wait for one another.
template <int SPLIT>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs A, int rows)
{
    constexpr int kPerCta = 4 / SPLIT;
    __shared__ float4 sum[4][32];
    __shared__ float sum_l[4];
    const Batch &B = A.b;
    wait_previous_grid();
    allow_next_grid();
    const PartMeta m = reinterpret_cast<const PartMeta *>(A.ws)[blockIdx.x];
    if (!m.owner)
        return;
    const Seq s = load_seq(B, m.b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int piece = warp % SPLIT, n = m.last_cta - (int)blockIdx.x + 1;
    const int live_rows = min(rows, s.n * B.G - m.row0);
    const size_t size = (size_t)rows * kPartRow;
    const float *const own = part_slots(A.ws, gridDim.x) + (size_t)(2 * blockIdx.x) * size;
#pragma unroll 1
    for (int i = blockIdx.y * kPerCta + warp / SPLIT; i < live_rows; i += gridDim.y * kPerCta) {
        auto part = [&](int c) { return own + (size_t)(c == 0 ? 1 : 2 * c) * size + (size_t)i * kPartRow; };
        float l = 0.0f, big = -INFINITY;
        float4 o = make_float4(0, 0, 0, 0);
        for (int c = lane; c < n; c += 32)
            big = fmaxf(big, part(c)[kHd + 1]);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1)
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
#pragma unroll 4
        for (int c = piece; c < n; c += SPLIT) {
            const float *p = part(c);
            const float2 lm = *reinterpret_cast<const float2 *>(p + kHd);
            const float4 x = *reinterpret_cast<const float4 *>(p + 4 * lane);
            const float b = big == -INFINITY ? 0.0f : exp2f(lm.y - big);
            l = fmaf(lm.x, b, l);
            o.x = fmaf(x.x, b, o.x);
            o.y = fmaf(x.y, b, o.y);
            o.z = fmaf(x.z, b, o.z);
            o.w = fmaf(x.w, b, o.w);
        }
        if (SPLIT > 1) {   // the CTA's warps are at the same row
            __syncthreads();
            sum[warp][lane] = o;
            if (lane == 0)
                sum_l[warp] = l;
            __syncthreads();
            if (piece != 0)
                continue;
#pragma unroll
            for (int k = 1; k < SPLIT; ++k) {
                const float4 x = sum[warp + k][lane];
                l += sum_l[warp + k];
                o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            }
        }
        const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
        const int r = m.row0 + i, tok = div_G(B, r), g = r - tok * B.G;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(A.out) +
                                  ((int64_t)(s.row0 + tok) * B.Hq + m.h * B.G + g) * kHd)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

// A decode call's few rows can span every CTA, so four warps share a row; a prefill block has 256 rows of
// two or three parts.
cudaError_t launch_join(const AttnArgs &a, int grid, int rows, cudaStream_t s)
{
    const bool few = rows <= kMaxDecodeRows;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // most CTAs find nothing to join: a grid of few keeps their launch short
    cfg.gridDim = dim3(grid, few ? (rows < 8 ? rows : 8) : 32);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few ? attn_join_kernel<4> : attn_join_kernel<1>, a, rows);
}

}  // namespace attn
}  // namespace gdn
