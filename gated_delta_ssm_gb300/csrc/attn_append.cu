// attn_append.cu -- gdn_attn_append: rotate a batch's q and k by position,
// quantise k and v to e4m3 with one power-of-two scale per page and head, and
// write them into the paged cache.
//
// Bound by memory: every input element is read once, q written as bf16 and k, v
// as one byte. Work is cut so that no block waits for another:
//   cache blocks  one CTA per (sequence, page the call touches, KV head, K or V).
//                 It sees all of the page's new tokens at once, so the page's
//                 scale is a block reduction over values that stay in registers.
//   q blocks      kQRows (token, head) rows of one sequence per CTA.
// Eight threads share a row of 128, each with two 8-element pieces that hold the
// two members of 8 rotation pairs, so a pair never leaves its thread:
//   halves        pieces u*8 and rot/2 + u*8 while u < rot/16, then the 16
//                 unrotated elements rot + (u - rot/16)*16 ..;
//   interleaved   elements u*16 .. u*16 + 15.
// Either way thread u's angles are u*8 .. u*8 + 7 of the position's table row.
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_append_error;

constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100
constexpr int kQRows = 64;                            // (token, head) rows per q block

struct Row16 {
    float a[8], b[8];
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

// First elements of thread u's two pieces.
__device__ __forceinline__ void pieces(int u, int rot, int interleaved, int &ca, int &cb)
{
    if (!interleaved && u * 16 < rot) {
        ca = u * 8;
        cb = rot / 2 + u * 8;
    } else if (!interleaved) {
        ca = rot + (u - rot / 16) * 16;
        cb = ca + 8;
    } else {
        ca = u * 16;
        cb = ca + 8;
    }
}

// a*c - b*s and b*c + a*s with the rounding error of the second product carried
// along, so that the result is within about an ulp even where the terms cancel.
__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s)
{
    const float w = __fmul_rn(b, s), e = __fmaf_rn(-b, s, w);
    const float x = __fadd_rn(__fmaf_rn(a, c, -w), e);
    const float t = __fmul_rn(a, s), f = __fmaf_rn(a, s, -t);
    b = __fadd_rn(__fmaf_rn(b, c, t), f);
    a = x;
}

__device__ __forceinline__ void rotate_row(Row16 &r, const AppendArgs &A, int u, int pos)
{
    if (u * 16 >= A.rot)
        return;
    float c[8], s[8];
    const int64_t at = (int64_t)pos * (A.rot / 2) + u * 8;
    load8(A.cos + at, c);
    load8(A.sin + at, s);
    if (A.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair(r.a[2 * i], r.a[2 * i + 1], c[i], s[i]);
            rotate_pair(r.b[2 * i], r.b[2 * i + 1], c[4 + i], s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rotate_pair(r.a[i], r.b[i], c[i], s[i]);
    }
}

// The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), at least 2^-100.
__device__ __forceinline__ float pow2_scale(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 126;              // amax = m 2^e, m in [0.5, 1)
    const int x = e - 9 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return x <= -100 ? kMinScale : __uint_as_float((uint32_t)(x + 127) << 23);
}

__device__ __forceinline__ uint32_t codes4(float x, float y, float z, float w)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z, w), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ float code_value(uint32_t byte)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
    return __half2float(__half(h));
}

__device__ __forceinline__ uint4 pack_bf16(const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// |v| where v is finite, else 0 (and `bad` is set).
__device__ __forceinline__ float finite_abs(float v, bool &bad)
{
    const float m = fabsf(v);
    const bool ok = m < __uint_as_float(0x7f800000u);   // false for infinities and NaN
    bad |= !ok;
    return ok ? m : 0.0f;
}

template <typename T, int NT, int PASSES>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ AppendArgs A,
                                                    unsigned n_blocks, unsigned cache_ctas,
                                                    unsigned q_ctas)
{
    const Batch &B = A.b;
    const int tid = threadIdx.x, u = tid & 7, r = tid >> 3;
    unsigned item = blockIdx.x;
    int ca, cb;
    pieces(u, A.rot, A.interleaved, ca, cb);

    if (item >= cache_ctas) {   // ---- rotate q
        item -= cache_ctas;
        const int b = (int)(item / q_ctas), chunk = (int)(item % q_ctas);
        const Seq s = load_seq(B, b);
        const int64_t rows = (int64_t)s.n * B.Hq;
        const T *q = static_cast<const T *>(A.q);
        __nv_bfloat16 *qo = static_cast<__nv_bfloat16 *>(A.q_out);
        if (s.L > A.n_positions && A.rot > 0)
            return;             // the cache blocks report it
        Row16 x[2];
#pragma unroll
        for (int i = 0; i < kQRows / (NT / 8); ++i) {
            const int64_t row = (int64_t)chunk * kQRows + i * (NT / 8) + r;
            if (row >= rows)
                break;
            const int tok = (int)(row / B.Hq), h = (int)(row - (int64_t)tok * B.Hq);
            const T *src = q + (int64_t)(s.row0 + tok) * A.q_stride + h * kHd;
            Row16 &y = x[i & 1];
            load8(src + ca, y.a);
            load8(src + cb, y.b);
            rotate_row(y, A, u, max(s.L - s.n + tok, 0));
            __nv_bfloat16 *dst = qo + ((int64_t)(s.row0 + tok) * B.Hq + h) * kHd;
            *reinterpret_cast<uint4 *>(dst + ca) = pack_bf16(y.a);
            *reinterpret_cast<uint4 *>(dst + cb) = pack_bf16(y.b);
        }
        return;
    }

    // ---- one page of K or V of one head
    const int which = (int)(item % 2), h = (int)(item / 2 % (unsigned)B.Hkv);
    item /= 2 * (unsigned)B.Hkv;
    const int b = (int)(item / n_blocks), j = (int)(item % n_blocks);
    const Seq s = load_seq(B, b);
    if (!s.ok || (s.L > A.n_positions && A.rot > 0 && s.n > 0)) {
        if (tid == 0)
            atomicOr(&g_append_error, kErrMeta);
        return;
    }
    const int p_first = max(s.L - s.n, 0);          // first position written
    const int blk = p_first / B.P + j;
    const int p0 = max(p_first, blk * B.P);         // this block's new positions [p0, p1)
    const int p1 = min(s.L, (blk + 1) * B.P);
    if (s.n == 0 || p0 >= p1)
        return;
    const int page = __ldg(B.page_table + (int64_t)b * B.max_pages + blk);
    if (page < 0 || page >= B.n_pages) {
        if (tid == 0)
            atomicOr(&g_append_error, kErrMeta);
        return;
    }
    const T *src = static_cast<const T *>(which ? A.v : A.k);
    const int64_t stride = which ? A.v_stride : A.k_stride;
    const int64_t head = (int64_t)page * B.Hkv + h;
    uint8_t *codes = (which ? B.v : B.k) + head * B.P * kHd;
    float *scale = (which ? B.v_scale : B.k_scale) + head;
    const int first_row = s.row0 + s.n - s.L;       // token row of position 0

    Row16 x[PASSES];
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int pos = p0 + i * (NT / 8) + r;
        if (pos < p1) {
            const T *row = src + (int64_t)(first_row + pos) * stride + h * kHd;
            load8(row + ca, x[i].a);
            load8(row + cb, x[i].b);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int pos = p0 + i * (NT / 8) + r;
        if (pos < p1) {
            if (!which)
                rotate_row(x[i], A, u, pos);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                amax = fmaxf(amax, finite_abs(x[i].a[e], bad));
                amax = fmaxf(amax, finite_abs(x[i].b[e], bad));
            }
        }
    }
    if (bad)
        atomicOr(&g_append_error, kErrNonFinite);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    __shared__ float warp_max[NT / 32];
    if ((tid & 31) == 0)
        warp_max[tid >> 5] = amax;
    const bool fresh = p0 == blk * B.P;
    const float s_old = fresh ? 0.0f : *scale;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i)
        amax = fmaxf(amax, warp_max[i]);
    const float s_new = fmaxf(s_old, pow2_scale(amax));
    const float inv = __frcp_rn(s_new);             // exact: s_new is a power of two
    if (tid == 0)
        *scale = s_new;                             // every thread has read s_old
    if (!fresh && s_new > s_old) {                  // the page's other codes move to the new scale
        const float ratio = s_old * inv;
        const int lo = p0 - blk * B.P, hi = p1 - blk * B.P;
        for (int c = tid; c < B.P * kHd / 16; c += NT) {
            const int slot = c >> 3;
            if (slot >= lo && slot < hi)
                continue;
            uint4 *at = reinterpret_cast<uint4 *>(codes) + c;
            const uint4 w = *at;
            uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                in[e] = codes4(code_value(in[e] & 255) * ratio, code_value(in[e] >> 8 & 255) * ratio,
                               code_value(in[e] >> 16 & 255) * ratio, code_value(in[e] >> 24) * ratio);
            *at = make_uint4(in[0], in[1], in[2], in[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int pos = p0 + i * (NT / 8) + r;
        if (pos < p1) {
            float *a = x[i].a, *c = x[i].b;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = a[e] == a[e] ? a[e] * inv : 0.0f;   // NaN is held as 0
                c[e] = c[e] == c[e] ? c[e] * inv : 0.0f;
            }
            uint8_t *dst = codes + (pos - blk * B.P) * kHd;
            *reinterpret_cast<uint2 *>(dst + ca) =
                make_uint2(codes4(a[0], a[1], a[2], a[3]), codes4(a[4], a[5], a[6], a[7]));
            *reinterpret_cast<uint2 *>(dst + cb) =
                make_uint2(codes4(c[0], c[1], c[2], c[3]), codes4(c[4], c[5], c[6], c[7]));
        }
    }
}

template <typename T>
static cudaError_t launch_typed(const AppendArgs &a, cudaStream_t s)
{
    const Batch &B = a.b;
    // a call of n tokens touches at most this many pages of a sequence
    const int n_blocks = (int)(((int64_t)B.max_q + 2 * B.P - 2) / B.P);
    const int64_t cache_ctas = (int64_t)B.n_seq * n_blocks * B.Hkv * 2;
    const int q_ctas = a.q ? (int)(((int64_t)B.max_q * B.Hq + kQRows - 1) / kQRows) : 0;
    const int64_t ctas = cache_ctas + (int64_t)B.n_seq * q_ctas;
    if (ctas > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas);
    const unsigned nb = (unsigned)n_blocks, nc = (unsigned)cache_ctas, nq = (unsigned)q_ctas;
    switch (B.P) {
    case 16: append_kernel<T, 128, 1><<<grid, 128, 0, s>>>(a, nb, nc, nq); break;
    case 32: append_kernel<T, 256, 1><<<grid, 256, 0, s>>>(a, nb, nc, nq); break;
    case 64: append_kernel<T, 256, 2><<<grid, 256, 0, s>>>(a, nb, nc, nq); break;
    default: append_kernel<T, 256, 4><<<grid, 256, 0, s>>>(a, nb, nc, nq); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs &a, bool bf16, cudaStream_t s)
{
    return bf16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

cudaError_t take_append_error(int *code)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_error, sizeof(int));
    if (e == cudaSuccess && v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_append_error, &zero, sizeof(int));
    }
    *code = v;
    return e;
}

}  // namespace attn
}  // namespace gdn
