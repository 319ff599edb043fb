// attn_append.cu -- gdn_attn_append: rotate a batch's q and k by position,
// quantise k and v to e4m3 with one power-of-two scale per page and head, and
// write them into the paged cache.
//
// Bound by memory: every input element is read once, q written as bf16 and k, v
// as one byte. Work is cut so that no group of threads waits for another:
//   cache groups  a CTA (or a warp, where a call brings a sequence at most four
//                 tokens) per page the call touches, KV head, K or V. It sees all
//                 of the page's new tokens at once, so the page's scale is a
//                 reduction over values that stay in registers.
//   q groups      eight threads per (token, few heads).
// Eight threads share a row of 128, each with two 8-element pieces that hold the
// two members of 8 rotation pairs, so a pair never leaves its thread:
//   halves        pieces u*8 and rot/2 + u*8 while u < rot/16, then the 16
//                 unrotated elements rot + (u - rot/16)*16 ..;
//   interleaved   elements u*16 .. u*16 + 15.
// Either way thread u's angles are u*8 .. u*8 + 7 of the position's table row.
//
// A key's code is that of its exact rotation: the few values that 32 bits put on a rounding border are turned again
// and rounded to odd. The rotation of q is within about a unit of 32 bits before its one rounding to bf16.
//
// Measured: 4 x 8192 tokens, 16 q heads on 4, bf16: 74 us, 5.2 TB/s of the bytes it cannot do without. Its warps
// wait for loads (5.6 of 12 cycles an issue); 64 registers, four CTAs of 256 threads an SM, measured best (three
// CTAs: 76.7 us; 512 threads: 83 us; before the angles were shared by a token's heads: 102 us). The same in float32:
// 106 us, 5.5 TB/s, although its forms for more than four tokens a sequence spill (252 bytes a thread at pages of 16
// and 32, about 360 at 64 and 128). A single token: the call's 8 us on the host.
#include <cfloat>
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_append_error;

constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100

struct Row16 {
    float a[8], b[8];
};

// Eight elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 x, y;
    __device__ __forceinline__ void load(const float *p)
    {
        x = __ldg(reinterpret_cast<const float4 *>(p));
        y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    }
};
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    Raw8<float> r;
    r.load(p);
    r.get(v);
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
// along, so that the result is within about an ulp even where the terms cancel. An
// infinite product has no such error: it would be inf - inf, NaN. If FINAL, fmaxf drops
// that NaN, and the infinite sum stands whatever finite number is added. (4 x 8192 tokens:
// 73.7 us, 73.6 without, 75.2 in keys too.) Otherwise the NaN comes out, and turn_to_odd,
// which every row with a NaN meets, takes the plain sum.
template <bool FINAL>
__device__ __forceinline__ void rotate_pair(float &a, float &b, float c, float s)
{
    const float w = __fmul_rn(b, s), e = __fmaf_rn(-b, s, w);
    const float x = __fadd_rn(__fmaf_rn(a, c, -w), FINAL ? fmaxf(e, -FLT_MAX) : e);
    const float t = __fmul_rn(a, s), f = __fmaf_rn(a, s, -t);
    b = __fadd_rn(__fmaf_rn(b, c, t), FINAL ? fmaxf(f, -FLT_MAX) : f);
    a = x;
}

struct Angles {
    float c[8], s[8];
};

// Thread u's eight angles of a position.
__device__ __forceinline__ void load_angles(Angles &t, const AppendArgs &A, int u, int pos)
{
    if (u * 16 < A.rot) {
        const int64_t at = (int64_t)pos * (A.rot / 2) + u * 8;
        load8(A.cos + at, t.c);
        load8(A.sin + at, t.s);
    }
}

template <bool FINAL>
__device__ __forceinline__ void rotate_row(Row16 &r, const AppendArgs &A, int u, const Angles &t)
{
    if (u * 16 >= A.rot)
        return;
    if (A.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair<FINAL>(r.a[2 * i], r.a[2 * i + 1], t.c[i], t.s[i]);
            rotate_pair<FINAL>(r.b[2 * i], r.b[2 * i + 1], t.c[4 + i], t.s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rotate_pair<FINAL>(r.a[i], r.b[i], t.c[i], t.s[i]);
    }
}

// a*c - b*s rounded to odd: to the neighbour in 32 bits whose last bit is set, unless it is exact. Rounding that to
// e4m3 rounds the exact value, and a value just above 448 s stays above it; rounded to nearest, a value within 2^-25
// of itself of such a border would be taken to lie on it. The products are split into two numbers each and added
// with their errors. A sum that is not finite has no error: it is the plain one.
__device__ __forceinline__ float turn_to_odd(float a, float c, float b, float s)
{
    const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p), w = __fmul_rn(b, s), we = __fmaf_rn(b, s, -w);
    const float h = __fsub_rn(p, w), z = __fsub_rn(h, p);
    const float t = __fsub_rn(__fsub_rn(p, __fsub_rn(h, z)), __fadd_rn(w, z));
    const float l = __fadd_rn(t, __fsub_rn(pe, we));
    const float x = __fadd_rn(h, l), r = __fsub_rn(l, __fsub_rn(x, h));   // the exact value is x + r
    if (!(fabsf(r) > 0.0f))
        return r == r ? x : __fmaf_rn(a, c, -w);
    const int bits = __float_as_int(x);
    return bits & 1 ? x : __int_as_float((bits ^ __float_as_int(r)) < 0 ? bits - 1 : bits + 1);
}

// Whether a value's last 19 bits are within 2 of zero, as they are beside every border of e4m3 times a power of two:
// midpoints have four bits behind the leading one at most, 448 two, and rotate_pair is within about a unit. So are
// those of infinities and of NaN (0x7fffffff).
__device__ __forceinline__ bool beside_border(const Row16 &x)
{
    uint32_t m = ~0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        m = min(m, min((__float_as_uint(x.a[e]) + 2) & 0x7ffffu, (__float_as_uint(x.b[e]) + 2) & 0x7ffffu));
    return m <= 4;
}

__device__ __forceinline__ float load_again(const float *p) { return *const_cast<const volatile float *>(p); }
__device__ __forceinline__ float load_again(const __nv_bfloat16 *p)
{
    return __uint_as_float((uint32_t)*reinterpret_cast<const volatile unsigned short *>(p) << 16);
}

// rotate_row of this thread's pieces of `row`, rounded to odd; y holds rotate_row's result. Few rows come here, so
// inputs and angles are loaded again, one pair at a time, and cost the others no registers.
template <typename T>
__device__ __forceinline__ void rotate_row_to_odd(Row16 &y, const T *row, const AppendArgs &A, int u, int pos)
{
    const int64_t at = (int64_t)pos * (A.rot / 2) + u * 8;
    int ca, cb;
    pieces(u, A.rot, A.interleaved, ca, cb);
    auto pair = [&](float &ya, float &yb, int ia, int ib, int i) {
        const float a = load_again(row + ia), b = load_again(row + ib);
        const float c = load_again(A.cos + at + i), s = load_again(A.sin + at + i);
        ya = turn_to_odd(a, c, b, s);
        yb = turn_to_odd(b, c, -a, s);
    };
    if (A.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pair(y.a[2 * i], y.a[2 * i + 1], ca + 2 * i, ca + 2 * i + 1, i);
            pair(y.b[2 * i], y.b[2 * i + 1], cb + 2 * i, cb + 2 * i + 1, 4 + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            pair(y.a[i], y.b[i], ca + i, cb + i, i);
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

// FEW: a warp per page, head and K or V (a page gets at most four tokens), eight of them per CTA; otherwise a
// CTA each. HPT: q heads per thread, which share the token's angles.
template <typename T, int NT, int PASSES, bool FEW, int HPT>
__global__ void __launch_bounds__(NT, 1024 / NT) append_kernel(const __grid_constant__ AppendArgs A, unsigned n_blocks,
                                                    unsigned cache_items, unsigned cache_ctas, unsigned q_ctas)
{
    constexpr int kGroup = FEW ? 32 : NT, kTok = kGroup / 8;   // threads of a group, tokens per pass
    const Batch &B = A.b;
    const int tid = threadIdx.x, u = tid & 7;
    int ca, cb;
    pieces(u, A.rot, A.interleaved, ca, cb);
    wait_previous_grid();
    allow_next_grid();

    if (blockIdx.x >= cache_ctas) {   // ---- rotate q
        const unsigned item = blockIdx.x - cache_ctas;
        const int b = (int)(item / q_ctas), r = (int)(item % q_ctas) * (NT / 8) + (tid >> 3);
        const int groups = (B.Hq + HPT - 1) / HPT, tok = r / groups, h0 = (r - tok * groups) * HPT;
        const Seq s = load_seq(B, b);
        if (tok >= s.n || (s.L > A.n_positions && A.rot > 0))
            return;                   // the cache groups report positions past the table
        GDN_CHECK(g_append_error, b < B.n_seq && s.row0 + tok < B.n_tokens && h0 < B.Hq &&
                                      (A.rot == 0 || max(s.L - s.n + tok, 0) < A.n_positions));
        const T *src = static_cast<const T *>(A.q) + (int64_t)(s.row0 + tok) * A.q_stride + h0 * kHd;
        __nv_bfloat16 *dst =
            static_cast<__nv_bfloat16 *>(A.q_out) + ((int64_t)(s.row0 + tok) * B.Hq + h0) * kHd;
        Angles t;
        load_angles(t, A, u, max(s.L - s.n + tok, 0));
        constexpr int kAtOnce = HPT < 2 ? HPT : 2;
#pragma unroll 1
        for (int i0 = 0; i0 < HPT && h0 + i0 < B.Hq; i0 += kAtOnce) {
            Raw8<T> x[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (h0 + i0 + i < B.Hq) {
                    x[i][0].load(src + (i0 + i) * kHd + ca);
                    x[i][1].load(src + (i0 + i) * kHd + cb);
                }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (h0 + i0 + i < B.Hq) {
                    Row16 y;
                    x[i][0].get(y.a);
                    x[i][1].get(y.b);
                    rotate_row<true>(y, A, u, t);
                    *reinterpret_cast<uint4 *>(dst + (i0 + i) * kHd + ca) = pack_bf16(y.a);
                    *reinterpret_cast<uint4 *>(dst + (i0 + i) * kHd + cb) = pack_bf16(y.b);
                }
        }
        return;
    }

    // ---- one page of K or V of one head
    const int g = FEW ? tid & 31 : tid, r = g >> 3;
    unsigned item = FEW ? blockIdx.x * (NT / 32) + (tid >> 5) : blockIdx.x;
    if (item >= cache_items)
        return;
    const int which = (int)(item % 2), h = (int)(item / 2 % (unsigned)B.Hkv);
    item /= 2 * (unsigned)B.Hkv;
    const int b = (int)(item / n_blocks), j = (int)(item % n_blocks);
    const Seq s = load_seq(B, b);
    if (!s.ok || (s.L > A.n_positions && A.rot > 0 && s.n > 0)) {
        if (g == 0)
            atomicOr(&g_append_error, kErrMeta);
        return;
    }
    const int page_shift = 31 - __clz(B.P);
    const int p_first = max(s.L - s.n, 0);          // first position written
    const int blk = (p_first >> page_shift) + j;
    const int p0 = max(p_first, blk << page_shift); // this page's new positions [p0, p1)
    const int p1 = min(s.L, (blk + 1) << page_shift);
    if (s.n == 0 || p0 >= p1)
        return;
    GDN_CHECK(g_append_error, b < B.n_seq && h < B.Hkv && blk >= 0 && blk < B.max_pages && p1 - p0 <= PASSES * kTok &&
                                  s.row0 + s.n - s.L + p0 >= s.row0 && s.row0 + s.n - s.L + p1 <= B.n_tokens &&
                                  (A.rot == 0 || p1 <= A.n_positions));
    const int page = __ldg(B.page_table + (int64_t)b * B.max_pages + blk);
    const T *src = static_cast<const T *>(which ? A.v : A.k);
    const int64_t stride = which ? A.v_stride : A.k_stride;
    const int first_row = s.row0 + s.n - s.L;       // token row of position 0

    Raw8<T> raw[PASSES][2];
    Row16 x[PASSES];
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int pos = p0 + i * kTok + r;
        if (pos < p1) {
            const T *row = src + (int64_t)(first_row + pos) * stride + h * kHd;
            raw[i][0].load(row + ca);
            raw[i][1].load(row + cb);
        }
    }
    if (page < 0 || page >= B.n_pages) {
        if (g == 0)
            atomicOr(&g_append_error, kErrMeta);
        return;
    }
    const int64_t head = (int64_t)page * B.Hkv + h;
    uint8_t *codes = (which ? B.v : B.k) + head * B.P * kHd;
    float *scale = (which ? B.v_scale : B.k_scale) + head;
    const bool fresh = p0 == blk << page_shift;
    const float s_old = fresh ? 0.0f : *scale;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int pos = p0 + i * kTok + r;
        if (pos < p1) {
            raw[i][0].get(x[i].a);
            raw[i][1].get(x[i].b);
            if (!which) {
                Angles t;
                load_angles(t, A, u, pos);
                rotate_row<false>(x[i], A, u, t);
                if (u * 16 < A.rot && beside_border(x[i]))   // one row in some thousands
                    rotate_row_to_odd(x[i], src + (int64_t)(first_row + pos) * stride + h * kHd, A, u, pos);
            }
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
    if (!FEW) {
        __shared__ float warp_max[NT / 32];
        if ((tid & 31) == 0)
            warp_max[tid >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT / 32; ++i)
            amax = fmaxf(amax, warp_max[i]);
    } else {
        __syncwarp();
    }
    const float s_new = fmaxf(s_old, pow2_scale(amax));
    const float inv = __frcp_rn(s_new);             // exact: s_new is a power of two
    if (g == 0)
        *scale = s_new;                             // every thread has read s_old
    if (!fresh && s_new > s_old) {                  // the page's other codes move to the new scale
        const float ratio = s_old * inv;
        const int lo = p0 - (blk << page_shift), hi = p1 - (blk << page_shift);
#pragma unroll 1
        for (int c = g; c < B.P * kHd / 16; c += kGroup) {
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
        const int pos = p0 + i * kTok + r;
        if (pos < p1) {
            float *a = x[i].a, *c = x[i].b;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = a[e] == a[e] ? a[e] * inv : 0.0f;   // NaN is held as 0
                c[e] = c[e] == c[e] ? c[e] * inv : 0.0f;
            }
            uint8_t *dst = codes + (pos - (blk << page_shift)) * kHd;
            *reinterpret_cast<uint2 *>(dst + ca) =
                make_uint2(codes4(a[0], a[1], a[2], a[3]), codes4(a[4], a[5], a[6], a[7]));
            *reinterpret_cast<uint2 *>(dst + cb) =
                make_uint2(codes4(c[0], c[1], c[2], c[3]), codes4(c[4], c[5], c[6], c[7]));
        }
    }
}

template <typename T, int NT, int PASSES, bool FEW, int HPT>
static cudaError_t launch_form(const AppendArgs &a, cudaStream_t s)
{
    const Batch &B = a.b;
    // a call of n tokens touches at most this many pages of a sequence
    const int64_t n_blocks = ((int64_t)B.max_q + 2 * B.P - 2) / B.P;
    const int64_t items = (int64_t)B.n_seq * n_blocks * B.Hkv * 2;
    const int64_t cache_ctas = FEW ? (items + NT / 32 - 1) / (NT / 32) : items;
    const int64_t groups = (B.Hq + HPT - 1) / HPT;
    const int64_t q_ctas = a.q ? (B.max_q * groups + NT / 8 - 1) / (NT / 8) : 0;
    const int64_t ctas = cache_ctas + (int64_t)B.n_seq * q_ctas;
    if (items > 0x7fffffff || ctas > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel<T, NT, PASSES, FEW, HPT>, a, (unsigned)n_blocks, (unsigned)items,
                              (unsigned)cache_ctas, (unsigned)q_ctas);
}

template <typename T>
static cudaError_t launch_typed(const AppendArgs &a, cudaStream_t s)
{
    const Batch &B = a.b;
    if (B.max_q <= 4)
        return launch_form<T, 256, 1, true, 1>(a, s);
    switch (B.P) {
    case 16: return launch_form<T, 128, 1, false, 4>(a, s);
    case 32: return launch_form<T, 256, 1, false, 4>(a, s);
    case 64: return launch_form<T, 256, 2, false, 4>(a, s);
    default: return launch_form<T, 512, 2, false, 4>(a, s);
    }
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
