// attn_prefill.cu -- gdn_attn_prefill: attention of many tokens per sequence
// over the paged e4m3 cache.
//
// Mathematics. The (token, head of the group) rows of one KV head are taken 256
// at a time, as two tiles A and B of 128, against tiles of 128 keys. Scores are
// S = Q K^T with the key codes read as the pages lie in shared memory and q as
// two e4m3 numbers (q times a power of two is hi + lo exactly): two 8-bit
// products at twice the 16-bit rate, so K is never converted. The softmax runs
// online without looking for maxima: weights are 2^(s - m) with a reference m
// that starts at 0 and moves only when a tile's weights leave 2^-60 .. 2^60.
// Weights and sums are floating numbers of 8 exponent bits, so the reference
// costs range, not precision. Weights are rounded to bf16 (as many bits as the
// result has) and multiply V, converted exactly from codes to bf16 with its
// power-of-two page scale, O += P V, accumulated in 32 bits in tensor memory.
//
// Bound by the tensor core: 4 * 128 flops per visible (row, key). While it works
// on one tile, the other tile's 128 threads turn scores into weights. The grid
// has one CTA per SM; all (q block, key tile) pairs of the batch are cut into
// equal contiguous shares, and q blocks that span shares are joined by a second
// kernel, so causal and ragged blocks of any number fill the GPU.
//
// Measured: 4 x 8192 tokens, 16 q heads on 4: 861 us, 1.28 PFLOP/s. The products
// of a pair of tiles take 2051 cycles back to back; with the other roles' shared
// memory traffic and the chain scores, weights, output they take 2800 to 3000.
// 1024 tokens behind 32768, 32 heads on 4, cap 50: 624 us; two exponentials and half
// a reciprocal a score keep their pipe 56% busy, the tensor pipe is at 37%, issue
// slots at 55%: the rest is the chain's latency. Window 1000, 6 prompts: 84 us. A
// block there is 9.4 tiles of 2800 to 3000 cycles and about 12000 cycles for q and
// the output, 44 to 51 us for the 2.1 blocks a CTA gets; start, join and waits
// between them are the rest, not taken apart further.
// Loops are short on purpose: unrolled further, fetching instructions stalls them.
//
// Roles of a CTA (512 threads): warp 0 copies pages, warps 1 and 2 issue the
// products of tiles A and B, warp 3 walks the share (attn_share.cuh), warps 4-7
// and 8-11 split q and hold a row each of tiles A and B, warps 12-15 convert V.
#include "attn_share.cuh"
#include "attn_tc.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_attn_prefill_error;

namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;                    // q rows per block
constexpr int kOver = 6;                      // what a block costs besides its tiles, in tiles
constexpr int kWhole = 8;                     // most tiles of blocks that are not worth splitting
constexpr int kKs = 2, kVs = 2, kVb = 2;      // stages: K codes, V codes, V in bf16
constexpr uint32_t kQAt = 0;                  // [A, B][hi, lo] 128 rows of 128 bytes
constexpr uint32_t kKAt = kQAt + 4 * kTileBytes;
constexpr uint32_t kVAt = kKAt + kKs * kTileBytes;
constexpr uint32_t kBAt = kVAt + kVs * kTileBytes;
constexpr uint32_t kEnd = kBAt + kVb * 2 * kTileBytes;
constexpr uint32_t kTmemCols = 512;           // S of A, S of B, O of A, O of B: 128 each
constexpr float kMostSum = 0x1p60f, kLeastSum = 0x1p-60f;   // of weights against a reference that stays

template <int N>
__device__ __forceinline__ void registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

struct Shared {
    uint64_t k_full[kKs], k_free[kKs], v_full[kVs], v_free[kVs], b_full[kVb], b_free[kVb];
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_half[2], o_done[2], drain[2];
    uint32_t tmem;
    volatile int abort;
    ShareShared<kThreads> share;
    Ring ring;
    Seg now[8];                // the segment that each warp of rows is at
    float f[2][128];           // |scale| log2 e / (power of two of the q row)
};

// 32 columns of this thread's lane, without waiting; tmem_wait makes them usable.
__device__ __forceinline__ void tmem_get32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                   "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// The registers are operands of the wait, so nothing that uses them moves above it.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two codes (bytes 1 and 3 of x, the other bytes zero) as bf16 numbers times 2^-120: sign, then the
// code's 4 + 3 exponent and mantissa bits under bf16's 8 + 7, subnormals included.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t x)
{
    return ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <int CAP>
__device__ __forceinline__ float score(float s, float fk, float cap2, float inv_cap2)
{
    if constexpr (CAP != kNoCap)
        return cap2 * tanh_cap(s * fk * inv_cap2);
    else
        return s * fk;
}

// 16 columns of this thread's lane, without waiting, and the wait for them.
__device__ __forceinline__ void tmem_get16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}

// Which columns of the tile a row sees: [lo, hi], but for the pages in `bad` (bits).
struct RowMask {
    int lo, hi, page_shift;
    uint32_t bad;
    __device__ __forceinline__ uint32_t operator()(int q4) const   // bit e: column 32 q4 + e is visible
    {
        const int h = hi - 32 * q4, o = lo - 32 * q4;
        uint32_t v = h >= 31 ? 0xffffffffu : h < 0 ? 0u : (2u << h) - 1u;
        v &= o <= 0 ? 0xffffffffu : o > 31 ? 0u : 0xffffffffu << o;
        if (bad >> ((32 * q4) >> page_shift) & 1)
            v &= 0xffff0000u;
        if (bad >> ((32 * q4 + 16) >> page_shift) & 1)
            v &= 0x0000ffffu;
        return v;
    }
};

// What a score of 16 neighbouring columns is multiplied by: the row's factor and the page's scale.
struct RowFactor {
    float f, ks;               // ks of lane p: the tile's page p
    int page_shift;
    __device__ __forceinline__ float operator()(int sixteenth) const
    {
        return f * __shfl_sync(0xffffffffu, ks, (16 * sixteenth) >> page_shift);
    }
};

// Sixteen columns' weights, as bf16 pairs, against a reference; adds them to sum and returns the columns seen.
template <bool WHOLE>
__device__ __forceinline__ uint32_t weights16(uint32_t (&v)[16], uint32_t *y, int c, const RowMask &mask_of,
                                              const RowFactor &factor, uint64_t sub2, uint64_t (&sum)[2])
{
    const uint32_t mask = WHOLE ? 0xffffu : mask_of(c / 2) >> (16 * (c & 1)) & 0xffffu;
    const float fk = factor(c);
    const uint64_t fk2 = pack2(fk, fk);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float2 z = unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), fk2, sub2));
        z.x = ex2(z.x);
        z.y = ex2(z.y);
        if (!WHOLE) {
            z.x = mask >> e & 1 ? z.x : 0.0f;
            z.y = mask >> (e + 1) & 1 ? z.y : 0.0f;
        }
        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(z.x, z.y));
        y[e / 2] = pack_bf16x2(z.x, z.y);
    }
    return mask;
}

// Weights of a row against the reference as it is: one pass, no maximum. Each half of the tile (64 keys) is
// stored if every row of the warp is within range; otherwise its scores are left as they were and slow(half)
// takes the form that moves the reference. In range: the weights sum to at most 2^60, and those of the row so
// far to at least 2^-60 where it has seen a key, so that what the 8 exponent bits of weights and sums cannot
// hold is below 2^-60 of the row's total. first() is called once the first half's weights are in place.
template <bool WHOLE, typename S, typename H>
__device__ __forceinline__ void row_weights(uint32_t s_at, const RowMask &mask_of, const RowFactor &factor, float &ref,
                                            float &l, S slow, H first)
{
    uint32_t x[2][16], y[32];
    tmem_get16(s_at, x[0]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint64_t sum[2] = {0, 0};
        const uint64_t sub2 = pack2(-ref, -ref);
        uint32_t seen = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 4 * half + i;
            uint32_t(&v)[16] = x[c & 1];
            tmem_wait16(v);
            if (c < 7)
                tmem_get16(s_at + 16 * (c + 1), x[(c + 1) & 1]);
            seen |= weights16<WHOLE>(v, y + 8 * i, c, mask_of, factor, sub2, sum);
            if (c == 4)        // one step late: the store of the first half's weights has ended by itself
                first();
        }
        const float2 t = unpack2(add2(sum[0], sum[1]));
        const float add = t.x + t.y;
        if (__all_sync(0xffffffffu, add <= kMostSum && (l + add >= kLeastSum || seen == 0))) {
            l += add;
            tc::tmem_st16u(s_at + 32 * half, *reinterpret_cast<uint32_t(*)[16]>(y));
            tc::tmem_st16u(s_at + 32 * half + 16, *reinterpret_cast<uint32_t(*)[16]>(y + 16));
        } else {
            slow(half);
        }
    }
}

// 8 columns of this thread's lane.
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}

// Weights of a row whose scores are capped at no more than kMostCap: the weights themselves stay within the
// range of the numbers that hold them, so no reference is needed, and no maximum. In base 2 the capped score is
// c - 2 c / (1 + e^(2 s / cap)); its absolute error, c 2^-22, is far below a bf16 weight's rounding. One
// reciprocal serves two keys: exponents are held to 60, where tanh is 1.
template <bool WHOLE>
__device__ __forceinline__ float half_weights_capped(uint32_t s_at, int half_tile, const RowMask &mask_of,
                                                     const RowFactor &factor, float c)
{
    uint64_t sum[2] = {0, 0};
    const uint64_t one = pack2(1.0f, 1.0f), c2 = pack2(c, c), m2c = pack2(-2.0f * c, -2.0f * c);
    const float f = 2.0f * kLog2e / c;    // factor() gives base-2 scores: 2 log2 e s / cap = (2 log2 e / c) (s log2 e)
#pragma unroll 2
    for (int x = 4 * half_tile; x < 4 * half_tile + 4; ++x) {   // 16 columns at a time
        uint32_t v[16], y[8];
        tmem_get16(s_at + 16 * x, v);
        tmem_wait16(v);
        const uint32_t mask = WHOLE ? 0xffffu : mask_of(x / 2) >> (16 * (x & 1));
        const float fk = factor(x) * f;
        const uint64_t fk2 = pack2(fk, fk);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            float2 a = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            if (!WHOLE) {   // columns that are not seen may hold NaN, and pairs share a reciprocal
                a.x = mask >> i & 1 ? a.x : 0.0f;
                a.y = mask >> (i + 1) & 1 ? a.y : 0.0f;
            }
            a = unpack2(mul2(pack2(a.x, a.y), fk2));
            a = unpack2(add2(pack2(ex2(min_nan(a.x, 60.0f)), ex2(min_nan(a.y, 60.0f))), one));
            const float r = rcp(a.x * a.y);
            const float2 w = unpack2(fma2(mul2(pack2(r, r), pack2(a.y, a.x)), m2c, c2));
            float2 z = make_float2(ex2(w.x), ex2(w.y));
            if (!WHOLE) {
                z.x = mask >> i & 1 ? z.x : 0.0f;
                z.y = mask >> (i + 1) & 1 ? z.y : 0.0f;
            }
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(z.x, z.y));
            y[i / 2] = pack_bf16x2(z.x, z.y);
        }
        tmem_st8u(s_at + 8 * x, y);
    }
    const float2 t = unpack2(add2(sum[0], sum[1]));
    return t.x + t.y;
}

// 16 bytes to shared memory without passing through registers; zeros where `have` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}

// The largest visible score of this thread's row in half a tile, -inf for none. The cap is monotonic and
// factors are not negative, so each 16 columns' raw maximum stands for them.
template <int CAP>
__device__ __forceinline__ float half_max(uint32_t s_at, int half_tile, const RowMask &mask_of, const RowFactor &factor,
                                          float cap2, float inv_cap2)
{
    float top = -INFINITY;
#pragma unroll 1
    for (int q4 = 2 * half_tile; q4 < 2 * half_tile + 2; ++q4) {
        uint32_t v[32];
        tmem_get32(s_at + 32 * q4, v);
        tmem_wait32(v);
        const uint32_t mask = mask_of(q4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float mx[2];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float s = (mask >> (16 * half + e)) & 1 ? __uint_as_float(v[16 * half + e]) : -INFINITY;
                mx[e & 1] = e < 2 ? s : fmaxf(mx[e & 1], s);
            }
            const float most = fmaxf(mx[0], mx[1]);
            const float sc = score<CAP>(most, factor(2 * q4 + half), cap2, inv_cap2);
            top = fmaxf(top, most > -INFINITY ? sc : -INFINITY);
        }
    }
    return top;
}

// Weights of half a tile, 2^(score - sub), as bf16 pairs over the scores' columns; returns their sum. Weights
// of 32 keys take 16 columns, over scores already read.
template <int CAP>
__device__ __forceinline__ float half_weights_at(uint32_t s_at, int half_tile, const RowMask &mask_of,
                                                 const RowFactor &factor, float sub, float cap2, float inv_cap2)
{
    float sum = 0.0f;
#pragma unroll 1
    for (int q4 = 2 * half_tile; q4 < 2 * half_tile + 2; ++q4) {
        uint32_t v[32], y[16];
        tmem_get32(s_at + 32 * q4, v);
        tmem_wait32(v);
        const uint32_t mask = mask_of(q4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float fk = factor(2 * q4 + half);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float z[2];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const float s = __uint_as_float(v[16 * half + e + o]);
                    z[o] = ex2(CAP ? score<CAP>(s, fk, cap2, inv_cap2) - sub : fmaf(s, fk, -sub));
                    z[o] = (mask >> (16 * half + e + o)) & 1 ? z[o] : 0.0f;
                    sum += z[o];
                }
                y[8 * half + e / 2] = pack_bf16x2(z[0], z[1]);
            }
        }
        tc::tmem_st16u(s_at + 16 * q4, y);
    }
    return sum;
}

// Half a tile in the form that moves the reference: the maximum first. o_bar, where it is not 0, is the barrier
// (and parity) behind which O holds what the row has summed so far. Returns the reference and the sum.
// Not inlined: it is hardly ever run, and its four copies would crowd the loop that it stands in.
template <int CAP>
__device__ __noinline__ float2 slow_half(uint32_t s_at, uint32_t o_at, int half, RowMask mask_of, RowFactor factor,
                                         float ref, float l, float cap2, float inv_cap2, uint32_t o_bar,
                                         uint32_t o_parity, uint64_t lim, volatile int *abort)
{
    const float top = half_max<CAP>(s_at, half, mask_of, factor, cap2, inv_cap2);
    // up where a weight would pass 2^8, down to a row's first keys
    const bool move = top > ref + 8.0f || (l == 0.0f && top < ref && top > -INFINITY);
    if (__any_sync(0xffffffffu, move)) {
        const float to = move ? top : ref;
        const float a = move && l > 0.0f ? ex2(ref - to) : 1.0f;   // l = 0: so is O
        ref = to;
        l *= a;
        if (o_bar != 0) {
            if (!wait_phase(o_bar, o_parity, lim, abort))
                *abort = 1;
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll 1
            for (int q4 = 0; q4 < 8; ++q4) {
                uint32_t v[16];
                tmem_get16(o_at + 16 * q4, v);
                tmem_wait16(v);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
                tc::tmem_st16u(o_at + 16 * q4, v);
            }
        }
    }
    l += half_weights_at<CAP>(s_at, half, mask_of, factor, ref, cap2, inv_cap2);
    return make_float2(ref, l);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v)
{
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared sh;
    const Batch &B = A.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem_addr(dyn) + 1023u) & ~1023u;
    uint8_t *const mem = dyn + (base - tc::smem_addr(dyn));

    if (tid == 0) {
        auto init = [&](uint64_t &bar, uint32_t n) { tc::mbar_init(tc::smem_addr(&bar), n); };
        for (int i = 0; i < kKs; ++i)
            init(sh.k_full[i], 1), init(sh.k_free[i], 2);
        for (int i = 0; i < kVs; ++i)
            init(sh.v_full[i], 1), init(sh.v_free[i], 128);
        for (int i = 0; i < kVb; ++i)
            init(sh.b_full[i], 128), init(sh.b_free[i], 2);
        for (int i = 0; i < 2; ++i) {
            init(sh.q_full[i], 128);
            init(sh.s_full[i], 1);
            init(sh.p_half[i], 128), init(sh.p_full[i], 128);
            init(sh.o_half[i], 1), init(sh.o_done[i], 1);
            init(sh.drain[i], 1);
        }
        for (int i = 0; i < kRing; ++i)
            init(sh.ring.full[i], 1), init(sh.ring.free[i], kThreads / 32 - 1);   // every warp but the walker
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.abort = 0;
    }
    if (warp == 1)
        tc::tmem_alloc(tc::smem_addr(&sh.tmem), kTmemCols);
    if (tid == 96) {
        asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    }
    wait_previous_grid();
    Share share = {};
    if (B.n_seq > kFewSeqs)
        share = find_share<kRows, kOver, kWhole>(A, sh.share, tid, kThreads, [] { __syncthreads(); });
    PartMeta *const meta = reinterpret_cast<PartMeta *>(A.ws);
    float *const parts = part_slots(A.ws, gridDim.x);
    if (tid == 128)   // the thread that may describe a block later
        meta[blockIdx.x].owner = 0;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    allow_next_grid();

    const uint32_t tmem = sh.tmem;
    const uint64_t lim = A.wait_ns;
    const int page_shift = 31 - __clz(B.P);
    bool failed = false;
    // A wait that gives up stops the CTA's copies and products and ends every other wait; the loops
    // run on to their ends. For whole warps.
    auto wait = [&](const uint64_t &bar, uint32_t parity) {
        if (!wait_phase(tc::smem_addr(&bar), parity, lim, &sh.abort)) {
            sh.abort = 1;
            failed = true;
        }
        __syncwarp();
    };
    auto wait_first = [&](const uint64_t &bar, uint32_t parity) {   // the CTA's first, whose limit a test sets
        if (!wait_phase(tc::smem_addr(&bar), parity, A.first_wait_ns, &sh.abort)) {
            sh.abort = 1;
            failed = true;
        }
        __syncwarp();
    };
    auto arrive = [&](const uint64_t &bar) { tc::mbar_arrive(tc::smem_addr(&bar)); };

    // Registers move to the two groups of warps that hold rows: 128 (88 + 160 + 160 + 96) of the 65,536 that the
    // CTA starts with are 64,512.
    if (warp < 4) {
        registers_down<88>();
        if (warp == 0) {
            // ------------------------------------------------------------ pages to shared memory
            int c = 0, issued = 0;
            const int per_tile = kTile >> page_shift;
#pragma unroll 1
            for (int k = 0;; ++k) {
                const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
                if (w.nt == 0)
                    break;
                GDN_CHECK(g_attn_prefill_error, seg_in_range(A, w));
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
                const int pg_lo = w.lo >> page_shift, pg_hi = w.hi >> page_shift;
                auto page_of = [&](int t) {   // this lane's page of the tile, -1: none wanted, -2: bad
                    const int pg = (w.kt + t) * per_tile + lane;
                    if (t >= w.nt || lane >= per_tile || pg < pg_lo || pg > pg_hi)
                        return -1;
                    GDN_CHECK(g_attn_prefill_error, pg >= 0 && pg < B.max_pages);
                    const int p = __ldg(table + pg);
                    return p >= 0 && p < B.n_pages ? p : -2;
                };
                int page = page_of(0);
#pragma unroll 1
                for (int t = 0; t < w.nt; ++t, ++c) {
                    const int next = page_of(t + 1);
                    const bool have = page >= 0;
                    if (page == -2)
                        atomicOr(&g_attn_prefill_error, kErrMeta);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * B.P * kHd;
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {   // K, then V
                        const int stages = part ? kVs : kKs, st = c % stages;
                        if (c >= stages)
                            wait(part ? sh.v_free[st] : sh.k_free[st], (c / stages - 1) & 1);
                        if (__any_sync(0xffffffffu, sh.abort != 0))
                            continue;
                        const uint32_t bar = tc::smem_addr(part ? &sh.v_full[st] : &sh.k_full[st]);
                        if (lane == 0)
                            tc::mbar_expect_tx(bar, bytes);
                        __syncwarp();
                        if (have)
                            copy_page(part ? &map_v : &map_k,
                                      base + (part ? kVAt : kKAt) + st * kTileBytes + lane * B.P * kHd, bar,
                                      page * B.Hkv + w.h);
                        issued = 2 * c + part + 1;
                    }
                    page = next;
                }
            }
            // after a wait that gave up: the copies in flight land before the CTA ends
            for (int i = max(0, issued - 2 * kKs); i < issued && sh.abort; ++i) {
                const int tile = i / 2, stages = i & 1 ? kVs : kKs;
                if ((issued - 1 - i) / 2 < stages)
                    tc::mbar_wait_ns(tc::smem_addr(i & 1 ? &sh.v_full[tile % stages] : &sh.k_full[tile % stages]),
                                     (tile / stages) & 1, lim);
            }
        } else if (warp < 3) {
            // ------------------------------------------------------------ products: warp 1 those of tile A, warp
            // 2 those of B. A thread's products run in the order of their issue, so S of the next tile may be
            // issued behind the product that reads P from the same columns.
            const int m = warp - 1;
            const bool leader = elect_one();
            constexpr uint32_t idesc_s = idesc_e4m3(128, 128);
            constexpr uint32_t idesc_o = tc::idesc_f16(128, 128) | 1u << 7 | 1u << 10 | tc::kIdescTransB;
            const uint32_t s_at = tmem + m * 128, o_at = tmem + 256 + m * 128;
            const uint64_t q = tc::sdesc_sw128(base + kQAt + 2 * m * kTileBytes);
            int k = 0, c = 0, left = take_seg(sh.ring, 0, wait, &sh.abort).nt;   // segment, tile, its tiles left: of the next scores
            bool fresh = true, begin = true;  // whether that tile, and that of the next output, begins its segment
            auto issue_scores = [&] {         // by one thread
                const int ks = c % kKs;
                if (!sh.abort) {
                    const uint64_t kd = tc::sdesc_sw128(base + kKAt + ks * kTileBytes);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < 4; ++s)   // 32 bytes of the rows at a time
                            mma_e4m3(s_at, q + part * (kTileBytes >> 4) + 2 * s, kd + 2 * s, idesc_s, part + s > 0);
                }
                tc::mma_commit(tc::smem_addr(&sh.s_full[m]));
                tc::mma_commit(tc::smem_addr(&sh.k_free[ks]));
            };
#pragma unroll 1
            for (int j = -1; j < c; ++j) {    // output of tile j, scores of tile j + 1
                const bool more = left > 0;
                if (more && c == 0)
                    wait_first(sh.k_full[0], 0);
                else if (more)
                    wait(sh.k_full[c % kKs], (c / kKs) & 1);
                if (j >= 0) {
                    const int vb = j % kVb;
                    wait(sh.b_full[vb], (j / kVb) & 1);
                    wait(sh.p_half[m], j & 1);
                    tc::fence_after_sync();
                    // 16 keys at a time: 8 columns of P, 2 KB of V; the first 64 while the others' weights form
                    const uint64_t v = tc::sdesc_sw128_mn(base + kBAt + vb * 2 * kTileBytes, kTileBytes, 1024);
                    if (leader) {
                        if (!sh.abort) {
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                tc::mma_f16_ta(o_at, s_at + 8 * s, v + 128 * s, idesc_o, s > 0 || !begin);
                        }
                        tc::mma_commit(tc::smem_addr(&sh.o_half[m]));
                    }
                    __syncwarp();
                    wait(sh.p_full[m], j & 1);
                    tc::fence_after_sync();
                    if (leader) {
                        if (!sh.abort) {
#pragma unroll
                            for (int s = 4; s < 8; ++s)
                                tc::mma_f16_ta(o_at, s_at + 8 * s, v + 128 * s, idesc_o, 1);
                        }
                        if (more && !fresh)
                            issue_scores();
                        tc::mma_commit(tc::smem_addr(&sh.o_done[m]));
                        tc::mma_commit(tc::smem_addr(&sh.b_free[vb]));
                    }
                    __syncwarp();
                }
                if (more && (fresh || j < 0)) {
                    wait(sh.q_full[m], k & 1);
                    tc::fence_after_sync();
                    if (leader)
                        issue_scores();
                    __syncwarp();
                }
                begin = fresh;
                if (more) {
                    ++c;
                    fresh = --left == 0;
                    if (fresh)
                        left = take_seg(sh.ring, ++k, wait, &sh.abort).nt;
                }
            }
            if (leader) {   // every product, and every arrival that a commit still owes, ends before the CTA does
                tc::mma_commit(tc::smem_addr(&sh.drain[m]));
                tc::mbar_wait_ns(tc::smem_addr(&sh.drain[m]), 0, lim);
            }
            __syncwarp();
        } else if (warp == 3) {
            if (B.n_seq <= kFewSeqs)
                share = find_share<kRows, kOver, kWhole>(A, sh.share, lane, 32, [] { __syncwarp(); });
            walk_share<kRows, kOver>(A, share, sh.ring, wait, &sh.abort);
            clear_empty(A, &g_attn_prefill_error);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ scores to weights: a row per thread
        registers_up<160>();
        const int m = (warp - 4) >> 2, row = (tid - 128) & 127, x = m * 128 + row;
        const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + m * 128 + lane_at, o_at = tmem + 256 + m * 128 + lane_at;
        const int per_tile = kTile >> page_shift;
        const int G = B.G, inv_G = 65536 / G + 1;   // y / G = y * inv_G >> 16 for y below 4096
        const float cap2 = A.softcap * kLog2e, inv_cap2 = CAP == kAnyCap ? 1.0f / cap2 : 0.0f;
        const float f_scale = fabsf(A.scale) * (0.5f * kLog2e), sign = A.scale < 0.0f ? -1.0f : 1.0f;
        int c = 0;
        Seg &w = sh.now[warp - 4];   // in shared memory: the loop over tiles has no registers to spare for it
        float ref = 0.0f, l = 0.0f;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg nx = take_seg(sh.ring, k, wait, &sh.abort);
            if (nx.nt > 0) {
                // The next segment's q rows, 32 by each warp, while the last segment's last product runs (the
                // products that read that segment's q are done: its scores were here). A row's bf16 pieces
                // land where its own two e4m3 rows will lie, dimensions 0-63 in hi's place, 64-127 in lo's.
                const uint32_t at = kQAt + 2 * m * kTileBytes;
                const int row_w = (warp & 3) * 32;
                const int y = nx.rem0 + m * 128 + row, dt = y * inv_G >> 16, t = nx.tok0 + dt;
                GDN_CHECK(g_attn_prefill_error, seg_in_range(A, nx) && y < 4096 && y - dt * G < G &&
                                                    (t >= nx.n || nx.row0 + t < B.n_tokens));
                const uint64_t mine = t < nx.n ? reinterpret_cast<uint64_t>(
                                                     static_cast<const __nv_bfloat16 *>(A.q) +
                                                     (int64_t)(nx.row0 + t) * A.q_stride + (nx.h * G + y - dt * G) * kHd)
                                               : 0;
                const int piece = lane & 15;
                const uint32_t dst = base + at + (piece >> 3) * kTileBytes;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int from = 2 * i + (lane >> 4), rr = row_w + from;
                    const uint64_t src = __shfl_sync(0xffffffffu, mine, from);
                    copy16(dst + (rr >> 3) * 1024 + (rr & 7) * 128 + (((piece & 7) ^ (rr & 7)) << 4),
                           src ? reinterpret_cast<const uint4 *>(src) + piece : static_cast<const uint4 *>(A.q),
                           src != 0);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                const int u = lane & 7;
#pragma unroll 2
                for (int rr = row_w + (lane >> 3); rr < row_w + 32; rr += 4) {
                    uint8_t *at_row = mem + at + (rr >> 3) * 1024 + (rr & 7) * 128;
                    const uint8_t *raw = at_row + (u >> 2) * kTileBytes;   // elements 16 u ..: pieces 2 u, 2 u + 1
                    float v[16];
                    unpack_q16(*reinterpret_cast<const uint4 *>(raw + ((((2 * u) & 7) ^ (rr & 7)) << 4)),
                               *reinterpret_cast<const uint4 *>(raw + ((((2 * u + 1) & 7) ^ (rr & 7)) << 4)), v);
                    float top = 0.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                    for (int i = 1; i < 8; i <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                    __syncwarp();   // the row is read before it is overwritten
                    store_q16(at_row + ((u ^ (rr & 7)) << 4), kTileBytes, v, sign * q_factor(top));
                    if (u == 0)
                        sh.f[m][rr] = f_scale * pow2i(1 - q_exponent(top));
                }
                tc::fence_smem_to_async();
                __syncwarp();
                arrive(sh.q_full[m]);
            }
            if (k > 0) {
                // ---- the last segment's rows
                wait(sh.o_done[m], (c - 1) & 1);
                tc::fence_after_sync();
                const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
                const int y = w.rem0 + x, dt = y * inv_G >> 16, tok = w.tok0 + dt, head = y - dt * G;
                const bool live = tok < w.n, joined = !w.whole;
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(A.out) +
                                                       ((int64_t)(w.row0 + tok) * B.Hq + w.h * G + head) * kHd);
                float *part = parts + ((size_t)(2 * blockIdx.x + (w.begins ? 1 : 0)) * kRows + x) * kPartRow;
                GDN_CHECK(g_attn_prefill_error, seg_in_range(A, w) && x < kRows && head >= 0 && head < G &&
                                                    (!live || w.row0 + tok < B.n_tokens));
#pragma unroll 1
                for (int q4 = 0; q4 < 4; ++q4) {
                    uint32_t v[32];
                    tmem_get32(o_at + 32 * q4, v);
                    tmem_wait32(v);
                    if (joined) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<uint4 *>(part)[8 * q4 + e] =
                                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t y[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                y[i] = pack_bf16x2(__uint_as_float(v[8 * e + 2 * i]) * inv,
                                                   __uint_as_float(v[8 * e + 2 * i + 1]) * inv);
                            out[4 * q4 + e] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if (joined) {
                    *reinterpret_cast<float2 *>(part + kHd) = make_float2(l, l == 0.0f ? kNoRef : ref);
                    if (w.begins && x == 0)
                        meta[blockIdx.x] = {w.b, w.h, w.blk, w.last_cta, 1, {}};
                }
                tc::fence_before_sync();
            }
            if (nx.nt == 0)
                break;
            __syncwarp();
            if (lane == 0)
                w = nx;
            __syncwarp();
            const int tok = nx.tok0 + ((nx.rem0 + x) * inv_G >> 16);
            const int limit = tok < nx.n ? nx.first + tok : -1;   // last position the row sees
            // positions of the tile's first and last row, for key tiles that all of its rows see whole
            const int tok_a = nx.tok0 + ((nx.rem0 + m * 128) * inv_G >> 16);
            const int tok_b = nx.tok0 + ((nx.rem0 + m * 128 + 127) * inv_G >> 16);
            const int all_to = tok_b < nx.n ? nx.first + tok_a : -1, all_from = nx.first + tok_b - A.window;
            const int32_t *table = B.page_table + (int64_t)nx.b * B.max_pages;
            const int pg_lo = nx.lo >> page_shift, pg_hi = nx.hi >> page_shift;
            // lane p: scale of the tile's page p; 0 marks a page the table does not have
            auto page_at = [&](int t) {
                const int pg = (nx.kt + t) * per_tile + lane;
                return t < nx.nt && lane < per_tile && pg >= pg_lo && pg <= pg_hi ? __ldg(table + pg) : -3;
            };
            auto scale_at = [&](int p) {
                return p == -3 ? 1.0f
                               : p >= 0 && p < B.n_pages ? __ldg(B.k_scale + (int64_t)p * B.Hkv + nx.h) : 0.0f;
            };
            int p_far = page_at(1);
            float ks_next = scale_at(page_at(0));
            const float f = sh.f[m][row];
            const int nt = nx.nt, kt = nx.kt;
            ref = 0.0f;
            l = 0.0f;
#pragma unroll 1
            for (int t = 0; t < nt; ++t, ++c) {
                const float ks = ks_next;
                ks_next = scale_at(p_far);
                p_far = page_at(t + 2);
                const uint32_t bad = __ballot_sync(0xffffffffu, ks == 0.0f);
                const int j0 = (kt + t) * kTile;
                const bool whole = j0 + kTile - 1 <= all_to && j0 > all_from && bad == 0;
                wait(sh.s_full[m], c & 1);
                tc::fence_after_sync();
                const RowMask mask_of = {limit - A.window + 1 - j0, limit - j0, page_shift, bad};
                const RowFactor factor = {f, ks, page_shift};
                auto first = [&] {     // the first 64 keys' weights are there
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    arrive(sh.p_half[m]);
                };
                auto slow = [&](int half) {
                    const uint32_t bar = half ? tc::smem_addr(&sh.o_half[m]) : t > 0 ? tc::smem_addr(&sh.o_done[m]) : 0u;
                    const float2 r = slow_half<CAP>(s_at, o_at, half, mask_of, factor, ref, l, cap2, inv_cap2, bar,
                                                    (half ? c : c - 1) & 1, lim, &sh.abort);
                    ref = r.x;
                    l = r.y;
                };
                if constexpr (CAP == kNoCap) {
                    if (whole)
                        row_weights<true>(s_at, mask_of, factor, ref, l, slow, first);
                    else
                        row_weights<false>(s_at, mask_of, factor, ref, l, slow, first);
                } else {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if constexpr (CAP == kAnyCap)
                            slow(half);
                        else
                            l += whole ? half_weights_capped<true>(s_at, half, mask_of, factor, cap2)
                                       : half_weights_capped<false>(s_at, half, mask_of, factor, cap2);
                        if (half == 0)
                            first();
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                arrive(sh.p_full[m]);
            }
        }
    } else {
        // ------------------------------------------------------------ V to bf16: a key per thread
        registers_down<96>();
        const int t128 = tid - 384;
        int c = 0;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
            if (w.nt == 0)
                break;
            const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
            auto page_at = [&](int t) {
                const int j = (w.kt + t) * kTile + t128;
                if (t >= w.nt || j < w.lo || j > w.hi)
                    return -1;
                GDN_CHECK(g_attn_prefill_error, j >= 0 && j >> page_shift < B.max_pages);
                const int p = __ldg(table + (j >> page_shift));
                return p >= 0 && p < B.n_pages ? p : -1;
            };
            auto scale_at = [&](int p) {
                return p >= 0 ? __ldg(B.v_scale + (int64_t)p * B.Hkv + w.h) : 0.0f;
            };
            int p_next = page_at(0), p_far = page_at(1);
            float vs_next = scale_at(p_next);
#pragma unroll 1
            for (int t = 0; t < w.nt; ++t, ++c) {
                const bool dead = p_next < 0;    // holds anything: its row is zero
                const float vs = vs_next;
                p_next = p_far;
                vs_next = scale_at(p_next);
                p_far = page_at(t + 2);
                // 2^120 vs in two factors that bf16 holds
                const int e = dead ? 0 : (int)(__float_as_uint(vs) >> 23) - 127 + 120;
                const int e1 = max(-126, min(e, 127)), e2 = e - e1;
                const uint32_t f1 = (uint32_t)(e1 + 127) << 7 | (uint32_t)(e1 + 127) << 23;
                const uint32_t f2 = (uint32_t)(e2 + 127) << 7 | (uint32_t)(e2 + 127) << 23;
                const int vst = c % kVs, vb = c % kVb;
                if (c >= kVb)
                    wait(sh.b_free[vb], (c / kVb - 1) & 1);
                wait(sh.v_full[vst], (c / kVs) & 1);
                const uint8_t *src = mem + kVAt + vst * kTileBytes + t128 * kHd;
                uint8_t *dst = mem + kBAt + vb * 2 * kTileBytes + (t128 >> 3) * 1024 + (t128 & 7) * 128;
#pragma unroll 1   // two or four pieces in flight are slower (865 against 896 and 930 us): their code crowds the others out
                for (int i = 0; i < 8; ++i) {
                    const uint4 raw = dead ? make_uint4(0, 0, 0, 0)
                                           : *reinterpret_cast<const uint4 *>(src + ((i ^ (t128 & 7)) << 4));
                    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
                    uint32_t o[8];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        o[2 * z] = mul_bf16x2(codes_bf16(__byte_perm(in[z], 0, 0x1404)), f1);
                        o[2 * z + 1] = mul_bf16x2(codes_bf16(__byte_perm(in[z], 0, 0x3424)), f1);
                    }
                    if (e2 != 0) {
#pragma unroll
                        for (int z = 0; z < 8; ++z)
                            o[z] = mul_bf16x2(o[z], f2);
                    }
                    // dimensions 16 i .. 16 i + 15: two 16-byte pieces of half i / 4
                    uint8_t *half = dst + (i >> 2) * kTileBytes;
                    const int p0 = (2 * i) & 7;
                    *reinterpret_cast<uint4 *>(half + ((p0 ^ (t128 & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(half + (((p0 + 1) ^ (t128 & 7)) << 4)) =
                        make_uint4(o[4], o[5], o[6], o[7]);
                }
                arrive(sh.v_free[vst]);
                tc::fence_smem_to_async();
                arrive(sh.b_full[vb]);
            }
        }
    }
    if (failed || sh.abort)
        atomicOr(&g_attn_prefill_error, kErrWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1)
        tc::tmem_dealloc(tmem, kTmemCols);
}

template <int CAP>
cudaError_t launch_cap(const AttnArgs &a, int grid, bool may_split, cudaStream_t s)
{
    CUtensorMap mk, mv;
    if (!encode_cache_map(&mk, a.b, a.b.k) || !encode_cache_map(&mv, a.b, a.b.v))
        return cudaErrorInvalidValue;
    constexpr int smem = kEnd + 1024;
    cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, attn_prefill_kernel<CAP>, a, mk, mv)) != cudaSuccess)
        return e;
    return may_split ? launch_join(a, grid, kRows, s) : cudaSuccess;
}

}  // namespace

size_t prefill_workspace_bytes(int sms) { return part_bytes((size_t)sms, kRows); }

cudaError_t launch_prefill(const AttnArgs &args, cudaStream_t s)
{
    AttnArgs a = args;
    const Batch &b = a.b;
    if (a.window == 0 || a.window > kNoWindow)
        a.window = kNoWindow;
    if (most_units(b, kRows, kOver) > kMostUnits)
        return cudaErrorInvalidConfiguration;
    const int64_t tiles = ((int64_t)b.max_pages * b.P + kTile - 1) / kTile;
    const int64_t blocks = ((int64_t)b.max_q * b.G + kRows - 1) / kRows * b.Hkv * b.n_seq;
    const int64_t units = tiles >= a.sm_count || blocks >= a.sm_count ? a.sm_count : (tiles + kOver) * blocks;
    const int grid = (int)(units < a.sm_count ? units : a.sm_count);
    // the kernel decides by the lengths; where the page table's width decides already, nothing is ever joined
    const bool may_split = tiles > kWhole || blocks > grid || b.n_seq > kFewSeqs;
    switch (cap_mode(a.softcap)) {
    case kNoCap: return launch_cap<kNoCap>(a, grid, may_split, s);
    case kLowCap: return launch_cap<kLowCap>(a, grid, may_split, s);
    default: return launch_cap<kAnyCap>(a, grid, may_split, s);
    }
}

cudaError_t take_prefill_error(int *code)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_prefill_error, sizeof(int));
    if (e == cudaSuccess && v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_attn_prefill_error, &zero, sizeof(int));
    }
    *code = v;
    return e;
}

}  // namespace attn
}  // namespace gdn
