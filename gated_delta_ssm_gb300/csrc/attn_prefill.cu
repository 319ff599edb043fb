// attn_prefill.cu -- gdn_attn_prefill: attention of many tokens per sequence
// over the paged e4m3 cache.
//
// Mathematics. The (token, head of the group) rows of one KV head are taken 256
// at a time, as two tiles A and B of 128, against tiles of 128 keys. Scores are
// S = Q K^T with the key codes read as the pages lie in shared memory and q as
// two e4m3 numbers (q times a power of two is hi + lo exactly): two 8-bit
// products at twice the 16-bit rate, so K is never converted. The softmax runs
// online with a lazy reference m: weights are 2^(s - m) and m moves only when a
// row's maximum exceeds it by 2^8, which bf16 weights and 32-bit sums hold
// without loss; output rows are rescaled then. Weights are rounded to bf16 (as
// many bits as the result has) and multiply V, converted exactly from codes to
// bf16 with its power-of-two page scale, O += P V, accumulated in 32 bits in
// tensor memory.
//
// Bound by the tensor core: 4 * 128 flops per visible (row, key). While it works
// on one tile, the other tile's 128 threads turn scores into weights. The grid
// has one CTA per SM; all (q block, key tile) pairs of the batch are cut into
// equal contiguous shares, and q blocks that span shares are joined by a second
// kernel, so causal and ragged blocks of any number fill the GPU.
//
// Roles of a CTA (512 threads): warp 0 copies pages, warps 1 and 2 issue the
// products of tiles A and B, warp 3 clears the outputs of sequences without
// keys, warps 4-7 and 8-11 split q and hold a row each of tiles A and B, warps
// 12-15 convert V.
#include "attn_tc.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_attn_prefill_error;

namespace {

constexpr int kThreads = 512;
constexpr int kRows = 256;                    // q rows per block
constexpr int kKs = 3, kVs = 2, kVb = 2;      // stages: K codes, V codes, V in bf16
constexpr uint32_t kQAt = 0;                  // [A, B][hi, lo] 128 rows of 128 bytes
constexpr uint32_t kKAt = kQAt + 4 * kTileBytes;
constexpr uint32_t kVAt = kKAt + kKs * kTileBytes;
constexpr uint32_t kBAt = kVAt + kVs * kTileBytes;
constexpr uint32_t kEnd = kBAt + kVb * 2 * kTileBytes;
constexpr uint32_t kTmemCols = 512;           // S of A, S of B, O of A, O of B: 128 each
// The reference moves when a row's weights of one tile sum to more than this: weights and sums are floating
// numbers of 8 exponent bits, so a reference that lags behind costs no precision, only range.
constexpr float kSlack = 8.0f, kSlackSum = 65536.0f;   // 128 weights of at most 2^8 sum to 2^15

struct Shared {
    uint64_t k_full[kKs], k_free[kKs], v_full[kVs], v_free[kVs], b_full[kVb], b_free[kVb];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], drain[2];
    uint32_t tmem;
    volatile int abort;
    int64_t warp_sum[kThreads / 32];
    int64_t start_off;         // the share's first unit, within its sequence
    int64_t head_units;        // units of one KV head of that sequence
    int start_b, start_h, start_q, start_t;
    float f[2][128];           // |scale| log2 e / (power of two of the q row)
};

// A sequence and its q blocks.
struct Blocks {
    Seq s;
    int first;                 // position of its first row
    int n;                     // q blocks, 0 where there are no keys
};

__device__ __forceinline__ Blocks seq_blocks(const AttnArgs &A, int b)
{
    Blocks q;
    q.s = load_seq(A.b, b);
    q.first = q.s.L - q.s.n;
    q.n = q.s.L > 0 ? (int)(((int64_t)q.s.n * A.b.G + kRows - 1) / kRows) : 0;
    return q;
}

// Key tiles of q block i: from the first that its first row sees to the last that its last row sees.
__device__ __forceinline__ void block_tiles(const AttnArgs &A, const Blocks &q, int i, int &t0, int &n)
{
    const int G = A.b.G;
    const int tok0 = i * kRows / G, tok1 = min((i * kRows + kRows - 1) / G, q.s.n - 1);
    t0 = max(0, q.first + tok0 - A.window + 1) / kTile;
    n = max(0, q.first + tok1) / kTile + 1 - t0;
}

// A CTA's share: segments (sequence, KV head, q block, tiles [t, end) counted from the block's first).
struct Walk {
    int b, h, i, t, end, t0, n, left;
    Blocks q;
    __device__ __forceinline__ bool begins() const { return t == 0; }
    __device__ __forceinline__ bool ends() const { return end == n; }
    __device__ __forceinline__ void cut(const AttnArgs &A)
    {
        block_tiles(A, q, i, t0, n);
        end = min(n, t + left);
    }
    __device__ __forceinline__ bool next(const AttnArgs &A)
    {
        left -= end - t;
        if (left <= 0)
            return false;
        t = 0;
        if (++i == q.n) {
            i = 0;
            if (++h == A.b.Hkv) {
                h = 0;
                do {
                    if (++b >= A.b.n_seq)
                        return false;
                    q = seq_blocks(A, b);
                } while (q.n == 0);
            }
        }
        cut(A);
        return true;
    }
};

__device__ __forceinline__ Walk walk_start(const AttnArgs &A, const Shared &sh, int count)
{
    Walk w;
    w.b = sh.start_b;
    w.h = sh.start_h;
    w.i = sh.start_q;
    w.t = sh.start_t;
    w.left = count;
    w.q = seq_blocks(A, w.b);
    w.cut(A);
    return w;
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

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

template <bool CAP>
__device__ __forceinline__ float score(float s, float fk, float cap2, float inv_cap2)
{
    if constexpr (CAP)
        return cap2 * tanh_cap(s * fk * inv_cap2);
    else
        return s * fk;
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

// Weights of a row that sees the whole tile, against the reference as it is: one pass, no maximum. They are
// stored if every row of the warp stayed within 2^kSlack summed; otherwise the scores are left as they were
// and the caller takes the form that moves the reference.
template <bool CAP, typename F>
__device__ __forceinline__ bool row_weights_once(uint32_t s_at, F factor, float ref, float &l, float cap2,
                                                 float inv_cap2)
{
    uint32_t x[2][16], y[64];
    uint64_t sum[2] = {0, 0};
    const uint64_t sub2 = pack2(-ref, -ref);
    tmem_get16(s_at, x[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t(&v)[16] = x[c & 1];
        tmem_wait16(v);
        if (c < 7)
            tmem_get16(s_at + 16 * (c + 1), x[(c + 1) & 1]);
        const float fk = factor(c);
        const uint64_t fk2 = pack2(fk, fk);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float s0 = __uint_as_float(v[e]), s1 = __uint_as_float(v[e + 1]);
            float2 z;
            if constexpr (CAP) {
                z.x = score<CAP>(s0, fk, cap2, inv_cap2) - ref;
                z.y = score<CAP>(s1, fk, cap2, inv_cap2) - ref;
            } else {
                z = unpack2(fma2(pack2(s0, s1), fk2, sub2));
            }
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(z.x, z.y));
            y[8 * c + e / 2] = pack_bf16x2(z.x, z.y);
        }
    }
    const float2 t = unpack2(add2(sum[0], sum[1]));
    const float add = t.x + t.y;
    if (!__all_sync(0xffffffffu, add <= kSlackSum))
        return false;
    l += add;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        tc::tmem_st16u(s_at + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(y + 16 * c));
    return true;
}

// 16 bytes to shared memory without passing through registers; zeros where `have` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}

// The largest visible score of this thread's row of the tile (128 columns at s_at), -inf for none. The cap
// is monotonic and factors are not negative, so each 16 columns' raw maximum stands for them.
template <bool CAP, bool WHOLE, typename M, typename F>
__device__ __forceinline__ float row_max(uint32_t s_at, M mask_of, F factor, float cap2, float inv_cap2)
{
    float top = -INFINITY;
#pragma unroll 1
    for (int q2 = 0; q2 < 2; ++q2) {
        uint32_t v[2][32];
        tmem_get32(s_at + 64 * q2, v[0]);
        tmem_get32(s_at + 64 * q2 + 32, v[1]);
        tmem_wait32(v[0]);
        tmem_wait32(v[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t mask = WHOLE ? 0xffffffffu : mask_of(2 * q2 + i);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float mx[2];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float s = __uint_as_float(v[i][16 * half + e]);
                    if (!WHOLE)
                        s = (mask >> (16 * half + e)) & 1 ? s : -INFINITY;
                    mx[e & 1] = e < 2 ? s : fmaxf(mx[e & 1], s);
                }
                const float most = fmaxf(mx[0], mx[1]);
                const float fk = factor(4 * q2 + 2 * i + half);
                const float sc = score<CAP>(most, fk, cap2, inv_cap2);
                top = fmaxf(top, WHOLE || most > -INFINITY ? sc : -INFINITY);
            }
        }
    }
    return top;
}

// Weights of the row, 2^(score - sub), as bf16 pairs over the scores' columns; returns their sum. Weights
// of 32 keys take 16 columns, over scores already read.
template <bool CAP, bool WHOLE, typename M, typename F>
__device__ __forceinline__ float row_weights(uint32_t s_at, M mask_of, F factor, float sub, float cap2,
                                             float inv_cap2)
{
    uint64_t sum[2] = {0, 0};
    const uint64_t sub2 = pack2(-sub, -sub);
#pragma unroll 1
    for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t v[32];
        tmem_get32(s_at + 32 * q4, v);
        tmem_wait32(v);
        const uint32_t mask = WHOLE ? 0xffffffffu : mask_of(q4);
        uint32_t y[16];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float fk = factor(2 * q4 + half);
            const uint64_t fk2 = pack2(fk, fk);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float s0 = __uint_as_float(v[16 * half + e]), s1 = __uint_as_float(v[16 * half + e + 1]);
                float2 z;
                if constexpr (CAP) {
                    z.x = score<CAP>(s0, fk, cap2, inv_cap2) - sub;
                    z.y = score<CAP>(s1, fk, cap2, inv_cap2) - sub;
                } else {
                    z = unpack2(fma2(pack2(s0, s1), fk2, sub2));
                }
                z.x = ex2(z.x);
                z.y = ex2(z.y);
                if (!WHOLE) {
                    z.x = (mask >> (16 * half + e)) & 1 ? z.x : 0.0f;
                    z.y = (mask >> (16 * half + e + 1)) & 1 ? z.y : 0.0f;
                }
                sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(z.x, z.y));
                y[8 * half + e / 2] = pack_bf16x2(z.x, z.y);
            }
        }
        tc::tmem_st16u(s_at + 16 * q4, y);
    }
    const float2 t = unpack2(add2(sum[0], sum[1]));
    return t.x + t.y;
}

template <bool CAP>
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
            init(sh.p_full[i], 128);
            init(sh.o_done[i], 1);
            init(sh.drain[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.abort = 0;
        sh.start_b = 0;
    }
    if (warp == 1)
        tc::tmem_alloc(tc::smem_addr(&sh.tmem), kTmemCols);
    wait_previous_grid();

    // ---- the batch's (q block, key tile) units, and where this CTA's share of them begins. A group of
    // `g` neighbouring lanes counts one sequence, or a thread several where there are more than threads.
    int g = 1;
    while (g < 32 && (int64_t)B.n_seq * g * 2 <= kThreads)
        g *= 2;
    const int per = g > 1 ? 1 : (B.n_seq + kThreads - 1) / kThreads;
    const int first_b = (tid / g) * per, sub = tid % g;
    auto units_of = [&](int b, int from, int step) {   // units of one KV head
        const Blocks q = seq_blocks(A, b);
        int64_t u = 0;
        for (int i = from; i < q.n; i += step) {
            int t0, n;
            block_tiles(A, q, i, t0, n);
            u += n;
        }
        return u;
    };
    int64_t mine = 0;
    for (int i = 0; i < per && first_b + i < B.n_seq; ++i)
        mine += units_of(first_b + i, sub, g);
    for (int m = 1; m < g; m <<= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, m);
    const int64_t one_head = mine;
    mine = sub == 0 ? mine * B.Hkv : 0;
    int64_t incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m)
            incl += up;
    }
    if (lane == 31)
        sh.warp_sum[warp] = incl;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        incl += i < warp ? sh.warp_sum[i] : 0;
        total += sh.warp_sum[i];
    }
    const int n_cta = (int)min((int64_t)gridDim.x, total);
    const bool works = (int)blockIdx.x < n_cta;
    const int64_t first = works ? share_begin(total, n_cta, blockIdx.x) : 0;
    const int count = works ? (int)(share_begin(total, n_cta, blockIdx.x + 1) - first) : 0;
    if (works && first < incl && first >= incl - mine) {
        int64_t at = incl - mine;
        for (int i = 0; i < per && first_b + i < B.n_seq; ++i) {
            const int64_t u = g > 1 ? one_head : units_of(first_b + i, 0, 1);
            if (first < at + u * B.Hkv) {
                sh.start_b = first_b + i;
                sh.start_off = first - at;
                sh.head_units = u;
                break;
            }
            at += u * B.Hkv;
        }
    }
    PartMeta *const meta = reinterpret_cast<PartMeta *>(A.ws);
    float *const parts = part_slots(A.ws, gridDim.x);
    if (tid == 0)
        meta[blockIdx.x].owner = 0;
    __syncthreads();
    if (works && warp == 0) {   // the block and tile of the share's first unit
        const Blocks q = seq_blocks(A, sh.start_b);
        const int h = (int)(sh.start_off / sh.head_units);
        const int64_t off = sh.start_off - h * sh.head_units;
        const int each = (q.n + 31) / 32, i0 = lane * each, i1 = min(q.n, i0 + each);
        int64_t u = 0;
        for (int i = i0; i < i1; ++i) {
            int t0, n;
            block_tiles(A, q, i, t0, n);
            u += n;
        }
        int64_t upto = u;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m)
                upto += up;
        }
        if (off < upto && off >= upto - u) {
            int64_t at = upto - u;
            for (int i = i0; i < i1; ++i) {
                int t0, n;
                block_tiles(A, q, i, t0, n);
                if (off < at + n) {
                    sh.start_h = h;
                    sh.start_q = i;
                    sh.start_t = (int)(off - at);
                    break;
                }
                at += n;
            }
        }
    }
    __syncthreads();
    allow_next_grid();

    const uint32_t tmem = sh.tmem;
    const uint64_t lim = A.wait_ns;
    bool failed = false;
    // A wait that gives up stops the CTA's copies and products and ends every other wait; the loops
    // run on to their ends.
    auto wait1 = [&](const uint64_t &bar, uint32_t parity) {
        if (!wait_phase(tc::smem_addr(&bar), parity, lim, &sh.abort)) {
            sh.abort = 1;
            failed = true;
        }
    };
    auto wait = [&](const uint64_t &bar, uint32_t parity) {
        wait1(bar, parity);
        __syncwarp();
    };
    auto arrive = [&](const uint64_t &bar) { tc::mbar_arrive(tc::smem_addr(&bar)); };

    if (warp == 0) {
        // ------------------------------------------------------------ pages to shared memory
        if (works) {
            Walk w = walk_start(A, sh, count);
            int c = 0, issued = 0;
            const int per_tile = kTile / B.P;
            do {
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
                // the pages any row of the block sees
                const int tok0 = w.i * kRows / B.G, tok1 = min((w.i * kRows + kRows - 1) / B.G, w.q.s.n - 1);
                const int pg_lo = max(0, w.q.first + tok0 - A.window + 1) / B.P;
                const int pg_hi = max(0, w.q.first + tok1) / B.P;
                auto page_of = [&](int t) {   // this lane's page of the tile, -1: none wanted, -2: bad
                    const int pg = (w.t0 + t) * per_tile + lane;
                    if (lane >= per_tile || pg < pg_lo || pg > pg_hi)
                        return -1;
                    const int p = __ldg(table + pg);
                    return p >= 0 && p < B.n_pages ? p : -2;
                };
                int page = page_of(w.t);
                for (int t = w.t; t < w.end; ++t, ++c) {
                    const int next = t + 1 < w.end ? page_of(t + 1) : -1;
                    const bool have = page >= 0;
                    if (page == -2)
                        atomicOr(&g_attn_prefill_error, kErrMeta);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * B.P * kHd;
                    const int ks = c % kKs, vs = c % kVs;
                    if (c >= kKs)
                        wait(sh.k_free[ks], (c / kKs - 1) & 1);
                    const bool go = !__any_sync(0xffffffffu, sh.abort != 0);
                    if (go) {
                        const uint32_t bar = tc::smem_addr(&sh.k_full[ks]);
                        if (lane == 0)
                            tc::mbar_expect_tx(bar, bytes);
                        __syncwarp();
                        if (have)
                            copy_page(&map_k, base + kKAt + ks * kTileBytes + lane * B.P * kHd, bar,
                                      page * B.Hkv + w.h);
                    }
                    if (c >= kVs)
                        wait(sh.v_free[vs], (c / kVs - 1) & 1);
                    if (go) {
                        const uint32_t bar = tc::smem_addr(&sh.v_full[vs]);
                        if (lane == 0)
                            tc::mbar_expect_tx(bar, bytes);
                        __syncwarp();
                        if (have)
                            copy_page(&map_v, base + kVAt + vs * kTileBytes + lane * B.P * kHd, bar,
                                      page * B.Hkv + w.h);
                        issued = c + 1;
                    }
                    page = next;
                }
            } while (w.next(A));
            // after a wait that gave up: the copies in flight land before the CTA ends
            for (int k = max(0, issued - kKs); k < issued && sh.abort; ++k) {
                tc::mbar_wait_ns(tc::smem_addr(&sh.k_full[k % kKs]), (k / kKs) & 1, lim);
                if (k >= issued - kVs)
                    tc::mbar_wait_ns(tc::smem_addr(&sh.v_full[k % kVs]), (k / kVs) & 1, lim);
            }
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------ products: warp 1 those of tile A, warp
        // 2 those of B. A thread's products run in the order of their issue, so S of the next tile may be
        // issued behind the product that reads P from the same columns.
        if (works) {
            const int m = warp - 1;
            const bool leader = elect_one();
            constexpr uint32_t idesc_s = idesc_e4m3(128, 128);
            constexpr uint32_t idesc_o = tc::idesc_f16(128, 128) | 1u << 7 | 1u << 10 | tc::kIdescTransB;
            const uint32_t s_at = tmem + m * 128, o_at = tmem + 256 + m * 128;
            const uint64_t q = tc::sdesc_sw128(base + kQAt + 2 * m * kTileBytes);
            Walk w = walk_start(A, sh, count);
            int seg = 0, t = w.t, c = 0;      // the next tile of scores
            bool fresh = true, begin = true;  // whether it, and the tile of the next output, begins its segment
            auto issue_scores = [&] {         // by one thread
                const int ks = c % kKs;
                if (!sh.abort) {
                    const uint64_t k = tc::sdesc_sw128(base + kKAt + ks * kTileBytes);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < 4; ++s)   // 32 bytes of the rows at a time
                            mma_e4m3(s_at, q + part * (kTileBytes >> 4) + 2 * s, k + 2 * s, idesc_s,
                                     part + s > 0);
                }
                tc::mma_commit(tc::smem_addr(&sh.s_full[m]));
                tc::mma_commit(tc::smem_addr(&sh.k_free[ks]));
            };
            auto advance = [&] {
                ++c;
                fresh = ++t == w.end;
                if (fresh) {
                    ++seg;
                    if (w.next(A))
                        t = w.t;
                }
            };
#pragma unroll 1
            for (int j = -1; j < count; ++j) {   // output of tile j, scores of tile j + 1
                const bool more = c < count;
                if (more)
                    wait(sh.k_full[c % kKs], (c / kKs) & 1);
                if (j >= 0) {
                    const int vb = j % kVb;
                    wait(sh.b_full[vb], (j / kVb) & 1);
                    wait(sh.p_full[m], j & 1);
                    tc::fence_after_sync();
                    if (leader) {
                        if (!sh.abort) {
                            const uint64_t v = tc::sdesc_sw128_mn(base + kBAt + vb * 2 * kTileBytes, kTileBytes, 1024);
#pragma unroll
                            for (int s = 0; s < 8; ++s)   // 16 keys: 8 columns of P, 2 KB of V
                                tc::mma_f16_ta(o_at, s_at + 8 * s, v + 128 * s, idesc_o, s > 0 || !begin);
                        }
                        if (more && !fresh)
                            issue_scores();
                        tc::mma_commit(tc::smem_addr(&sh.o_done[m]));
                        tc::mma_commit(tc::smem_addr(&sh.b_free[vb]));
                    }
                    __syncwarp();
                    begin = fresh;
                }
                if (more) {
                    if (fresh) {
                        wait(sh.q_full[m], seg & 1);
                        tc::fence_after_sync();
                        if (leader)
                            issue_scores();
                        __syncwarp();
                    }
                    advance();
                }
            }
            if (sh.abort && leader) {   // products in flight end before the tensor memory is freed
                tc::mma_commit(tc::smem_addr(&sh.drain[m]));
                tc::mbar_wait_ns(tc::smem_addr(&sh.drain[m]), 0, lim);
            }
            __syncwarp();
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ sequences without keys
        const int t32 = lane;
        for (int b = blockIdx.x; b < B.n_seq; b += gridDim.x) {
            const Blocks q = seq_blocks(A, b);
            if (!q.s.ok && t32 == 0)
                atomicOr(&g_attn_prefill_error, kErrMeta);
            if (q.s.ok && q.n == 0) {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(A.out) +
                                                     (int64_t)q.s.row0 * B.Hq * kHd);
                for (int64_t e = t32; e < (int64_t)q.s.n * B.Hq * (kHd / 8); e += 32)
                    o[e] = make_uint4(0, 0, 0, 0);
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ scores to weights: a row per thread
        if (works) {
            const int m = (warp - 4) >> 2, row = (tid - 128) & 127;
            const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_at = tmem + m * 128 + lane_at, o_at = tmem + 256 + m * 128 + lane_at;
            const int page_shift = 31 - __clz(B.P);
            const int per_tile = kTile / B.P;
            const float cap2 = A.softcap * kLog2e, inv_cap2 = CAP ? 1.0f / cap2 : 0.0f;
            Walk w = walk_start(A, sh, count);
            int c = 0;
            const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
            // The q rows of the segment that w is at, 32 by each warp. A row's bf16 pieces land where its own
            // two e4m3 rows will lie, dimensions 0-63 in hi's place and 64-127 in lo's.
            auto load_q = [&] {
                const uint32_t at = kQAt + 2 * m * kTileBytes;
                const int row_w = (warp & 3) * 32;
#pragma unroll 4
                for (int e = lane; e < 32 * 16; e += 32) {
                    const int rr = row_w + (e >> 4), piece = e & 15;
                    const int r = w.i * kRows + m * 128 + rr, tok = r / B.G, gh = r - tok * B.G;
                    const bool have = tok < w.q.s.n;
                    const __nv_bfloat16 *src =
                        static_cast<const __nv_bfloat16 *>(A.q) +
                        (have ? (int64_t)(w.q.s.row0 + tok) * A.q_stride + (w.h * B.G + gh) * kHd + piece * 8 : 0);
                    copy16(base + at + (piece >> 3) * kTileBytes + (rr >> 3) * 1024 + (rr & 7) * 128 +
                               (((piece & 7) ^ (rr & 7)) << 4),
                           src, have);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                const int u = lane & 7;
#pragma unroll 1
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
                    for (int k = 1; k < 8; k <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                    __syncwarp();   // the row is read before it is overwritten
                    store_q16(at_row + ((u ^ (rr & 7)) << 4), kTileBytes, v, sign * q_factor(top));
                    if (u == 0)
                        sh.f[m][rr] = fabsf(A.scale) * kLog2e * pow2i(-q_exponent(top));
                }
                tc::fence_smem_to_async();
                __syncwarp();
                arrive(sh.q_full[m]);
            };
            load_q();
            bool more = true;
            do {
                const int r = w.i * kRows + m * 128 + row;       // row of the sequence and head
                const int tok = r / B.G;
                const bool live = tok < w.q.s.n;
                const int limit = live ? w.q.first + tok : -1;   // last position it sees
                // positions of the tile's first and last row, for a tile that all of them see whole
                const int tok_a = (w.i * kRows + m * 128) / B.G, tok_b = (w.i * kRows + m * 128 + 127) / B.G;
                const int all_to = tok_b < w.q.s.n ? w.q.first + tok_a : -1;
                const int all_from = w.q.first + tok_b - A.window;
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
                const int b_tok1 = min((w.i * kRows + kRows - 1) / B.G, w.q.s.n - 1);
                const int pg_lo = max(0, w.q.first + w.i * kRows / B.G - A.window + 1) / B.P;
                const int pg_hi = max(0, w.q.first + b_tok1) / B.P;
                // lane p: scale of the tile's page p; 0 marks a page the table does not have
                auto page_at = [&](int t) {
                    const int pg = (w.t0 + t) * per_tile + lane;
                    return t < w.end && lane < per_tile && pg >= pg_lo && pg <= pg_hi ? __ldg(table + pg) : -3;
                };
                auto scale_at = [&](int p) {
                    return p == -3 ? 1.0f
                                   : p >= 0 && p < B.n_pages ? __ldg(B.k_scale + (int64_t)p * B.Hkv + w.h) : 0.0f;
                };
                int p_far = page_at(w.t + 1);
                float ks_next = scale_at(page_at(w.t));
                const float f = sh.f[m][row];
                float ref = -INFINITY, l = 0.0f;
                for (int t = w.t; t < w.end; ++t, ++c) {
                    const float ks = ks_next;
                    ks_next = scale_at(p_far);
                    p_far = page_at(t + 2);
                    const uint32_t bad = __ballot_sync(0xffffffffu, ks == 0.0f);
                    const int j0 = (w.t0 + t) * kTile;
                    const bool whole = j0 + kTile - 1 <= all_to && j0 > all_from && bad == 0;
                    const int hi = limit - j0, lo = limit - A.window + 1 - j0;   // visible columns [lo, hi]
                    // bit e: column 32 q4 + e is visible
                    auto mask_of = [&](int q4) {
                        const int h = hi - 32 * q4, o = lo - 32 * q4;
                        uint32_t v = h >= 31 ? 0xffffffffu : h < 0 ? 0u : (2u << h) - 1u;
                        v &= o <= 0 ? 0xffffffffu : o > 31 ? 0u : 0xffffffffu << o;
                        if (bad >> ((32 * q4) >> page_shift) & 1)
                            v &= 0xffff0000u;
                        if (bad >> ((32 * q4 + 16) >> page_shift) & 1)
                            v &= 0x0000ffffu;
                        return v;
                    };
                    auto factor = [&](int half) {   // of 16 columns
                        return f * __shfl_sync(0xffffffffu, ks, (16 * half) >> page_shift);
                    };
                    wait(sh.s_full[m], c & 1);
                    tc::fence_after_sync();
                    if (!whole || !__all_sync(0xffffffffu, ref > -INFINITY) ||
                        !row_weights_once<CAP>(s_at, factor, ref, l, cap2, inv_cap2)) {
                        float top = -INFINITY;
                        if (whole)
                            top = row_max<CAP, true>(s_at, mask_of, factor, cap2, inv_cap2);
                        else
                            top = row_max<CAP, false>(s_at, mask_of, factor, cap2, inv_cap2);
                        // the reference moves when a weight would pass 2^kSlack, or is the row's first
                        const bool move = top > ref + kSlack || (ref == -INFINITY && top > ref);
                        if (__any_sync(0xffffffffu, move)) {
                            const float to = move ? top : ref;
                            const float a = move ? ex2(ref - to) : 1.0f;
                            ref = to;
                            l *= a;
                            if (t > w.t) {
                                wait(sh.o_done[m], (c - 1) & 1);
                                tc::fence_after_sync();
    #pragma unroll 1
                                for (int q4 = 0; q4 < 4; ++q4) {
                                    uint32_t x[32];
                                    tmem_get32(o_at + 32 * q4, x);
                                    tmem_wait32(x);
    #pragma unroll
                                    for (int half = 0; half < 2; ++half) {
                                        uint32_t y[16];
    #pragma unroll
                                        for (int e = 0; e < 16; ++e)
                                            y[e] = __float_as_uint(__uint_as_float(x[16 * half + e]) * a);
                                        tc::tmem_st16u(o_at + 32 * q4 + 16 * half, y);
                                    }
                                }
                            }
                        }
                        const float sub = ref == -INFINITY ? 0.0f : ref;
                        if (whole)
                            l += row_weights<CAP, true>(s_at, mask_of, factor, sub, cap2, inv_cap2);
                        else
                            l += row_weights<CAP, false>(s_at, mask_of, factor, sub, cap2, inv_cap2);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    arrive(sh.p_full[m]);
                }
                // The products that read the segment's q are done (its last scores are here): the next
                // segment's q goes in, and its first scores are formed while this one's rows are written.
                const bool whole_block = w.begins() && w.ends(), begins = w.begins();
                const int seg_b = w.b, seg_h = w.h, seg_row = w.i * kRows, seg_row0 = w.q.s.row0;
                const int64_t end_unit = first + count - w.left + (w.n - w.t);   // past the block's last tile
                more = w.next(A);
                if (more)
                    load_q();
                wait(sh.o_done[m], (c - 1) & 1);
                tc::fence_after_sync();
                if (whole_block) {
                    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
                    const int gh = r - tok * B.G;
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(A.out) +
                                         ((int64_t)(seg_row0 + tok) * B.Hq + seg_h * B.G + gh) * kHd;
#pragma unroll 1
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t x[32];
                        tmem_get32(o_at + 32 * q4, x);
                        tmem_wait32(x);
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t y[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    y[i] = pack_bf16x2(__uint_as_float(x[16 * e + 2 * i]) * inv,
                                                       __uint_as_float(x[16 * e + 2 * i + 1]) * inv);
                                uint4 *at = reinterpret_cast<uint4 *>(out + 32 * q4 + 16 * e);
                                at[0] = make_uint4(y[0], y[1], y[2], y[3]);
                                at[1] = make_uint4(y[4], y[5], y[6], y[7]);
                            }
                        }
                    }
                } else {
                    const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
                    float *dst = parts + ((size_t)slot * kRows + m * 128 + row) * kPartRow;
#pragma unroll 1
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t x[32];
                        tmem_get32(o_at + 32 * q4, x);
                        tmem_wait32(x);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<uint4 *>(dst)[8 * q4 + e] =
                                make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    }
                    *reinterpret_cast<float2 *>(dst + kHd) = make_float2(l, ref);
                    if (begins && m == 0 && row == 0)
                        meta[blockIdx.x] = {seg_b, seg_h, seg_row, share_of(total, n_cta, end_unit - 1), 1, {}};
                }
                tc::fence_before_sync();
            } while (more);
        }
    } else {
        // ------------------------------------------------------------ V to bf16: a key per thread
        if (works) {
            const int t128 = tid - 384;
            Walk w = walk_start(A, sh, count);
            int c = 0;
            do {
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
                const int tok1 = min((w.i * kRows + kRows - 1) / B.G, w.q.s.n - 1);
                const int j_lo = max(0, w.q.first + w.i * kRows / B.G - A.window + 1);
                const int j_hi = w.q.first + tok1;               // last position any row sees
                auto page_at = [&](int t) {
                    const int j = (w.t0 + t) * kTile + t128;
                    if (t >= w.end || j < j_lo || j > j_hi)
                        return -1;
                    const int p = __ldg(table + j / B.P);
                    return p >= 0 && p < B.n_pages ? p : -1;
                };
                auto scale_at = [&](int p) {
                    return p >= 0 ? __ldg(B.v_scale + (int64_t)p * B.Hkv + w.h) : 0.0f;
                };
                int p_next = page_at(w.t), p_far = page_at(w.t + 1);
                float vs_next = scale_at(p_next);
                for (int t = w.t; t < w.end; ++t, ++c) {
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
                    wait(sh.v_full[vst], (c / kVs) & 1);
                    const uint8_t *src = mem + kVAt + vst * kTileBytes + t128 * kHd;
                    if (c >= kVb)
                        wait(sh.b_free[vb], (c / kVb - 1) & 1);
                    uint8_t *dst = mem + kBAt + vb * 2 * kTileBytes + (t128 >> 3) * 1024 + (t128 & 7) * 128;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        const uint4 raw = dead ? make_uint4(0, 0, 0, 0)
                                               : *reinterpret_cast<const uint4 *>(src + ((k ^ (t128 & 7)) << 4));
                        const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[2 * i] = mul_bf16x2(codes_bf16(__byte_perm(in[i], 0, 0x1404)), f1);
                            o[2 * i + 1] = mul_bf16x2(codes_bf16(__byte_perm(in[i], 0, 0x3424)), f1);
                        }
                        if (e2 != 0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                o[i] = mul_bf16x2(o[i], f2);
                        }
                        // dimensions 16 k .. 16 k + 15: two 16-byte pieces of half k / 4
                        uint8_t *half = dst + (k >> 2) * kTileBytes;
                        const int p0 = (2 * k) & 7;
                        *reinterpret_cast<uint4 *>(half + ((p0 ^ (t128 & 7)) << 4)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(half + (((p0 + 1) ^ (t128 & 7)) << 4)) =
                            make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    arrive(sh.v_free[vst]);
                    tc::fence_smem_to_async();
                    arrive(sh.b_full[vb]);
                }
            } while (w.next(A));
        }
    }
    if (failed)
        atomicOr(&g_attn_prefill_error, kErrWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1)
        tc::tmem_dealloc(tmem, kTmemCols);
}

template <bool CAP>
cudaError_t launch_cap(const AttnArgs &a, int grid, cudaStream_t s)
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
    return launch_join(a, grid, kRows, s);
}

}  // namespace

size_t prefill_workspace_bytes(int sms) { return part_bytes((size_t)sms, kRows); }

cudaError_t launch_prefill(const AttnArgs &args, cudaStream_t s)
{
    AttnArgs a = args;
    const Batch &b = a.b;
    if (a.window == 0 || a.window > kNoWindow)
        a.window = kNoWindow;
    const int64_t tiles = ((int64_t)b.max_pages * b.P + kTile - 1) / kTile;
    const int64_t blocks = ((int64_t)b.max_q * b.G + kRows - 1) / kRows * b.Hkv * b.n_seq;
    const int grid = (int)(tiles >= a.sm_count || blocks >= a.sm_count || tiles * blocks >= a.sm_count
                               ? a.sm_count : tiles * blocks);
    return a.softcap > 0.0f ? launch_cap<true>(a, grid, s) : launch_cap<false>(a, grid, s);
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
