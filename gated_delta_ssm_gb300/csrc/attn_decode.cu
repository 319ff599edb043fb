// attn_decode.cu -- gdn_attn_decode: attention of one to a few tokens per
// sequence over the paged e4m3 cache.
//
// Mathematics. For the R = G * n rows (token, head of the group) of one KV head
// and a tile of 128 keys, the tensor core forms the transposed scores
// S^T[key][row] = K Q^T and the transposed output O^T[d][row] = V^T P^T, so that
// the 128 keys (and the 128 dimensions) fill its 128 rows and the few q rows are
// its columns. Both products read the cache's codes as they lie in shared
// memory: nothing is converted. Q and P are each split into two e4m3 numbers,
// hi + lo. A bf16 q row scaled by a power of two so that its largest value is
// below 256 is hi + lo exactly (down to 2^-17 of that largest value); a weight
// keeps 2^-8 of itself, as many bits as bf16 has.
//   The key scale of a page and the value scale 2^e enter the exponent:
// w = s f ks + e, P = 2^(w - max w + 8) <= 256, the maximum taken over the 32
// keys of one warp, which are also one step (K = 32) of the second product. Each
// warp's product has tensor memory of its own, so warps need not agree on a
// maximum and never wait for one another, and the steps of P are fine for every
// 32 keys, however far below the row's largest weight they lie. The partial
// products are joined in 32-bit registers, O += O_w 2^(max_w - ref); the sum of
// weights takes P 2^-e before P is rounded.
//
// Bound by memory: 256 bytes of codes per key and KV head. The batch's tiles are
// shared out equally over the CTAs (attn_share.cuh); a (sequence, head) that
// spans CTAs leaves 32-bit partial results which a second kernel joins.
//
// Measured: 64 sequences of 800 to 8191 tokens, 32 q heads on 8, one token each:
// 102 us, 5.6 TB/s (DRAM busy 71% of the time, the tensor pipe 8%). One sequence
// of 131071 tokens, 4 KV heads: 42 us, of which about 8 pass before the first
// tile is used and 5 in the join; between them the codes come at 4.7 TB/s, not the
// memory's rate. 32 drafts of four tokens, cap 30, R = 32: 63 us. A tile there takes
// about 8100 warp instructions, and issue slots are 43% busy: what is waited for is
// the chain copy, scores, weights, output, join of a tile (loads 2.5, fixed latencies
// 1.5, barriers 1.3 of 9.3 cycles an issue). Four groups of softmax warps there take
// 70 us, two columns' loops unrolled 73 us.
//
// Roles of a CTA: warp 0 copies pages to shared memory, warp 1 issues the
// products, warp 2 splits the q rows of the next segment, warp 3 walks the share,
// one or two groups of four warps hold a key per thread and turn scores into
// weights, and the last four warps hold a dimension per thread and join the
// products.
#include <cfloat>

#include "attn_share.cuh"
#include "attn_tc.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_attn_decode_error;

namespace {

constexpr int kOver = 1;     // what a block costs besides its tiles, in tiles
constexpr int kWhole = 3;    // most tiles of blocks that are not worth splitting

template <int NR>            // rows, padded
struct Cfg {
    // tiles in flight, K and V counted apart (item 2 i is K of tile i, 2 i + 1 its V)
    static constexpr int kItems = NR == 16 ? 5 : NR == 32 ? 8 : 6;
    static constexpr int kCtas = NR == 16 ? 2 : 1;               // CTAs per SM
    static constexpr uint32_t kRowBytes = NR * kHd;              // one e4m3 operand of NR rows
    static constexpr uint32_t kQ = kItems * kTileBytes;          // [2 segments][hi, lo]
    static constexpr uint32_t kP = kQ + 4 * kRowBytes;           // [2 tiles][hi, lo]
    static constexpr uint32_t kO32 = kP + 4 * kRowBytes;         // a segment's joined products, float [NR][128]
    static constexpr uint32_t kEnd = kO32 + 4 * kRowBytes;
    // tensor memory: S of two tiles, then the four warps' products of kO tiles
    static constexpr int kO = NR == 64 ? 1 : 2;
    static constexpr uint32_t kTmemCols = NR == 16 ? 256 : 512;
    static constexpr int kLs = (NR + 31) / 32;
    // groups of four warps that turn scores into weights, eight rows in turn each
    static constexpr int kWgs = NR == 16 ? 1 : 2;
    static constexpr int kThreads = 256 + 128 * kWgs;
};

template <int NR>
struct Shared {
    uint64_t full[Cfg<NR>::kItems], empty[Cfg<NR>::kItems], drain;
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2], q_full[2], q_free[2], l_full[2], l_free[2], coef_full[4];
    uint32_t tmem;
    volatile int abort;
    ShareShared<Cfg<NR>::kThreads> share;
    Ring ring;
    float4 top[4][NR];         // of four tiles: the warps' maxima of each row,
    float4 scale[2][NR];       // and, of two, 2^(maximum - o_ref)
    float f[2][NR];            // scale * log2 e / (power of two of the q row)
    int limit[2][NR];          // position of each row
    float l_sum[2][4][NR], l_ref[2][4][NR];
    float o_ref[NR];
};

// 8 columns of this thread's lane, without waiting, and the wait for them.
__device__ __forceinline__ void tmem_get8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait8(uint32_t (&r)[8], float (&v)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(r[i]);
}

// 4 columns of each of the four warps' products, `step` columns apart, without waiting, and the wait.
__device__ __forceinline__ void tmem_get4x4(uint32_t taddr, uint32_t step, uint32_t (&r)[4][4])
{
#pragma unroll
    for (int w = 0; w < 4; ++w)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[w][0]), "=r"(r[w][1]), "=r"(r[w][2]), "=r"(r[w][3]) : "r"(taddr + w * step));
}
__device__ __forceinline__ void tmem_wait4x4(uint32_t (&r)[4][4])
{
#pragma unroll
    for (int w = 0; w < 4; ++w)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[w][0]), "+r"(r[w][1]), "+r"(r[w][2]), "+r"(r[w][3]) :: "memory");
}

// Sums over the warp of eight values per lane: lane i gets that of value i & 7. Halving the values each lane
// carries takes 9 exchanges where eight separate sums take 40.
__device__ __forceinline__ float sum8(const float (&v)[8], int lane)
{
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = lane & 4 ? v[i + 4] : v[i], give = lane & 4 ? v[i] : v[i + 4];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = lane & 2 ? a[i + 2] : a[i], give = lane & 2 ? a[i] : a[i + 2];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    {
        const float keep = lane & 1 ? b[1] : b[0], give = lane & 1 ? b[0] : b[1];
        c = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    return c + __shfl_xor_sync(0xffffffffu, c, 16);
}

template <int NR>
__global__ void __launch_bounds__(Cfg<NR>::kThreads, Cfg<NR>::kCtas)
attn_decode_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v)
{
    using C = Cfg<NR>;
    constexpr int kThreads = C::kThreads;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared<NR> sh;
    const Batch &B = A.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem_addr(dyn) + 1023u) & ~1023u;
    uint8_t *const mem = dyn + (base - tc::smem_addr(dyn));
    const int R = B.G * B.max_q, chunks = (R + 7) / 8;   // rows are handled eight at a time

    if (tid == 0) {
        auto init = [&](uint64_t &bar, uint32_t n) { tc::mbar_init(tc::smem_addr(&bar), n); };
        for (int i = 0; i < C::kItems; ++i)
            init(sh.full[i], 1), init(sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            init(sh.s_full[i], 1);
            init(sh.p_full[i], 128 * C::kWgs);
            init(sh.o_full[i], 1);
            init(sh.o_free[i], 128);
            init(sh.q_full[i], 32);
            init(sh.q_free[i], 128 * C::kWgs + 1);
            init(sh.l_full[i], 128 * C::kWgs);
            init(sh.l_free[i], 128);
        }
        for (int i = 0; i < 4; ++i)
            init(sh.coef_full[i], 4 * C::kWgs);
        for (int i = 0; i < kRing; ++i)
            init(sh.ring.full[i], 1), init(sh.ring.free[i], kThreads / 32 - 1);   // every warp but the walker
        init(sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.abort = 0;
    }
    if (warp == 1)
        tc::tmem_alloc(tc::smem_addr(&sh.tmem), C::kTmemCols);
    // rows of Q and P that no q row uses stay zero
    for (uint32_t i = tid; i < 8 * C::kRowBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(mem + C::kQ)[i] = make_uint4(0, 0, 0, 0);
    if (tid < 2 * NR) {
        sh.f[tid / NR][tid % NR] = 0.0f;
        sh.limit[tid / NR][tid % NR] = -1;
    }
    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    }
    tc::fence_smem_to_async();

    wait_previous_grid();
    Share share = {};
    if (B.n_seq > kFewSeqs)
        share = find_share<kMaxDecodeRows, kOver, kWhole>(A, sh.share, tid, kThreads, [] { __syncthreads(); });
    PartMeta *const meta = reinterpret_cast<PartMeta *>(A.ws);
    float *const parts = part_slots(A.ws, gridDim.x);
    if (tid == kThreads - 128)   // the thread that may describe a block later
        meta[blockIdx.x].owner = 0;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    allow_next_grid();

    const uint32_t tmem = sh.tmem;
    const uint64_t lim = A.wait_ns;
    const int page_shift = 31 - __clz(B.P), inv_G = 65536 / B.G + 1;   // r / G = r * inv_G >> 16 for r below 4096
    bool failed = false;
    // A wait that gives up stops the CTA's copies and products and ends every other wait; the loops
    // run on to their ends. wait is for whole warps.
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
    auto wait_first = [&](const uint64_t &bar, uint32_t parity) {   // the CTA's first, whose limit a test sets
        if (!wait_phase(tc::smem_addr(&bar), parity, A.first_wait_ns, &sh.abort)) {
            sh.abort = 1;
            failed = true;
        }
        __syncwarp();
    };
    auto arrive = [&](const uint64_t &bar) { tc::mbar_arrive(tc::smem_addr(&bar)); };

    if (warp == 0) {
        // ------------------------------------------------------------ pages to shared memory
        int i = 0, issued = 0;
        const int per_tile = kTile >> page_shift;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
            if (w.nt == 0)
                break;
            GDN_CHECK(g_attn_decode_error, seg_in_range(A, w));
            const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
            const int pg_lo = w.lo >> page_shift, pg_hi = w.hi >> page_shift;
            auto page_of = [&](int t) {   // this lane's page of the tile, -1: none wanted, -2: bad
                const int pg = (w.kt + t) * per_tile + lane;
                if (t >= w.nt || lane >= per_tile || pg < pg_lo || pg > pg_hi)
                    return -1;
                GDN_CHECK(g_attn_decode_error, pg >= 0 && pg < B.max_pages);
                const int p = __ldg(table + pg);
                return p >= 0 && p < B.n_pages ? p : -2;
            };
            int page = page_of(0), page2 = page_of(1);
#pragma unroll 1
            for (int t = 0; t < w.nt; ++t) {
                const int page3 = page_of(t + 2);
                const bool have = page >= 0;
                if (page == -2)
                    atomicOr(&g_attn_decode_error, kErrMeta);
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * B.P * kHd;
#pragma unroll 1
                for (int part = 0; part < 2; ++part, ++i) {   // K, then V
                    const int st = i % C::kItems;
                    if (i >= C::kItems)
                        wait(sh.empty[st], (i / C::kItems - 1) & 1);
                    if (__any_sync(0xffffffffu, sh.abort != 0))
                        continue;
                    const uint32_t bar = tc::smem_addr(&sh.full[st]);
                    if (lane == 0)
                        tc::mbar_expect_tx(bar, bytes);
                    __syncwarp();
                    if (have)
                        copy_page(part ? &map_v : &map_k, base + st * kTileBytes + lane * B.P * kHd, bar,
                                  page * B.Hkv + w.h);
                    issued = i + 1;
                }
                page = page2;
                page2 = page3;
            }
        }
        // after a wait that gave up: the copies in flight land before the CTA ends
        for (int k = max(0, issued - C::kItems); k < issued && sh.abort; ++k)
            tc::mbar_wait_ns(tc::smem_addr(&sh.full[k % C::kItems]), (k / C::kItems) & 1, lim);
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool leader = elect_one();
        constexpr uint32_t idesc_s = idesc_e4m3(128, NR);
        constexpr uint32_t idesc_o = idesc_e4m3(128, NR) | kIdescTransA;
        int k = 0, c = 0, left = take_seg(sh.ring, 0, wait, &sh.abort).nt;   // segment, tile, its tiles left: of the next scores
#pragma unroll 1
        for (int j = -2; j < c; ++j) {      // scores of tile j + 2 behind the output of tile j
            if (j >= 0) {
                const int item = 2 * j + 1, st = item % C::kItems, par = j & 1, ob = j % C::kO;
                if (j >= C::kO)
                    wait(sh.o_free[ob], (j / C::kO - 1) & 1);
                wait(sh.full[st], (item / C::kItems) & 1);
                wait(sh.p_full[par], (j / 2) & 1);
                tc::fence_after_sync();
                if (leader) {
                    if (!sh.abort) {
                        const uint64_t v = tc::sdesc_sw128_mn(base + st * kTileBytes, 1024, 1024);
                        const uint64_t p = tc::sdesc_sw128(base + C::kP + par * 2 * C::kRowBytes);
#pragma unroll
                        for (int s = 0; s < 4; ++s)   // a warp's 32 keys: 4 KB of V, 32 bytes of P's rows
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_e4m3(tmem + (2 + 4 * ob + s) * NR, v + 256 * s,
                                         p + part * (C::kRowBytes >> 4) + 2 * s, idesc_o, part);
                    }
                    tc::mma_commit(tc::smem_addr(&sh.o_full[ob]));
                    tc::mma_commit(tc::smem_addr(&sh.empty[st]));
                }
                __syncwarp();
            }
            if (left > 0) {
                const int item = 2 * c, st = item % C::kItems;
                wait(sh.q_full[k & 1], (k >> 1) & 1);
                if (c == 0)
                    wait_first(sh.full[st], 0);
                else
                    wait(sh.full[st], (item / C::kItems) & 1);
                tc::fence_after_sync();
                if (leader) {
                    if (!sh.abort) {
                        const uint64_t kd = tc::sdesc_sw128(base + st * kTileBytes);
                        const uint64_t q = tc::sdesc_sw128(base + C::kQ + (k & 1) * 2 * C::kRowBytes);
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int s = 0; s < 4; ++s)   // 32 bytes of the 128-byte rows at a time
                                mma_e4m3(tmem + (c & 1) * NR, kd + 2 * s, q + part * (C::kRowBytes >> 4) + 2 * s,
                                         idesc_s, part + s > 0);
                    }
                    tc::mma_commit(tc::smem_addr(&sh.s_full[c & 1]));
                    tc::mma_commit(tc::smem_addr(&sh.empty[st]));
                    if (left == 1)
                        tc::mma_commit(tc::smem_addr(&sh.q_free[k & 1]));
                }
                __syncwarp();
                ++c;
                if (--left == 0)
                    left = take_seg(sh.ring, ++k, wait, &sh.abort).nt;
            }
        }
        if (leader) {   // every product, and every arrival that a commit still owes, ends before the CTA does
            tc::mma_commit(tc::smem_addr(&sh.drain));
            tc::mbar_wait_ns(tc::smem_addr(&sh.drain), 0, lim);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ q rows, four at a time
        const int u = lane & 7, r4 = lane >> 3;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
            if (w.nt == 0)
                break;
            const int par = k & 1;
            if (k >= 2)
                wait(sh.q_free[par], (k / 2 - 1) & 1);
#pragma unroll 2
            for (int r = r4; r < ((R + 3) & ~3); r += 4) {
                const int tok = r * inv_G >> 16, g = r - tok * B.G;
                const bool live = tok < w.n;
                GDN_CHECK(g_attn_decode_error,
                          r < NR && (!live || (w.row0 + tok < B.n_tokens && w.h * B.G + g < B.Hq)));
                float v[16] = {};
                if (live)
                    load_q16(static_cast<const __nv_bfloat16 *>(A.q) + (int64_t)(w.row0 + tok) * A.q_stride +
                                 (w.h * B.G + g) * kHd + u * 16,
                             v);
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                for (int m = 1; m < 8; m <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                store_q16(mem + C::kQ + par * 2 * C::kRowBytes + (r >> 3) * 1024 + (r & 7) * 128 +
                              ((u ^ (r & 7)) << 4),
                          C::kRowBytes, v, q_factor(top));
                if (u == 0) {
                    sh.f[par][r] = A.scale * (0.5f * kLog2e) * pow2i(1 - q_exponent(top));   // halved: it may be huge
                    sh.limit[par][r] = live ? w.first + tok : -1;
                }
            }
            tc::fence_smem_to_async();
            arrive(sh.q_full[par]);
        }
    } else if (warp == 3) {
        if (B.n_seq <= kFewSeqs)
            share = find_share<kMaxDecodeRows, kOver, kWhole>(A, sh.share, lane, 32, [] { __syncwarp(); });
        walk_share<kMaxDecodeRows, kOver>(A, share, sh.ring, wait, &sh.abort);
        clear_empty(A, &g_attn_decode_error);
    } else if (warp < 4 + 4 * C::kWgs) {
        // ------------------------------------------------------------ scores to weights: a key per thread
        const int t128 = tid & 127, wq = warp & 3, wg = (warp >> 2) - 1;
        const int row8 = lane & 7;
        const uint32_t s_at = tmem + ((uint32_t)(wq * 32) << 16);
        const float cap2 = A.softcap * kLog2e, cap_in = 2.0f * kLog2e / cap2;
        const int cap = cap_mode(A.softcap);
        int i = 0;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
            if (w.nt == 0)
                break;
            const int par_q = k & 1;
            const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
            // lane r holds the sum of weights and its reference for row r (and 32 + r) of this warp's keys
            float l[C::kLs], big[C::kLs];
#pragma unroll
            for (int e = 0; e < C::kLs; ++e)
                l[e] = 0.0f, big[e] = -INFINITY;
            auto page_at = [&](int t) {
                const int j = (w.kt + t) * kTile + t128;
                if (t >= w.nt || j < w.lo || j > w.hi)
                    return -1;
                GDN_CHECK(g_attn_decode_error, j >= 0 && j >> page_shift < B.max_pages);
                const int p = __ldg(table + (j >> page_shift));
                return p >= 0 && p < B.n_pages ? p : -1;
            };
            auto scale_at = [&](const float *s, int p) {
                return p >= 0 ? __ldg(s + (int64_t)p * B.Hkv + w.h) : 1.0f;
            };
            int p_next = page_at(0), p_far = page_at(1);
            float ks_next = scale_at(B.k_scale, p_next), vs_next = scale_at(B.v_scale, p_next);
            wait(sh.q_full[par_q], (k >> 1) & 1);
#pragma unroll 1
            for (int t = 0; t < w.nt; ++t, ++i) {
                const int par = i & 1;
                const float ks = ks_next, vs = vs_next;
                const bool dead = p_next < 0;
                p_next = p_far;
                ks_next = scale_at(B.k_scale, p_next);
                vs_next = scale_at(B.v_scale, p_next);
                p_far = page_at(t + 2);
                const int j0 = (w.kt + t) * kTile, j = j0 + t128;
                // whether every row sees all of the warp's keys
                const bool whole = __all_sync(0xffffffffu, !dead && j <= w.first && j > w.first + w.n - 1 - A.window);
                const float ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
                const float iv = pow2i(127 - (int)(__float_as_uint(vs) >> 23));
                uint8_t *const prow = mem + C::kP + par * 2 * C::kRowBytes + (t128 & 15);
                wait(sh.s_full[par], (i >> 1) & 1);
                tc::fence_after_sync();
                uint32_t next[8];
                tmem_get8(s_at + par * NR + 8 * wg, next);
#pragma unroll 1
                for (int c = wg; c < chunks; c += C::kWgs) {
                    float x[8];
                    tmem_wait8(next, x);
                    if (c + C::kWgs < chunks)
                        tmem_get8(s_at + par * NR + 8 * (c + C::kWgs), next);
                    const float4 f0 = *reinterpret_cast<const float4 *>(&sh.f[par_q][8 * c]);
                    const float4 f1 = *reinterpret_cast<const float4 *>(&sh.f[par_q][8 * c + 4]);
                    const uint64_t f2[4] = {pack2(f0.x, f0.y), pack2(f0.z, f0.w), pack2(f1.x, f1.y), pack2(f1.z, f1.w)};
                    const uint64_t ks2 = pack2(ks, ks), ev2 = pack2(ev, ev);
                    if (cap == kNoCap) {
#pragma unroll
                        for (int r = 0; r < 8; r += 2) {
                            const float2 y = unpack2(fma2(pack2(x[r], x[r + 1]), mul2(f2[r / 2], ks2), ev2));
                            x[r] = y.x, x[r + 1] = y.y;
                        }
                    } else if (cap == kLowCap) {   // c - 2 c / (1 + e^(2 s / cap)); tanh is 1 past an exponent of 60
#pragma unroll
                        for (int r = 0; r < 8; r += 2) {
                            const float2 y = unpack2(mul2(pack2(x[r], x[r + 1]), mul2(f2[r / 2], ks2)));
                            const float a = 1.0f + ex2(min_nan(y.x * cap_in, 60.0f));
                            const float b = 1.0f + ex2(min_nan(y.y * cap_in, 60.0f));
                            x[r] = fmaf(rcp(a), -2.0f * cap2, cap2 + ev);
                            x[r + 1] = fmaf(rcp(b), -2.0f * cap2, cap2 + ev);
                        }
                    } else {
                        const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            x[r] = fmaf(cap2, tanh_cap(x[r] * (f[r] * ks) / cap2), ev);
                    }
                    if (!whole) {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int at = sh.limit[par_q][8 * c + r];
                            x[r] = dead || j > at || j <= at - A.window ? -INFINITY : x[r];
                        }
                    }
                    float mine = -INFINITY, sums[8];
                    uint8_t *const p8 = prow + c * 1024;
#pragma unroll
                    for (int r = 0; r < 8; r += 2) {
                        const float m0 = redux_max(x[r]), m1 = redux_max(x[r + 1]);
                        mine = row8 == r ? m0 : row8 == r + 1 ? m1 : mine;
                        // P is 2^(w - max + 8): at most 256; a row without visible keys has no maximum
                        const float2 y = unpack2(add2(pack2(x[r], x[r + 1]), pack2(8.0f - fmaxf(m0, kNoRef),
                                                                                   8.0f - fmaxf(m1, kNoRef))));
                        const float z0 = ex2(y.x), z1 = ex2(y.y);
                        const float2 q = unpack2(mul2(pack2(z0, z1), pack2(iv, iv)));
                        sums[r] = q.x, sums[r + 1] = q.y;
                        uint32_t h8, l8;
                        split_e4m3(z0, z1, h8, l8);
                        uint8_t *a = p8 + r * 128 + (((t128 >> 4) ^ r) << 4);
                        uint8_t *b = p8 + (r + 1) * 128 + (((t128 >> 4) ^ (r + 1)) << 4);
                        a[0] = (uint8_t)h8;
                        b[0] = (uint8_t)(h8 >> 8);
                        a[C::kRowBytes] = (uint8_t)l8;
                        b[C::kRowBytes] = (uint8_t)(l8 >> 8);
                    }
                    const float sum = sum8(sums, lane);
                    if ((lane >> 3) == (c & 3)) {     // the lane that keeps row 8 c + (lane & 7)
                        reinterpret_cast<float *>(&sh.top[i & 3][8 * c + row8])[wq] = mine;
#pragma unroll
                        for (int e = 0; e < C::kLs; ++e) {
                            if (e != c >> 2)
                                continue;
                            const float grown = fmaxf(big[e], mine);
                            if (grown > -INFINITY) {
                                l[e] = fmaf(l[e], ex2(big[e] - grown), sum * ex2(mine - grown));
                                big[e] = grown;
                            } else {
                                l[e] += sum;          // zero, or NaN
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    arrive(sh.coef_full[i & 3]);
                if (dead && wg == 0) {
                    // nothing of the cache lies here, or nothing that may be seen: any code, NaN among
                    // them; its value row is cleared so that weight 0 gives 0
                    const int item = 2 * i + 1, st = item % C::kItems;
                    wait1(sh.full[st], (item / C::kItems) & 1);
                    uint4 *row = reinterpret_cast<uint4 *>(mem + st * kTileBytes + t128 * kHd);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        row[c] = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
                tc::fence_smem_to_async();
                tc::fence_before_sync();
                arrive(sh.p_full[par]);
            }
            arrive(sh.q_free[par_q]);
            if (k >= 2)
                wait(sh.l_free[par_q], (k / 2 - 1) & 1);
#pragma unroll
            for (int e = 0; e < C::kLs; ++e)
                if (32 * e + lane < NR && ((lane >> 3) & (C::kWgs - 1)) == wg) {
                    sh.l_sum[par_q][wq][32 * e + lane] = l[e];
                    sh.l_ref[par_q][wq][32 * e + lane] = big[e];
                }
            arrive(sh.l_full[par_q]);
        }
    } else {
        // ------------------------------------------------------------ products joined: a dimension per thread
        const int d = tid & 127, wq = warp & 3;
        const uint32_t o_at = tmem + 2 * NR + ((uint32_t)(wq * 32) << 16);
        int i = 0;
#pragma unroll 1
        for (int k = 0;; ++k) {
            const Seg w = take_seg(sh.ring, k, wait, &sh.abort);
            if (named_any(1, 128, w.nt == 0))   // the four warps meet at barriers, so they end together
                break;
            const int par_q = k & 1;
            float o[NR];               // O of row r is o 2^o_ref[r]
#pragma unroll
            for (int r = 0; r < NR; ++r)
                o[r] = 0.0f;
            named_sync(1, 128);        // the last segment's rows are out
            if (d < NR)
                sh.o_ref[d] = kNoRef;
            named_sync(1, 128);
#pragma unroll 1
            for (int t = 0; t < w.nt; ++t, ++i) {
                const int ob = i % C::kO;
                wait(sh.coef_full[i & 3], (i >> 2) & 1);
                // a (row, warp) pair per thread: its scale. The references lag, by 2^20 at most: sums of 32 bits do
                // not mind, with values down to 2^-75 neither (l holds their reciprocals)
                bool move = false;
#pragma unroll
                for (int e = 0; e < (4 * NR + 127) / 128; ++e) {
                    const int r = 32 * e + (d >> 2);
                    if (r < R) {
                        const float m = reinterpret_cast<const float *>(&sh.top[i & 3][r])[d & 3] - sh.o_ref[r];
                        move |= m > 20.0f;
                        reinterpret_cast<float *>(&sh.scale[i & 1][r])[d & 3] = ex2(m);
                    }
                }
                if (named_any(1, 128, move)) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r % 4 == 0 && r >= R)
                            break;
                        const float4 m = sh.top[i & 3][r];
                        const float ref = sh.o_ref[r];
                        o[r] *= ex2(ref - fmaxf(ref, fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w))));
                    }
                    named_sync(1, 128);
                    if (d < R) {
                        const float4 m = sh.top[i & 3][d];
                        const float ref = fmaxf(sh.o_ref[d], fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)));
                        sh.o_ref[d] = ref;
                        sh.scale[i & 1][d] = make_float4(ex2(m.x - ref), ex2(m.y - ref), ex2(m.z - ref), ex2(m.w - ref));
                    }
                    named_sync(1, 128);
                }
                wait(sh.o_full[ob], (i / C::kO) & 1);
                tc::fence_after_sync();
                uint32_t next[2][4][4];
                tmem_get4x4(o_at + 4 * ob * NR, NR, next[0]);
#pragma unroll
                for (int c = 0; c < NR / 4; ++c) {
                    if (4 * c >= R)
                        break;
                    uint32_t(&x)[4][4] = next[c & 1];
                    tmem_wait4x4(x);
                    if (c + 1 < NR / 4 && 4 * c + 4 < R)
                        tmem_get4x4(o_at + 4 * ob * NR + 4 * c + 4, NR, next[(c + 1) & 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 4 * c + e;
                        const float4 m = sh.scale[i & 1][r];
                        o[r] = fmaf(__uint_as_float(x[0][e]), m.x, o[r]);
                        o[r] = fmaf(__uint_as_float(x[1][e]), m.y, o[r]);
                        o[r] = fmaf(__uint_as_float(x[2][e]), m.z, o[r]);
                        o[r] = fmaf(__uint_as_float(x[3][e]), m.w, o[r]);
                    }
                }
                tc::fence_before_sync();
                arrive(sh.o_free[ob]);
            }
            // through shared memory, so that a warp writes whole rows and the code does not know their number
            float *const stage = reinterpret_cast<float *>(mem + C::kO32);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                stage[r * kHd + d] = o[r];
            named_sync(1, 128);
            wait(sh.l_full[par_q], (k >> 1) & 1);
            const int rows = w.n * B.G;
            float *part = parts + (size_t)(2 * blockIdx.x + (w.begins ? 1 : 0)) * R * kPartRow;
#pragma unroll 1
            for (int r = wq; r < rows; r += 4) {
                GDN_CHECK(g_attn_decode_error, r < R && w.row0 + r / B.G < B.n_tokens && seg_in_range(A, w));
                const float at = sh.o_ref[r];
                float l = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    l += sh.l_sum[par_q][e][r] * ex2(sh.l_ref[par_q][e][r] - at);
                const float4 x = *reinterpret_cast<const float4 *>(stage + r * kHd + 4 * lane);
                if (w.whole) {
                    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
                    const int tok = r * inv_G >> 16, g = r - tok * B.G;
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv);
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
                    reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(A.out) +
                                              ((int64_t)(w.row0 + tok) * B.Hq + w.h * B.G + g) * kHd)[lane] =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                } else {
                    // l counts 2^-e for values of 2^e: over pages of zeros alone (e = -100) it can be infinite,
                    // and the join would turn that into NaN where it scales the part to nothing
                    *reinterpret_cast<float4 *>(part + r * kPartRow + 4 * lane) = x;
                    if (lane == 0)
                        *reinterpret_cast<float2 *>(part + r * kPartRow + kHd) = make_float2(min_nan(l, FLT_MAX), at);
                }
            }
            if (!w.whole && w.begins && d == 0)
                meta[blockIdx.x] = {w.b, w.h, 0, w.last_cta, 1, {}};
            arrive(sh.l_free[par_q]);
        }
    }
    if (failed)
        atomicOr(&g_attn_decode_error, kErrWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1)
        tc::tmem_dealloc(tmem, C::kTmemCols);
}

int row_pad(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
int most_ctas(int rows, int sms) { return sms * (row_pad(rows) == 16 ? Cfg<16>::kCtas : 1); }

template <int NR>
cudaError_t launch_rows(const AttnArgs &a, int grid, bool may_split, cudaStream_t s)
{
    CUtensorMap mk, mv;
    if (!encode_cache_map(&mk, a.b, a.b.k) || !encode_cache_map(&mv, a.b, a.b.v))
        return cudaErrorInvalidValue;
    constexpr int smem = Cfg<NR>::kEnd + 1024;
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Cfg<NR>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<NR>, a, mk, mv)) != cudaSuccess)
        return e;
    return may_split ? launch_join(a, grid, a.b.G * a.b.max_q, s) : cudaSuccess;
}

}  // namespace

size_t decode_workspace_bytes(int rows, int sms)
{
    return part_bytes((size_t)most_ctas(rows, sms), (size_t)rows);
}

// Calls of up to 16 rows run two CTAs an SM, and so can use more than those of a few rows more.
size_t decode_workspace_for_up_to(int rows, int sms)
{
    const size_t own = decode_workspace_bytes(rows, sms), few = decode_workspace_bytes(rows < 16 ? rows : 16, sms);
    return own > few ? own : few;
}

cudaError_t launch_decode(const AttnArgs &args, cudaStream_t s)
{
    AttnArgs a = args;
    const Batch &b = a.b;
    if (a.window == 0 || a.window > kNoWindow)
        a.window = kNoWindow;
    const int rows = b.G * b.max_q, most = most_ctas(rows, a.sm_count);
    if (most_units(b, kMaxDecodeRows, kOver) > kMostUnits)
        return cudaErrorInvalidConfiguration;
    const int64_t tiles = ((int64_t)b.max_pages * b.P + kTile - 1) / kTile, blocks = (int64_t)b.n_seq * b.Hkv;
    const int64_t units = (tiles + kOver) * blocks;
    const int grid = (int)(units < most ? units : most);
    // the kernel decides by the lengths; where the page table's width decides already, nothing is ever joined
    const bool may_split = tiles > kWhole || blocks > grid || b.n_seq > kFewSeqs;
    switch (row_pad(rows)) {
    case 16: return launch_rows<16>(a, grid, may_split, s);
    case 32: return launch_rows<32>(a, grid, may_split, s);
    default: return launch_rows<64>(a, grid, may_split, s);
    }
}

cudaError_t take_decode_error(int *code)
{
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_decode_error, sizeof(int));
    if (e == cudaSuccess && v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_attn_decode_error, &zero, sizeof(int));
    }
    *code = v;
    return e;
}

}  // namespace attn
}  // namespace gdn
