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
// below 256 is hi + lo exactly (down to 2^-18 of that largest value); a weight
// keeps 2^-8 of itself, as many bits as bf16 has.
//   The key scale of a page and the value scale 2^e enter the exponent:
// w = s f ks + e, P = 2^(w - max w + 8) <= 256 over the tile, so a tile's own
// largest weight sets the steps of P. Tiles are joined in 32-bit registers,
// O = O alpha + O_tile beta, not by the tensor core's accumulator; the sum of
// weights takes P 2^-e before P is rounded.
//
// Bound by memory: 256 bytes of codes per key and KV head. The batch's tiles are
// counted over (sequence, KV head), and the grid's CTAs take equal contiguous
// shares of them, so ragged lengths cost nothing; a (sequence, head) that spans
// CTAs leaves 32-bit partial results which a second kernel joins.
//
// Roles of a CTA: warp 0 copies pages to shared memory, warp 1 issues the
// products, warps 2-3 split the q rows of the next (sequence, head), warps 4-7
// hold a key each and turn scores into weights, warps 8-11 hold a dimension each
// and join the tiles.
#include "attn_tc.cuh"
#include "cluster.cuh"
#include "gdn_device.cuh"

namespace gdn {
namespace attn {

static __device__ int g_attn_decode_error;

namespace {

constexpr int kThreads = 384;

template <int NR>
struct Cfg {
    // tiles in flight, K and V counted apart (item 2 i is K of tile i, 2 i + 1 its V)
    static constexpr int kItems = NR == 16 ? 5 : NR == 32 ? 10 : 8;
    static constexpr int kCtas = NR == 16 ? 2 : 1;               // CTAs per SM
    static constexpr uint32_t kRowBytes = NR * kHd;              // one e4m3 operand of NR rows
    static constexpr uint32_t kQ = kItems * kTileBytes;          // [2 segments][hi, lo]
    static constexpr uint32_t kP = kQ + 4 * kRowBytes;           // [2 tiles][hi, lo]
    static constexpr uint32_t kEnd = kP + 4 * kRowBytes;
    static constexpr uint32_t kTmemCols = 4 * NR;
};

template <int NR>
struct Shared {
    uint64_t full[Cfg<NR>::kItems], empty[Cfg<NR>::kItems], drain;
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2], q_full[2], q_free[2], l_full[2], l_free[2], coef_full[4];
    uint32_t tmem;
    volatile int abort;
    int start_b;
    int64_t start_off;
    int64_t warp_sum[kThreads / 32];
    float4 coef[4][NR];        // {tile max, alpha, beta} of each row, four tiles deep
    float f[2][NR];            // scale * log2 e / (power of two of the q row)
    int limit[2][NR];          // position of each row
    float warp_max[4][NR];
    float l_sum[2][4][NR];
    float w_max[2][NR];
};

// The tiles of a sequence: keys [lo, L) that any of its rows can see.
struct Tiles {
    Seq s;
    int lo, t0, n;
};

__device__ __forceinline__ Tiles seq_tiles(const AttnArgs &A, int b)
{
    Tiles t;
    t.s = load_seq(A.b, b);
    const int first = t.s.L - t.s.n;              // position of the first row
    t.lo = max(0, first - A.window + 1);
    t.t0 = t.lo / kTile;
    t.n = t.s.n > 0 && t.s.L > 0 ? (t.s.L + kTile - 1) / kTile - t.t0 : 0;
    return t;
}

// A CTA's share of the batch: segments (sequence, KV head, tiles [t, end)).
struct Walk {
    int b, h, t, end;          // current segment, tiles counted from the sequence's first
    int left;                  // tiles of the share from t on
    Tiles q;
    __device__ __forceinline__ bool begins() const { return t == 0; }
    __device__ __forceinline__ bool ends() const { return end == q.n; }
    __device__ __forceinline__ void cut() { end = min(q.n, t + left); }
    __device__ __forceinline__ bool next(const AttnArgs &A)   // false at the end of the share
    {
        left -= end - t;
        if (left <= 0)
            return false;
        t = 0;
        if (++h == A.b.Hkv) {
            h = 0;
            do {
                if (++b >= A.b.n_seq)
                    return false;
                q = seq_tiles(A, b);
            } while (q.n == 0);
        }
        cut();
        return true;
    }
};

template <typename S>
__device__ __forceinline__ Walk walk_start(const AttnArgs &A, const S &sh, int count)
{
    Walk w;
    w.b = sh.start_b;
    w.q = seq_tiles(A, w.b);
    w.h = (int)(sh.start_off / w.q.n);
    w.t = (int)(sh.start_off - (int64_t)w.h * w.q.n);
    w.left = count;
    w.cut();
    return w;
}

template <int NR>
__global__ void __launch_bounds__(kThreads, Cfg<NR>::kCtas)
attn_decode_kernel(const __grid_constant__ AttnArgs A, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v)
{
    using C = Cfg<NR>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared<NR> sh;
    const Batch &B = A.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (tc::smem_addr(dyn) + 1023u) & ~1023u;
    uint8_t *const mem = dyn + (base - tc::smem_addr(dyn));
    const int R = B.G * B.max_q, Rp = (R + 3) & ~3;

    if (tid == 0) {
        for (int i = 0; i < C::kItems; ++i) {
            tc::mbar_init(tc::smem_addr(&sh.full[i]), 1);
            tc::mbar_init(tc::smem_addr(&sh.empty[i]), 1);
        }
        tc::mbar_init(tc::smem_addr(&sh.drain), 1);
        for (int i = 0; i < 4; ++i)
            tc::mbar_init(tc::smem_addr(&sh.coef_full[i]), 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_addr(&sh.s_full[i]), 1);
            tc::mbar_init(tc::smem_addr(&sh.p_full[i]), 128);
            tc::mbar_init(tc::smem_addr(&sh.o_full[i]), 1);
            tc::mbar_init(tc::smem_addr(&sh.o_free[i]), 128);
            tc::mbar_init(tc::smem_addr(&sh.q_full[i]), 64);
            tc::mbar_init(tc::smem_addr(&sh.q_free[i]), 129);
            tc::mbar_init(tc::smem_addr(&sh.l_full[i]), 128);
            tc::mbar_init(tc::smem_addr(&sh.l_free[i]), 128);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.abort = 0;
        sh.start_b = 0;
    }
    if (warp == 1)
        tc::tmem_alloc(tc::smem_addr(&sh.tmem), C::kTmemCols);
    // rows of P that no q row uses stay zero
    for (uint32_t i = tid; i < 4 * C::kRowBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(mem + C::kP)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_smem_to_async();

    wait_previous_grid();
    // ---- the batch's tiles, and where this CTA's share of them begins
    const int per = (B.n_seq + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < B.n_seq)
            mine += seq_tiles(A, b).n;
    }
    mine *= B.Hkv;
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
    int64_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        before += i < warp ? sh.warp_sum[i] : 0;
        total += sh.warp_sum[i];
    }
    incl += before;
    const int n_cta = (int)min((int64_t)gridDim.x, total);
    const bool works = (int)blockIdx.x < n_cta;
    const int64_t first = works ? share_begin(total, n_cta, blockIdx.x) : 0;
    const int count = works ? (int)(share_begin(total, n_cta, blockIdx.x + 1) - first) : 0;
    if (works && first < incl && first >= incl - mine) {   // one thread's sequences hold it
        int64_t at = incl - mine;
        for (int i = 0; i < per && tid * per + i < B.n_seq; ++i) {
            const int64_t u = (int64_t)seq_tiles(A, tid * per + i).n * B.Hkv;
            if (first < at + u) {
                sh.start_b = tid * per + i;
                sh.start_off = first - at;
                break;
            }
            at += u;
        }
    }
    PartMeta *const meta = reinterpret_cast<PartMeta *>(A.ws);
    float *const parts = part_slots(A.ws, gridDim.x);
    if (tid == 0)
        meta[blockIdx.x].owner = 0;
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

    if (warp == 0) {
        // ------------------------------------------------------------ pages to shared memory
        if (works) {
            Walk w = walk_start(A, sh, count);
            int i = 0, issued = 0;
            const int per_tile = kTile / B.P;
            do {
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
                const int pg_lo = w.q.lo / B.P, pg_hi = (w.q.s.L - 1) / B.P;
                auto page_of = [&](int t) {   // this lane's page of the tile, -1: none wanted, -2: bad
                    const int pg = (w.q.t0 + t) * per_tile + lane;
                    if (lane >= per_tile || pg < pg_lo || pg > pg_hi)
                        return -1;
                    const int p = __ldg(table + pg);
                    return p >= 0 && p < B.n_pages ? p : -2;
                };
                int page = page_of(w.t);
                for (int t = w.t; t < w.end; ++t) {
                    const int next = t + 1 < w.end ? page_of(t + 1) : -1;
                    const bool have = page >= 0;
                    if (page == -2)
                        atomicOr(&g_attn_decode_error, kErrMeta);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * B.P * kHd;
#pragma unroll
                    for (int part = 0; part < 2; ++part, ++i) {
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
                    page = next;
                }
            } while (w.next(A));
            // after a wait that gave up: the copies in flight land before the CTA ends
            for (int k = max(0, issued - C::kItems); k < issued && sh.abort; ++k)
                tc::mbar_wait_ns(tc::smem_addr(&sh.full[k % C::kItems]), (k / C::kItems) & 1, lim);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        if (works && lane == 0) {
            constexpr uint32_t idesc_s = idesc_e4m3(128, NR);
            constexpr uint32_t idesc_o = idesc_e4m3(128, NR) | kIdescTransA;
            Walk w = walk_start(A, sh, count);
            int i = 0, seg = 0, t = w.t;   // the next tile of scores: i of the share, t of segment seg
            auto scores = [&]() {
                if (i == count)
                    return;
                const int item = 2 * i, st = item % C::kItems;
                wait1(sh.q_full[seg & 1], (seg >> 1) & 1);
                wait1(sh.full[st], (item / C::kItems) & 1);
                tc::fence_after_sync();
                if (!sh.abort) {
                    const uint64_t k = tc::sdesc_sw128(base + st * kTileBytes);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint64_t q =
                            tc::sdesc_sw128(base + C::kQ + ((seg & 1) * 2 + part) * C::kRowBytes);
#pragma unroll
                        for (int s = 0; s < 4; ++s)   // 32 bytes of the 128-byte rows at a time
                            mma_e4m3(tmem + (i & 1) * NR, k + 2 * s, q + 2 * s, idesc_s, part + s > 0);
                    }
                }
                tc::mma_commit(tc::smem_addr(&sh.s_full[i & 1]));
                tc::mma_commit(tc::smem_addr(&sh.empty[st]));
                ++i;
                if (++t == w.end) {
                    tc::mma_commit(tc::smem_addr(&sh.q_free[seg & 1]));
                    ++seg;
                    if (w.next(A))
                        t = w.t;
                }
            };
            scores();
            scores();
            for (int j = 0; j < count; ++j) {
                const int item = 2 * j + 1, st = item % C::kItems, k = j & 1;
                if (j >= 2)
                    wait1(sh.o_free[k], (j / 2 - 1) & 1);
                wait1(sh.full[st], (item / C::kItems) & 1);
                wait1(sh.p_full[k], (j / 2) & 1);
                tc::fence_after_sync();
                if (!sh.abort) {
                    const uint64_t v = tc::sdesc_sw128_mn(base + st * kTileBytes, 1024, 1024);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint64_t p = tc::sdesc_sw128(base + C::kP + (k * 2 + part) * C::kRowBytes);
#pragma unroll
                        for (int s = 0; s < 4; ++s)   // 32 keys: 4 KB of V, 32 bytes of P's rows
                            mma_e4m3(tmem + 2 * NR + k * NR, v + 256 * s, p + 2 * s, idesc_o, part + s > 0);
                    }
                }
                tc::mma_commit(tc::smem_addr(&sh.o_full[k]));
                tc::mma_commit(tc::smem_addr(&sh.empty[st]));
                scores();
            }
            if (sh.abort) {   // products in flight end before the tensor memory is freed
                tc::mma_commit(tc::smem_addr(&sh.drain));
                tc::mbar_wait_ns(tc::smem_addr(&sh.drain), 0, lim);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------ q rows
        const int t64 = tid - 64, u = t64 & 7, r8 = t64 >> 3;
        // sequences without keys: nobody else looks at them
        for (int b = blockIdx.x; b < B.n_seq; b += gridDim.x) {
            const Tiles q = seq_tiles(A, b);
            if (!q.s.ok && t64 == 0)
                atomicOr(&g_attn_decode_error, kErrMeta);
            if (q.s.ok && q.n == 0) {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(A.out) +
                                                     (int64_t)q.s.row0 * B.Hq * kHd);
                for (int64_t c = t64; c < (int64_t)q.s.n * B.Hq * (kHd / 8); c += 64)
                    o[c] = make_uint4(0, 0, 0, 0);
            }
        }
        if (works) {
            Walk w = walk_start(A, sh, count);
            int seg = 0;
            do {
                const int k = seg & 1;
                if (seg >= 2)
                    wait(sh.q_free[k], (seg / 2 - 1) & 1);
                for (int r = r8; r < NR; r += 8) {
                    const int tok = r / B.G, g = r - tok * B.G;
                    const bool live = tok < w.q.s.n;
                    float v[16] = {};
                    if (live)
                        load_q16(static_cast<const __nv_bfloat16 *>(A.q) +
                                     (int64_t)(w.q.s.row0 + tok) * A.q_stride + (w.h * B.G + g) * kHd + u * 16,
                                 v);
                    float top = 0.0f;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        top = fmaxf(top, fabsf(v[e]));
#pragma unroll
                    for (int m = 1; m < 8; m <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                    const int ex = q_exponent(top);
                    store_q16(mem + C::kQ + k * 2 * C::kRowBytes + (r >> 3) * 1024 + (r & 7) * 128 +
                                  ((u ^ (r & 7)) << 4),
                              C::kRowBytes, v, q_factor(top));
                    if (u == 0) {
                        sh.f[k][r] = A.scale * kLog2e * pow2i(-ex);
                        sh.limit[k][r] = live ? w.q.s.L - w.q.s.n + tok : -1;
                    }
                }
                tc::fence_smem_to_async();
                tc::mbar_arrive(tc::smem_addr(&sh.q_full[k]));
                ++seg;
            } while (w.next(A));
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ scores to weights: a key per thread
        if (works) {
            const int t = tid - 128, wq = warp & 3;
            const uint32_t lane_at = (uint32_t)(wq * 32) << 16;
            Walk w = walk_start(A, sh, count);
            int i = 0, seg = 0;
            float l[NR], big = -INFINITY;   // big: this thread's row's running maximum (thread t < NR)
            const float cap2 = A.softcap * kLog2e, inv_cap2 = A.softcap > 0.0f ? 1.0f / cap2 : 0.0f;
            do {
                const int k = seg & 1;
                const int L = w.q.s.L, first_row = L - w.q.s.n;
                const int32_t *table = B.page_table + (int64_t)w.b * B.max_pages;
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    l[r] = 0.0f;
                big = -INFINITY;
                auto page_at = [&](int tl) {
                    const int j = (w.q.t0 + tl) * kTile + t;
                    if (tl >= w.end || j < w.q.lo || j >= L)
                        return -1;
                    const int p = __ldg(table + j / B.P);
                    return p >= 0 && p < B.n_pages ? p : -1;
                };
                auto scale_at = [&](const float *s, int p) {
                    return p >= 0 ? __ldg(s + (int64_t)p * B.Hkv + w.h) : 1.0f;
                };
                int p_next = page_at(w.t), p_far = page_at(w.t + 1);
                float ks_next = scale_at(B.k_scale, p_next), vs_next = scale_at(B.v_scale, p_next);
                wait(sh.q_full[k], (seg >> 1) & 1);
                for (int tl = w.t; tl < w.end; ++tl, ++i) {
                    const int par = i & 1;
                    const float ks = ks_next, vs = vs_next;
                    const bool dead = p_next < 0;
                    p_next = p_far;
                    ks_next = scale_at(B.k_scale, p_next);
                    vs_next = scale_at(B.v_scale, p_next);
                    p_far = page_at(tl + 2);
                    const int j0 = (w.q.t0 + tl) * kTile, j = j0 + t;
                    // every row sees the whole tile
                    const bool whole = j0 + kTile - 1 <= first_row && j0 > L - 1 - A.window;
                    const float ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
                    const float iv = 1.0f / vs;
                    wait(sh.s_full[par], (i >> 1) & 1);
                    tc::fence_after_sync();
                    float x[NR];
#pragma unroll
                    for (int c = 0; c < NR; c += 16)
                        tc::tmem_ld16(tmem + par * NR + c + lane_at, *reinterpret_cast<float(*)[16]>(x + c));
                    float mx[(NR + 31) / 32];
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r % 4 == 0 && r >= R)
                            break;
                        const float fk = sh.f[k][r] * ks;
                        if (A.softcap > 0.0f)
                            x[r] = fmaf(cap2, tanh_cap(x[r] * fk * inv_cap2), ev);
                        else
                            x[r] = fmaf(x[r], fk, ev);
                        bool hide = dead;
                        if (!whole) {
                            const int at = sh.limit[k][r];
                            hide |= j > at || j <= at - A.window;
                        }
                        x[r] = hide ? -INFINITY : x[r];
                        const float m = redux_max(x[r]);
                        if (lane == (r & 31))
                            mx[r / 32] = m;
                    }
#pragma unroll
                    for (int c = 0; c < (NR + 31) / 32; ++c)
                        if (c * 32 + lane < Rp)
                            sh.warp_max[wq][c * 32 + lane] = mx[c];
                    named_sync(1, 128);
                    if (t < Rp) {
                        const float top = fmaxf(fmaxf(sh.warp_max[0][t], sh.warp_max[1][t]),
                                                fmaxf(sh.warp_max[2][t], sh.warp_max[3][t]));
                        const float grown = fmaxf(big, top);
                        const bool none = grown == -INFINITY;
                        // P is 2^(w - top + 8): at most 256
                        sh.coef[i & 3][t] = make_float4(top == -INFINITY ? 0.0f : top - 8.0f,
                                                        none ? 1.0f : ex2(big - grown),
                                                        none ? 0.0f : ex2(top - grown), 0.0f);
                        big = grown;
                    }
                    named_sync(1, 128);
                    if (t == 0)
                        tc::mbar_arrive(tc::smem_addr(&sh.coef_full[i & 3]));
                    uint8_t *const prow = mem + C::kP + par * 2 * C::kRowBytes + (t & 15);
#pragma unroll
                    for (int r = 0; r < NR; r += 2) {
                        if (r % 4 == 0 && r >= R)
                            break;
                        const float4 c0 = sh.coef[i & 3][r], c1 = sh.coef[i & 3][r + 1];
                        const float p0 = ex2(x[r] - c0.x), p1 = ex2(x[r + 1] - c1.x);
                        l[r] = fmaf(l[r], c0.y, p0 * (c0.z * iv));
                        l[r + 1] = fmaf(l[r + 1], c1.y, p1 * (c1.z * iv));
                        uint32_t h8, l8;
                        split_e4m3(p0, p1, h8, l8);
                        uint8_t *a = prow + (r >> 3) * 1024 + (r & 7) * 128 + (((t >> 4) ^ (r & 7)) << 4);
                        uint8_t *b = prow + (r >> 3) * 1024 + ((r + 1) & 7) * 128 +
                                     (((t >> 4) ^ ((r + 1) & 7)) << 4);
                        a[0] = (uint8_t)h8;
                        b[0] = (uint8_t)(h8 >> 8);
                        a[C::kRowBytes] = (uint8_t)l8;
                        b[C::kRowBytes] = (uint8_t)(l8 >> 8);
                    }
                    if (dead) {
                        // nothing of the cache lies here, or nothing that may be seen: any code, NaN
                        // among them; its value row is cleared so that weight 0 gives 0
                        const int item = 2 * i + 1, st = item % C::kItems;
                        wait1(sh.full[st], (item / C::kItems) & 1);
                        uint4 *row = reinterpret_cast<uint4 *>(mem + st * kTileBytes + t * kHd);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            row[c] = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_smem_to_async();
                    tc::fence_before_sync();
                    tc::mbar_arrive(tc::smem_addr(&sh.p_full[par]));
                }
                tc::mbar_arrive(tc::smem_addr(&sh.q_free[k]));
                // the segment's sums and maxima
                if (seg >= 2)
                    wait(sh.l_free[k], (seg / 2 - 1) & 1);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    if (r % 4 == 0 && r >= R)
                        break;
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1)
                        l[r] += __shfl_xor_sync(0xffffffffu, l[r], m);
                    if (lane == 0)
                        sh.l_sum[k][wq][r] = l[r];
                }
                if (t < R)
                    sh.w_max[k][t] = big;
                tc::mbar_arrive(tc::smem_addr(&sh.l_full[k]));
                ++seg;
            } while (w.next(A));
        }
    } else {
        // ------------------------------------------------------------ tiles joined: a dimension per thread
        if (works) {
            const int d = tid - 256, wq = warp & 3;
            const uint32_t lane_at = (uint32_t)(wq * 32) << 16;
            Walk w = walk_start(A, sh, count);
            int i = 0, seg = 0;
            float o[NR];
            do {
                const int k = seg & 1;
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    o[r] = 0.0f;
                for (int tl = w.t; tl < w.end; ++tl, ++i) {
                    const int par = i & 1;
                    wait(sh.coef_full[i & 3], (i >> 2) & 1);
                    wait(sh.o_full[par], (i >> 1) & 1);
                    tc::fence_after_sync();
                    float x[NR];
#pragma unroll
                    for (int c = 0; c < NR; c += 16)
                        tc::tmem_ld16(tmem + 2 * NR + par * NR + c + lane_at,
                                      *reinterpret_cast<float(*)[16]>(x + c));
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r % 4 == 0 && r >= R)
                            break;
                        const float4 c = sh.coef[i & 3][r];
                        o[r] = fmaf(o[r], c.y, x[r] * c.z);
                    }
                    tc::fence_before_sync();
                    tc::mbar_arrive(tc::smem_addr(&sh.o_free[par]));
                }
                wait(sh.l_full[k], (seg >> 1) & 1);
                const bool whole = w.begins() && w.ends();
                const int rows = w.q.s.n * B.G;
                if (whole) {
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(A.out) +
                                         ((int64_t)w.q.s.row0 * B.Hq + (int64_t)w.h * B.G) * kHd + d;
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r >= rows)
                            break;
                        const float l = (sh.l_sum[k][0][r] + sh.l_sum[k][1][r]) +
                                        (sh.l_sum[k][2][r] + sh.l_sum[k][3][r]);
                        const int tok = r / B.G, g = r - tok * B.G;
                        out[((int64_t)tok * B.Hq + g) * kHd] =
                            __float2bfloat16_rn(l > 0.0f ? o[r] / l : (l == l ? 0.0f : l));
                    }
                } else {
                    const int slot = 2 * blockIdx.x + (w.begins() ? 1 : 0);
                    float *dst = parts + (size_t)slot * R * kPartRow;
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if (r >= rows)
                            break;
                        dst[r * kPartRow + d] = o[r];
                        if (d == 0) {
                            dst[r * kPartRow + kHd] = (sh.l_sum[k][0][r] + sh.l_sum[k][1][r]) +
                                                     (sh.l_sum[k][2][r] + sh.l_sum[k][3][r]);
                            dst[r * kPartRow + kHd + 1] = sh.w_max[k][r];
                        }
                    }
                    if (w.begins() && d == 0) {
                        const int64_t end_unit = first + count - w.left + (w.q.n - w.t);   // past its last tile
                        meta[blockIdx.x] = {w.b, w.h, 0, share_of(total, n_cta, end_unit - 1), 1, {}};
                    }
                }
                tc::mbar_arrive(tc::smem_addr(&sh.l_free[k]));
                ++seg;
            } while (w.next(A));
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
cudaError_t launch_rows(const AttnArgs &a, int grid, cudaStream_t s)
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<NR>, a, mk, mv)) != cudaSuccess)
        return e;
    return launch_join(a, grid, a.b.G * a.b.max_q, s);
}

}  // namespace

size_t decode_workspace_bytes(int rows, int sms)
{
    return part_bytes((size_t)most_ctas(rows, sms), (size_t)rows);
}

cudaError_t launch_decode(const AttnArgs &args, cudaStream_t s)
{
    AttnArgs a = args;
    const Batch &b = a.b;
    if (a.window == 0 || a.window > kNoWindow)
        a.window = kNoWindow;
    const int rows = b.G * b.max_q;
    const int64_t tiles = ((int64_t)b.max_pages * b.P + kTile - 1) / kTile * b.n_seq * b.Hkv;
    const int grid = (int)(tiles < most_ctas(rows, a.sm_count) ? tiles : most_ctas(rows, a.sm_count));
    switch (row_pad(rows)) {
    case 16: return launch_rows<16>(a, grid, s);
    case 32: return launch_rows<32>(a, grid, s);
    default: return launch_rows<64>(a, grid, s);
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
