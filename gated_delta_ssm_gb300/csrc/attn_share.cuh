// attn_share.cuh -- how the attention kernels share out a ragged batch.
//
// Work is counted in units of (block of q rows, tile of 128 keys): a sequence's rows, one per (token, head of
// the group) of a KV head, are cut into blocks, and a block meets the key tiles that its rows can see. A block
// counts OVER units on top, ahead of its tiles, for what it costs besides them (its q rows, its output). The
// units of the batch, in the order (sequence, KV head, block, tile), are cut into equal contiguous shares, one
// per CTA, whatever the lengths are; the lengths live on the device, so every CTA counts them itself. One warp
// of a CTA then walks the share and hands the other warps its segments (a block and a run of its tiles) through
// a ring in shared memory; that keeps the walk's code, sequence loads and divisions out of their loops.
#pragma once

#include "attn_device.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace attn {

constexpr int kTile = 128;            // keys per tile
constexpr int kNoWindow = 1 << 30;    // positions are below this
constexpr int kRing = 4;

// A run of key tiles of one block of q rows.
struct Seg {
    int nt, kt;               // tiles (0: the share is done), the first one's index
    int b, h;
    int row0, n, first;       // the sequence's token rows, tokens in the call, position of its first row
    int lo, hi;               // key positions that any row of the block sees
    int blk, tok0, rem0;      // the block's first row (token * G + head of the group), its token and head
    int begins, whole;        // whether the run holds the block's first tile; all of its tiles
    int last_cta;             // the CTA whose share holds the block's last tile
    int pad;
};
static_assert(sizeof(Seg) == 64, "copied as four 16-byte pieces");

struct Ring {
    Seg seg[kRing];
    uint64_t full[kRing], free[kRing];
};

// Batches of at most this many sequences are counted by the walking warp alone, larger ones by the whole CTA.
constexpr int kFewSeqs = 256;

template <int THREADS>
struct ShareShared {
    int warp_sum[THREADS / 32];
    int start_off, head_units;        // the share's first unit within its sequence; units of one KV head there
    int start_b;
    Seq start_seq;
};

// Units are 32-bit numbers: most_units bounds them on the host, by kMostUnits, for sequences that share no rows.
// Where q_start runs backwards, valid sequences can share rows and their units can be more. So sums stop at the
// largest number, and of more than kMostUnits units none is done: nothing could be found by a sum that wrapped.
// (The entry that runs backwards is reported by clear_empty.)
constexpr int kMostUnits = 2000000000;
__device__ __forceinline__ int add_units(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }

// Of `total` units, the first `more` of n_cta
// shares take each + 1, the others `each`: one short division for all that a walk needs.
struct Share {
    int n_cta, each, more;
    int first, count;                 // this CTA's first unit, and its units
    bool split;                       // whether blocks may be split (a unit is a tile, or a whole block)
    int b, off, head_units;           // the first unit's sequence, its place there, units of one KV head there
    Seq s;
};

__device__ __forceinline__ int share_of(const Share &r, int unit)
{
    const int bulk = r.more * (r.each + 1);
    return unit < bulk ? unit / (r.each + 1) : r.more + (unit - bulk) / r.each;
}

// At least the units of any batch of these dimensions.
inline double most_units(const Batch &b, int rows, int over)
{
    const double tiles = (double)(((int64_t)b.max_pages * b.P + kTile - 1) / kTile) + 1 + over;
    return ((double)b.n_tokens * b.G / rows + b.n_seq) * b.Hkv * tiles;
}

// Blocks of a sequence; none where there are no keys.
template <int ROWS>
__device__ __forceinline__ int blocks_of(const Batch &B, const Seq &s)
{
    return s.L > 0 ? (int)((unsigned)(s.n * B.G + ROWS - 1) / ROWS) : 0;
}

// Key positions [lo, hi] that block i of a sequence sees, at least [0, 0].
template <int ROWS>
__device__ __forceinline__ void block_keys(const AttnArgs &A, const Seq &s, int i, int &lo, int &hi)
{
    const int first = s.L - s.n;
    lo = max(0, first + div_G(A.b, i * ROWS) - A.window + 1);
    hi = max(0, first + min(div_G(A.b, i * ROWS + ROWS - 1), s.n - 1));
}

template <int ROWS>
__device__ __forceinline__ int block_tiles(const AttnArgs &A, const Seq &s, int i)
{
    int lo, hi;
    block_keys<ROWS>(A, s, i, lo, hi);
    return hi / kTile - lo / kTile + 1;
}

// A block's units: its tiles and OVER, or one where blocks are not split.
template <int ROWS, int OVER>
__device__ __forceinline__ int block_units(const AttnArgs &A, const Seq &s, int i, bool split)
{
    return split ? block_tiles<ROWS>(A, s, i) + OVER : 1;
}

// Tiles of one KV head of a sequence, of blocks from, from + step, ..; their number and the longest's tiles are
// added to `blocks` and `longest`.
template <int ROWS>
__device__ __forceinline__ int head_tiles(const AttnArgs &A, int b, int from, int step, int &blocks, int &longest)
{
    const Seq s = load_seq(A.b, b);
    const int n = blocks_of<ROWS>(A.b, s);
    int u = 0;
#pragma unroll 1
    for (int i = from; i < n; i += step) {
        const int t = block_tiles<ROWS>(A, s, i);
        u += t;
        longest = max(longest, t);
        ++blocks;
    }
    return u;
}

// Count the batch and find where this CTA's share begins, by `threads` threads of which this is number tid
// (whole warps). sync joins them.
template <int ROWS, int OVER, int WHOLE, int THREADS, typename Y>
__device__ __forceinline__ Share find_share(const AttnArgs &A, ShareShared<THREADS> &sh, int tid, int threads, Y sync)
{
    const Batch &B = A.b;
    const int warp = tid >> 5, lane = tid & 31;
    // a group of g neighbouring lanes counts one sequence, or a thread several where there are many
    int g = 1;
    while (g < 32 && B.n_seq * g * 2 <= threads)
        g *= 2;
    const int per = g > 1 ? 1 : (B.n_seq + threads - 1) / threads;
    const int first_b = (tid / g) * per, sub = tid % g;
    int mine = 0;
    int blocks = 0, longest = 0;
#pragma unroll 2
    for (int i = 0; i < per; ++i)
        if (first_b + i < B.n_seq)
            mine = add_units(mine, head_tiles<ROWS>(A, first_b + i, sub, g, blocks, longest));
    for (int m = 1; m < g; m <<= 1) {
        mine += __shfl_xor_sync(0xffffffffu, mine, m);
        blocks += __shfl_xor_sync(0xffffffffu, blocks, m);
    }
    // Few short blocks go to a CTA each, whole: to split them would cost more in joining than it saves.
    // (Looked at where one warp counts; a batch of more than kFewSeqs sequences is always split, which costs its few
    // split blocks a join.)
    bool split = true;
    if (threads == 32) {
        int all = sub == 0 ? blocks : 0;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, m);
            longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, m));
        }
        split = longest > WHOLE || (int64_t)all * B.Hkv > gridDim.x;
    }
    const int64_t head = split ? mine + (int64_t)OVER * blocks : blocks;
    const int one_head = (int)head;   // where it is used, of one sequence
    mine = sub == 0 ? (int)min(head * B.Hkv, (int64_t)0x7fffffff) : 0;
    int incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m)
            incl = add_units(incl, up);
    }
    Share r;
    int total = __shfl_sync(0xffffffffu, incl, 31);
    if (threads > 32) {
        if (lane == 31)
            sh.warp_sum[warp] = incl;
        sync();
        total = 0;
#pragma unroll 1
        for (int i = 0; i < threads / 32; ++i) {
            incl = add_units(incl, i < warp ? sh.warp_sum[i] : 0);
            total = add_units(total, sh.warp_sum[i]);
        }
    }
    if (total > kMostUnits)
        total = 0;
    const int c = blockIdx.x;
    r.n_cta = min((int)gridDim.x, total);
    r.each = r.n_cta > 0 ? total / r.n_cta : 1;
    r.more = total - r.each * r.n_cta;
    r.first = r.each * c + min(c, r.more);
    r.count = c < r.n_cta ? r.each + (c < r.more ? 1 : 0) : 0;
    if (r.count > 0 && r.first < incl && r.first >= incl - mine) {   // among this thread's sequences
        int at = incl - mine;
#pragma unroll 1
        for (int i = 0; i < per && first_b + i < B.n_seq; ++i) {
            int n = 0, most = 0, u = one_head;
            if (per > 1) {
                u = head_tiles<ROWS>(A, first_b + i, 0, 1, n, most);
                u = split ? u + OVER * n : n;
            }
            if (r.first < at + u * B.Hkv) {
                sh.start_b = first_b + i;
                sh.start_off = r.first - at;
                sh.head_units = u;
                sh.start_seq = load_seq(B, first_b + i);
                break;
            }
            at += u * B.Hkv;
        }
    }
    sync();
    r.split = split;
    r.b = sh.start_b;
    r.off = sh.start_off;
    r.head_units = sh.head_units;
    r.s = sh.start_seq;
    return r;
}

// One warp walks the share and fills the ring; `wait` is the kernel's bounded wait, *abort what it leaves when it
// gives up.
template <int ROWS, int OVER, typename W>
__device__ __forceinline__ void walk_share(const AttnArgs &A, const Share &r, Ring &ring, W wait,
                                           const volatile int *abort)
{
    const Batch &B = A.b;
    const int lane = threadIdx.x & 31;
    int b = 0, h = 0, i = 0, t = 0, n = 0;
    Seq s = {};
    if (r.count > 0) {   // the block and tile of the first unit: each lane looks through a part of the blocks
        b = r.b;
        s = r.s;
        n = blocks_of<ROWS>(B, s);
        h = r.off < r.head_units ? 0 : r.off / r.head_units;
        t = r.off - h * r.head_units;
    }
    if (n > 1) {
        const int off = t;
        const int each = (n + 31) / 32, i0 = min(n, lane * each), i1 = min(n, i0 + each);
        int u = 0;
#pragma unroll 1
        for (int k = i0; k < i1; ++k)
            u += block_units<ROWS, OVER>(A, s, k, r.split);
        int upto = u;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m)
                upto += up;
        }
        const bool here = off < upto && off >= upto - u;
        int at = upto - u;
        if (here)
#pragma unroll 1
            for (i = i0; i < i1; ++i) {
                const int k = block_units<ROWS, OVER>(A, s, i, r.split);
                if (off < at + k)
                    break;
                at += k;
            }
        const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        i = __shfl_sync(0xffffffffu, i, from & 31);
        t = __shfl_sync(0xffffffffu, off - at, from & 31);
    }
    int left = r.count;
    int unit = r.first;
#pragma unroll 1
    for (int k = 0;;) {
        Seg q = {};
        if (left > 0) {
            int lo, hi;
            block_keys<ROWS>(A, s, i, lo, hi);
            const int all = hi / kTile - lo / kTile + 1, units = r.split ? all + OVER : 1;
            const int end = min(units, t + left), t0 = r.split ? max(0, t - OVER) : 0;
            q.nt = r.split ? max(0, end - OVER) - t0 : all;
            q.kt = lo / kTile + t0;
            q.b = b, q.h = h, q.row0 = s.row0, q.n = s.n, q.first = s.L - s.n, q.lo = lo, q.hi = hi;
            q.blk = i * ROWS;
            q.tok0 = div_G(B, q.blk);
            q.rem0 = q.blk - q.tok0 * B.G;
            q.begins = t0 == 0;
            q.whole = q.nt == all;
            q.last_cta = share_of(r, unit + (units - t) - 1);
            left -= end - t;
            unit += end - t;
            t = 0;
            if (left > 0 && ++i == n) {
                i = 0;
                if (++h == B.Hkv) {
                    h = 0;
                    do {
                        if (++b >= B.n_seq) {   // not reached while the batch stays as it was counted
                            left = 0;
                            break;
                        }
                        s = load_seq(B, b);
                        n = blocks_of<ROWS>(B, s);
                    } while (n == 0);
                }
            }
            if (q.nt == 0)   // the share ends ahead of the block's first tile
                continue;
        }
        const int slot = k % kRing;
        if (k >= kRing)
            wait(ring.free[slot], (k / kRing - 1) & 1);
        if (__any_sync(0xffffffffu, *abort != 0))
            return;
        if (lane == 0) {
            ring.seg[slot] = q;
            tc::mbar_arrive(tc::smem_addr(&ring.full[slot]));
        }
        if (q.nt == 0)
            return;
        ++k;
    }
}

// Segment k of the ring, for a whole warp; its slot is handed back at once. After a wait that gave up there are
// no more segments: the walk has stopped, and what the slot holds is an old one.
template <typename W>
__device__ __forceinline__ Seg take_seg(Ring &ring, int k, W wait, const volatile int *abort)
{
    const int slot = k % kRing;
    wait(ring.full[slot], (k / kRing) & 1);
    Seg q = ring.seg[slot];
    if (__any_sync(0xffffffffu, *abort != 0))
        q.nt = 0;
    __syncwarp();   // every lane has read the slot (a vote orders no memory)
    if ((threadIdx.x & 31) == 0)
        tc::mbar_arrive(tc::smem_addr(&ring.free[slot]));
    return q;
}

// For GDN_CHECK: a segment lies in the batch. Everything that a role indexes with is one of its fields, or a thread's
// place within rows, tile or page beside them.
__device__ __forceinline__ bool seg_in_range(const AttnArgs &A, const Seg &w)
{
    const Batch &B = A.b;
    return w.b >= 0 && w.b < B.n_seq && w.h >= 0 && w.h < B.Hkv && w.row0 >= 0 && w.n >= 1 && w.n <= B.max_q &&
           w.row0 + w.n <= B.n_tokens && w.lo >= 0 && w.hi >= w.lo && w.hi < B.max_pages * B.P &&
           w.kt >= w.lo / kTile && w.kt + w.nt - 1 <= w.hi / kTile && w.blk >= 0 && w.blk < w.n * B.G &&
           w.tok0 * B.G + w.rem0 == w.blk && w.rem0 >= 0 && w.rem0 < B.G && w.last_cta >= (int)blockIdx.x &&
           w.last_cta < (int)gridDim.x && (w.begins || blockIdx.x > 0);
}

// Sequences without keys: nobody else looks at them. Their rows are zero, and bad entries are reported.
__device__ __forceinline__ void clear_empty(const AttnArgs &A, int *error)
{
    const Batch &B = A.b;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int b = blockIdx.x; b < B.n_seq; b += gridDim.x) {
        const Seq s = load_seq(B, b);
        if (!s.ok && lane == 0)
            atomicOr(error, kErrMeta);
        if (s.ok && s.L == 0) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(A.out) + (int64_t)s.row0 * B.Hq * kHd * 2);
            for (int64_t e = lane; e < (int64_t)s.n * B.Hq * (kHd / 8); e += 32)
                o[e] = make_uint4(0, 0, 0, 0);
        }
    }
}

}  // namespace attn
}  // namespace gdn
