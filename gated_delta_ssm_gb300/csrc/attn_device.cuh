// attn_device.cuh -- device helpers shared by the attention kernels: a
// sequence's entry of the batch description, checked before it is used.
#pragma once

#include <stdint.h>

#include "attn.h"

namespace gdn {
namespace attn {

constexpr int kHd = 128;   // head dimension

// One sequence of the batch: its token rows [row0, row0 + n) and its length L.
struct Seq {
    int row0, n, L;
    bool ok;
};

// y / G for y below 2^27: with e = inv_G G - 2^31 < 16, 2 y e stays below 2^32.
__device__ __forceinline__ int div_G(const Batch &B, int y) { return (int)__umulhi(2u * (uint32_t)y, B.inv_G); }

// Reads and checks sequence b. An entry out of range gives ok = false and n = 0.
__device__ __forceinline__ Seq load_seq(const Batch &B, int b)
{
    Seq s;
    s.row0 = __ldg(B.q_start + b);
    const int end = __ldg(B.q_start + b + 1);
    s.L = __ldg(B.kv_len + b);
    s.ok = s.row0 >= 0 && end >= s.row0 && end <= B.n_tokens && (int64_t)end - s.row0 <= B.max_q &&
           s.L >= 0 && (int64_t)s.L <= (int64_t)B.max_pages * B.P;
    s.n = s.ok ? end - s.row0 : 0;
    return s;
}

// ------------------------------------------------------------------ partial results
// Where a block of q rows spans several CTAs' shares, the CTA in which it begins describes it here and
// every CTA leaves a part: [2 * grid] slots of `rows` rows, after the descriptions in the workspace.
struct PartMeta {
    int b, h, row0, last_cta;   // row0: the block's first row, token * G + head of the group
    int owner, pad[3];
};
constexpr int kPartRow = kHd + 4;   // 128 sums, l, m, two unused
// The reference m of a row that a part sees no key of: below every other, so that the join goes by the parts that
// hold the row's keys, however low their scores lie; and finite: 2^(-inf - kNoRef) is 0.
constexpr float kNoRef = -1e30f;

__device__ __forceinline__ float *part_slots(uint8_t *ws, unsigned grid)
{
    return reinterpret_cast<float *>(ws + (size_t)grid * sizeof(PartMeta));
}
inline size_t part_bytes(size_t ctas, size_t rows)
{
    return ctas * (sizeof(PartMeta) + 2 * rows * kPartRow * sizeof(float));
}
cudaError_t launch_join(const AttnArgs &a, int grid, int rows, cudaStream_t s);

}  // namespace attn
}  // namespace gdn
