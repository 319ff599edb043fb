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

}  // namespace attn
}  // namespace gdn
