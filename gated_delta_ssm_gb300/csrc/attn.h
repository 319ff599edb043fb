// attn.h -- internal launch interface of the attention operators over the paged
// 8-bit key/value cache, between the C ABI (abi.cu) and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace attn {

constexpr int kErrMeta = 256;       // q_start, kv_len, page_table or a position out of range
constexpr int kErrNonFinite = 512;  // append: a key or value that is not finite
constexpr int kErrWait = 1024;      // a bounded wait gave up

constexpr int64_t kMostRows = (1 << 27) - 256;  // most (token, head of a group) rows of a call
constexpr int kMaxGroup = 16;       // most q heads per KV head
constexpr int kMaxDecodeRows = 64;  // most (head of a group, token) rows per KV head in a decode call

// What every attention kernel gets: the batch, the cache and its sizes.
struct Batch {
    uint8_t *k, *v;                 // e4m3 [n_pages][Hkv][P][128]
    float *k_scale, *v_scale;       // [n_pages][Hkv]
    const int32_t *page_table;      // [n_seq][max_pages]
    const int32_t *q_start, *kv_len;
    int n_seq, Hq, Hkv, G, P, n_pages, max_pages, n_tokens, max_q;
    uint32_t inv_G;                 // ceil(2^31 / G)
};

struct AppendArgs {
    Batch b;
    const void *q, *k, *v;          // act rows
    int64_t q_stride, k_stride, v_stride;
    const float *cos, *sin;         // [n_positions][rot / 2]
    int n_positions, rot, interleaved;
    void *q_out;                    // bf16 [n_tokens][Hq][128]
};

struct AttnArgs {
    Batch b;
    const void *q;                  // bf16 rows
    int64_t q_stride;
    void *out;                      // bf16 [n_tokens][Hq][128]
    float scale, softcap;
    int window;
    uint8_t *ws;
    int sm_count;
    uint64_t wait_ns, first_wait_ns;   // limits of the bounded waits, and of a CTA's first
};

cudaError_t launch_append(const AppendArgs &a, bool bf16, cudaStream_t s);
cudaError_t launch_decode(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_prefill(const AttnArgs &a, cudaStream_t s);
size_t decode_workspace_bytes(int rows, int sms);        // what a call of that many rows uses
size_t decode_workspace_for_up_to(int rows, int sms);   // the most that any call of up to that many uses
size_t prefill_workspace_bytes(int sms);
cudaError_t take_append_error(int *code);
cudaError_t take_decode_error(int *code);
cudaError_t take_prefill_error(int *code);

}  // namespace attn
}  // namespace gdn
