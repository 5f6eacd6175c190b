// Shared definitions of the serving kernels (paged key/value cache).
#pragma once

#include "saf_common.cuh"
#include "tc_util.cuh"

namespace saf {

// Kernel ids of the launch accounting, after those of saf_common.cuh.
constexpr int KID_ROPE_TABLE = 15, KID_KV_APPEND = 16, KID_PAGED_ATTN = 17, KID_PAGED_PREFIX = 18;

// Head kinds by value: bit h set = head h is one.
struct HeadBits {
    uint32_t w[kMaxHeads / 32];
    __host__ __device__ bool get(int h) const { return (w[h >> 5] >> (h & 31)) & 1u; }
};

// What the append kernel needs, by value.
struct AppendParams {
    saf_paged_kv kv;
    const __nv_bfloat16 *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];  // strides (batch, head, token) in elements
    __nv_bfloat16 *q_out, *k_out;
    const float* rope;
    int rot_dim, interleaved, pos_offset;
    HeadBits replaced;   // per query head
    HeadBits keyless;    // per K/V head: all its query heads are replaced
    const int32_t *page_table, *seq_lens, *q_lens;
    int max_pages, B, H, T, max_len;
};

// A paged attention call (checked by the ABI layer).
struct PagedCall {
    saf_paged_kv kv;
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;
    const float *a, *r;
    int pattern_len;
    HeadBits replaced;   // per query head
    HeadBits keyless;    // per K/V head: all its query heads are replaced
    const int32_t* prefix_table;
    int prefix_len;
    const int32_t *page_table, *seq_lens, *q_lens;
    int max_pages, B, H, T, max_len;
    char* ws;
};

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len);
cudaError_t launch_rope_table(float* table, int max_pos, int rot_dim, double base, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_paged_attn(const PagedCall& c, cudaStream_t stream);

}  // namespace saf
