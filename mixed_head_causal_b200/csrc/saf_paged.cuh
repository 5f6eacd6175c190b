// Shared definitions of the serving kernels (paged key/value cache).
#pragma once

#include <limits.h>

#include <algorithm>

#include "saf_common.cuh"
#include "tc_util.cuh"

namespace saf {

// Kernel ids of the launch accounting, after those of saf_common.cuh.
constexpr int KID_ROPE_TABLE = 15, KID_KV_APPEND = 16, KID_PAGED_ATTN = 17, KID_PAGED_PREFIX = 18, KID_PAGED_TC = 19,
              KID_PAGED_PREFIX_TC = 20;

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

// ------------------------------------------------------------------ device side
// One row of an item.  A replaced row looks its scores up: a at local key j is
// a[a0 + j], r is r[r0 - j], for j < vis.
struct RowInfo {
    long long a0, r0;
    int vis;        // keys it sees
    int out, part;  // its row of the output (-1: it has no token), and of the prefix's parts
    int replaced;   // its head + 1, or 0
};

// Division by a launch constant: n / d = (umulhi(n, m) + n) >> s for 0 <= n < 2^31, with 2^(s-1) < d <= 2^s and
// m = floor(2^32 (2^s - d) / d) + 1 (the round-up method of Granlund and Montgomery).  A few cycles, where the
// general division's code, cold at the start of a launch, costs hundreds.
struct Divisor {
    uint32_t m, s;
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
};
inline Divisor divisor(int d) {
    Divisor x{0, 0};
    while ((1ll << x.s) < d) ++x.s;
    x.m = (uint32_t)(((1ull << 32) * ((1ull << x.s) - (uint64_t)d)) / (uint64_t)d + 1);
    return x;
}

// What the attention kernels need, by value.
struct PagedParams {
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;
    const float *a, *r;
    int pattern_len, prefix_len;
    HeadBits replaced;
    const int32_t *table, *seq_lens, *q_lens;
    int table_stride, num_pages, log_page, Hkv;
    int B, H, T, G, R, max_len;  // R = G T rows of one (b, g)
    int nseq, rows, nrb;         // key sequences, rows of one item list entry, row blocks
    Divisor by_T, by_BT, by_nrb;
    int keyed;                   // K/V heads with keys: the first of order[]
    uint8_t order[kMaxHeads];    // K/V heads, those with keys first
    uint8_t heads[kMaxHeads];    // query heads group by group, the ordinary ones of a group first
    unsigned int *err, *counters;
    float* slots;                // pieces: two per CTA
    // What the prefix came to (or null): [parts][Hkv * B * R][64] O, then [parts][Hkv * B * R] m, and the same of l.
    float* part;
    int parts;
    int splits;                  // tensor-core kernel: stretches of the keys
};

__device__ __forceinline__ void report(unsigned int* err, unsigned int code) {
    atomicOr(err, 1u);
    atomicCAS(err + 1, 0u, code);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];\n" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// exp(x - m) for finite or -inf x <= m (m = -inf: no weight yet).
__device__ __forceinline__ float weight(float x, float m) { return tc::ex2((x - (m == kNegInf ? 0.f : m)) * kLog2e); }

template <bool PREFIX>
__device__ __forceinline__ int key_len(const PagedParams& p, int b) {
    return PREFIX ? p.prefix_len : min(max(p.seq_lens[b], 0), p.max_len);
}
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b) {
    return p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
}
// Row rr of the item list entry (b, g), head by head (the ordinary heads of the
// group first): with PREFIX (head, sequence, token), else (head, token) of sequence b.  n, pos0: the
// sequence's new tokens and the position of the first (with PREFIX they are
// looked up per row).
template <bool PREFIX>
__device__ __forceinline__ RowInfo row_info(const PagedParams& p, int b, int g, int len, int n, int pos0, int rr) {
    RowInfo x;
    x.a0 = x.r0 = 0;
    x.vis = x.part = 0;
    x.out = -1;
    x.replaced = 0;
    if (rr >= p.rows) return x;
    const int u = (PREFIX ? p.by_BT : p.by_T).div(rr), h = p.heads[g * p.G + u];
    const int rem = rr - u * (PREFIX ? p.B * p.T : p.T);
    const int rb = PREFIX ? p.by_T.div(rem) : b, t = PREFIX ? rem - rb * p.T : rem;
    if (PREFIX) {
        n = new_tokens(p, rb);
        pos0 = p.prefix_len + key_len<false>(p, rb) - n;
    }
    if (t >= n) return x;
    const int key_base = PREFIX ? 0 : p.prefix_len;  // position of local key 0
    const long long ph = (long long)h * p.pattern_len;
    x.vis = max(0, min(len, pos0 + t - key_base + 1));
    x.a0 = ph + key_base;
    x.r0 = ph + pos0 + t - key_base;
    x.out = (rb * p.H + h) * p.T + t;
    x.part = ((g * p.G + u) * p.B + rb) * p.T + t;
    x.replaced = p.replaced.get(h) ? h + 1 : 0;
    return x;
}

// What a finished row is joined with: the parts of the prefix.  M: the largest
// maximum; weight(part's m, M) scales a part.
__device__ __forceinline__ size_t part_rows(const PagedParams& p) { return (size_t)p.Hkv * p.B * p.R; }
__device__ __forceinline__ const float* part_m(const PagedParams& p, int k, int row) {
    return p.part + part_rows(p) * kHeadDim * p.parts + (size_t)k * part_rows(p) + row;
}
__device__ __forceinline__ float* part_o(const PagedParams& p, int k, int row) {
    return p.part + ((size_t)k * part_rows(p) + row) * kHeadDim;
}
__device__ __forceinline__ void store_part_ml(const PagedParams& p, int k, int row, float m, float l) {
    float* pm = const_cast<float*>(part_m(p, k, row));
    pm[0] = m;
    pm[part_rows(p) * p.parts] = l;
}
// Four columns of a row (from c) joined with the prefix's parts: o, m and l are updated.
__device__ __forceinline__ void join_parts(const PagedParams& p, int row, int c, float4& o, float& m, float& l) {
    float mm = m;
    for (int k = 0; k < p.parts; ++k) mm = fmaxf(mm, __ldcg(part_m(p, k, row)));
    const float f = weight(m, mm);
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    l *= f;
#pragma unroll 4
    for (int k = 0; k < p.parts; ++k) {
        const float* pm = part_m(p, k, row);
        const float fk = weight(__ldcg(pm), mm);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(part_o(p, k, row) + c));
        o = make_float4(o.x + fk * v.x, o.y + fk * v.y, o.z + fk * v.z, o.w + fk * v.w);
        l += fk * __ldcg(pm + part_rows(p) * p.parts);
    }
    m = mm;
}
// A finished row (four columns from c) to the output.
__device__ __forceinline__ void store_row(const PagedParams& p, const RowInfo& x, int c, float4 o, float m, float l) {
    const bool some = !(l == 0.f);  // also a NaN
    const float s = some ? __fdividef(1.f, l) : 0.f;
    *reinterpret_cast<uint2*>(p.o + (size_t)x.out * kHeadDim + c) =
        make_uint2(tc::pack_bf16x2(o.x * s, o.y * s), tc::pack_bf16x2(o.z * s, o.w * s));
    if (c == 0) p.lse[x.out] = some ? m + __logf(l) : kNegInf;
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// The cache as (d, slot, head, page), boxes of one page's rows (max_rows at most).
inline bool make_tmap_pages(const saf_paged_kv& kv, bool keys, int max_rows, CUtensorMap* out) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t st[3] = {keys ? kv.k_stride_slot : kv.v_stride_slot, keys ? kv.k_stride_head : kv.v_stride_head,
                           keys ? kv.k_stride_page : kv.v_stride_page};
    cuuint64_t dims[4] = {64, (cuuint64_t)kv.page_size, (cuuint64_t)kv.H_kv, (cuuint64_t)std::max(1, kv.num_pages)};
    cuuint64_t strides[3] = {(cuuint64_t)st[0] * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[2] * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)std::min(max_rows, kv.page_size), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, keys ? kv.k : kv.v, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor-core kernel (saf_paged_tc.cu): items of up to 128 rows, the keys of each in p.splits stretches.  With
// prefix, the stretches become p.parts = p.splits parts; else they are joined, through `slots` and `counters` where
// there are several.
constexpr int kTcCtas = 592;  // the most CTAs that stretches make: two waves of two on each of 148 SMs
inline int tc_items(int nseq, int H_kv, int rows) { return nseq * H_kv * ((rows + 127) / 128); }
int tc_splits(int items, int max_keys);
cudaError_t launch_paged_tc(const saf_paged_kv& kv, PagedParams& p, bool prefix, bool overlap, cudaStream_t stream);

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len);
cudaError_t launch_rope_table(float* table, int max_pos, int rot_dim, double base, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
cudaError_t launch_paged_attn(const PagedCall& c, cudaStream_t stream);

}  // namespace saf
