// Shared definitions of the serving kernels (paged key/value cache).
#pragma once

#include <limits.h>

#include <algorithm>

#include "saf_common.cuh"
#include "tc_util.cuh"

namespace saf {

// Kernel ids of the launch accounting, after those of saf_common.cuh.
constexpr int KID_ROPE_TABLE = 15, KID_KV_APPEND = 16, KID_PAGED_ATTN = 17, KID_PAGED_PREFIX = 18, KID_PAGED_TC = 19,
              KID_PAGED_PREFIX_TC = 20, KID_PAGED_JOIN = 21;

// Head kinds by value: bit h set = head h is one.
struct HeadBits {
    uint32_t w[kMaxHeads / 32];
    __host__ __device__ bool get(int h) const { return (w[h >> 5] >> (h & 31)) & 1u; }
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
    int units, log_page;       // groups of rows per token
    Divisor by_units, by_T;
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

// The item of several pieces whose first is this CTA's (pieces = 0: none).
struct __align__(16) SharedItem {
    int pieces, b, e, rb, len, n_rows, unused[2];
};

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
    int nseq;                    // key sequences (1 for the prefix)
    // The rows that share keys and an item list: entry e holds e_heads[e] of K/V head e_g[e]'s query heads, from
    // heads[e_g[e] * G + e_first[e]] on, hp[0] at most.  The keyed ones come first; the others' rows are all replaced:
    // hp[1] heads at most, each of a multiple of `pad` rows (those behind its tokens hold nothing).
    int entries, keyed, hp[2], pad, block_rows;
    uint8_t e_g[kMaxHeads], e_first[kMaxHeads];
    uint16_t e_heads[kMaxHeads];
    uint8_t heads[kMaxHeads];    // query heads group by group, the ordinary ones of a group first
    Divisor by_T, by_BT, by_BT_pad, by_block;
    unsigned int *err, *counters;
    long long wait_limit;        // cycles after which a wait gives up
    float* slots;                // pieces: two per CTA
    SharedItem* shared;          // per CTA, of the tensor-core kernel
    // What the prefix came to (or null): [part_rows][64] O, then m, then l, before the division; rows in the order of
    // heads[], sequence, token.
    float* part;
    int part_rows;
};

// Every wait on a barrier is bounded by PagedParams::wait_limit (about a second, see saf_selftest_serving_wait_limit);
// a role that gave up waits, by this bound, for what it has under way itself before the memory is let go.
constexpr long long kDrainLimit = 1ll << 31;

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
// Two bf16 as a pair of fp32.
__device__ __forceinline__ uint64_t pair_of(uint32_t w) {
    return tc::f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// What takes an O of rounded weights, whose sum is `rounded`, to the sum l of the weights themselves.
__device__ __forceinline__ float by_rounded(float l, float rounded) { return rounded > 0.f ? __fdividef(l, rounded) : 1.f; }
// exp(x - m) for finite or -inf x <= m (m = -inf: no weight yet).
__device__ __forceinline__ float weight(float x, float m) { return tc::ex2((x - (m == kNegInf ? 0.f : m)) * kLog2e); }

template <bool PREFIX>
__device__ __forceinline__ int key_len(const PagedParams& p, int b) {
    return PREFIX ? p.prefix_len : min(max(p.seq_lens[b], 0), p.max_len);
}
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b) {
    return p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
}
// Tokens of a head of a sequence's entries: with PREFIX those of the whole batch,
// else the sequence's new ones.
template <bool PREFIX>
__device__ __forceinline__ int head_rows(const PagedParams& p, int b) {
    return PREFIX ? p.B * p.T : new_tokens(p, b);
}
// n rows of a head with those that fill them up.
__host__ __device__ __forceinline__ int padded(int n, int pad) { return (n + pad - 1) & -pad; }
// Row rr of entry e of sequence b, head by head: with PREFIX (head, sequence,
// token), else (head, token).  len: keys; n: head_rows.
template <bool PREFIX>
__device__ __forceinline__ RowInfo row_info(const PagedParams& p, int b, int e, int len, int n, int rr) {
    RowInfo x;
    x.a0 = x.r0 = 0;
    x.vis = x.part = 0;
    x.out = -1;
    x.replaced = 0;
    const bool keyed = e < p.keyed;
    const int np = keyed ? n : padded(n, p.pad);
    if (rr >= p.e_heads[e] * np) return x;
    const int u = PREFIX ? (keyed ? p.by_BT : p.by_BT_pad).div(rr) : np == 1 ? rr : (int)((unsigned)rr / (unsigned)np);
    const int rem = rr - u * np;
    if (rem >= n) return x;
    const int rb = PREFIX ? p.by_T.div(rem) : b, t = PREFIX ? rem - rb * p.T : rem;
    const int hs = p.e_g[e] * p.G + p.e_first[e] + u, h = p.heads[hs];
    int pos = p.prefix_len + len - n + t;
    if (PREFIX) {
        const int n_new = new_tokens(p, rb);
        if (t >= n_new) return x;
        pos = p.prefix_len + key_len<false>(p, rb) - n_new + t;
    }
    const int key_base = PREFIX ? 0 : p.prefix_len;  // position of local key 0
    const long long ph = (long long)h * p.pattern_len;
    x.vis = max(0, min(len, pos - key_base + 1));
    x.a0 = ph + key_base;
    x.r0 = ph + pos - key_base;
    x.out = (rb * p.H + h) * p.T + t;
    x.part = (hs * p.B + rb) * p.T + t;
    x.replaced = p.replaced.get(h) ? h + 1 : 0;
    // (the index-checked build) its entries of a and r, the output's row and the part's
    [[maybe_unused]] const long long entries = (long long)p.H * p.pattern_len;
    if (!SAF_CHECKED_OK(p.err,
                        x.out >= 0 && x.out < p.B * p.H * p.T && x.part >= 0 && x.part < p.B * p.H * p.T &&
                            (!x.replaced || x.vis == 0 ||
                             (x.a0 >= 0 && x.a0 + x.vis <= entries && x.r0 < entries && x.r0 - x.vis + 1 >= 0)),
                        0x9401u)) {
        x.out = -1;
        x.vis = x.replaced = 0;
    }
    return x;
}

// Stretch boundaries of an axis (see AxisWalk): the first stretch that begins at
// unit x > 0 or later.
__device__ __forceinline__ int first_from(int per, int more, int x) {
    const int big = more * (per + 1);
    return x <= big ? (int)((unsigned)(x + per) / (unsigned)(per + 1))
                    : more + (int)((unsigned)(x - big + per - 1) / (unsigned)per);
}
// The CTAs that share the item that begins at unit `start`: how many, and the
// first (where there are several).
__device__ __forceinline__ int pieces_of(int per, int more, int item_units, int snap, int start, int tile_units, int& c_first) {
    // the stretches that begin strictly inside the item, by more than a snap
    const int in_lo = start + item_units + snap + 1, in_hi = start + item_units + tile_units - snap;
    const int c1 = in_lo < in_hi ? first_from(per, more, in_lo) : 0, c2 = in_lo < in_hi ? first_from(per, more, in_hi) : 0;
    c_first = c1 - 1;
    return c2 - c1 + 1;
}
// Four columns of a row (from c) joined with what the prefix came to: o, m and l are updated.
__device__ __forceinline__ void join_part(const PagedParams& p, int row, int c, float4& o, float& m, float& l) {
    const float* ml = p.part + (size_t)p.part_rows * kHeadDim + row;
    const float4 o2 = __ldcg(reinterpret_cast<const float4*>(p.part + (size_t)row * kHeadDim + c));
    const float m2 = __ldcg(ml), l2 = __ldcg(ml + p.part_rows);
    const float mm = fmaxf(m, m2), f = weight(m, mm), f2 = weight(m2, mm);
    o = make_float4(o.x * f + o2.x * f2, o.y * f + o2.y * f2, o.z * f + o2.z * f2, o.w * f + o2.w * f2);
    l = l * f + l2 * f2;
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
// A row that has all its keys (four columns from c): with PREFIX the part that the
// batch's own keys are joined to, else the output.
template <bool PREFIX>
__device__ __forceinline__ void finish_row(const PagedParams& p, const RowInfo& x, int c, float4 o, float m, float l) {
    if (x.out < 0) return;
    if (PREFIX) {
        *reinterpret_cast<float4*>(p.part + (size_t)x.part * kHeadDim + c) = o;
        if (c == 0) {
            p.part[(size_t)p.part_rows * kHeadDim + x.part] = m;
            p.part[(size_t)p.part_rows * (kHeadDim + 1) + x.part] = l;
        }
    } else {
        if (p.part) join_part(p, x.part, c, o, m, l);
        store_row(p, x, c, o, m, l);
    }
}

// ---------------------------------------------------------------- the axis of tiles
// Items (sequence b, entry, row block) one after the other, each kItem units that
// stand for no tile (its own cost) and kUnit or kUnitKeyless per tile; every CTA
// takes an equal stretch, moved to an item's end where it would end within kSnap
// units of one.  A: these constants, and the tile sizes (keys) of entries with and
// without keys.
struct Stretch {
    int b, e, rb, len, n_rows, n;  // item; its sequence's keys and head_rows; its tiles (one without keys still takes one,
                                   // empty, tile: its rows are written)
    bool keyed;
    int t0, t1;                    // this CTA's tiles of it
    int pieces, c_first;           // CTAs that share it, and the first of them
};
template <class A, bool PREFIX>
struct AxisWalk {
    const PagedParams& p;
    int total, ctas, per, more;    // units; stretch c begins at c * per + min(c, more)
    int u, end, b, base, len, nr;  // next unit, end of the stretch, current sequence: first unit, keys, head_rows
    __device__ __forceinline__ static int tiles_of(int len, bool keyed) {
        const int tk = keyed ? A::kTile : A::kTileKeyless;
        return max(1, (len + tk - 1) / tk);
    }
    __device__ __forceinline__ static int item_units(int tiles, bool keyed) {
        return tiles * (keyed ? A::kUnit : A::kUnitKeyless) + A::kItem;
    }
    __device__ __forceinline__ int blocks_of(int rows, bool keyed) const {
        return p.by_block.div((keyed ? p.hp[0] * rows : p.hp[1] * padded(rows, p.pad)) + p.block_rows - 1);
    }
    __device__ __forceinline__ int seq_units(int n, int rows) const {
        return p.keyed * blocks_of(rows, true) * item_units(tiles_of(n, true), true) +
               (p.entries - p.keyed) * blocks_of(rows, false) * item_units(tiles_of(n, false), false);
    }
    // The item that unit u of a sequence is in; returns its first unit.
    __device__ __forceinline__ int item_at(int base_u, int n_keys, int rows, int unit, Stretch& x) const {
        int nrb = blocks_of(rows, true), off = unit - base_u;
        x.n = tiles_of(n_keys, true);
        const int keyed_units = p.keyed * nrb * item_units(x.n, true);
        x.keyed = off < keyed_units;
        int first = 0;
        if (!x.keyed) {
            x.n = tiles_of(n_keys, false);
            nrb = blocks_of(rows, false);
            off -= keyed_units;
            first = p.keyed;
        }
        const int units = item_units(x.n, x.keyed), block = (int)((unsigned)off / (unsigned)units);
        x.e = nrb == 1 ? block : (int)((unsigned)block / (unsigned)nrb);
        x.rb = block - x.e * nrb;
        x.e += first;
        return unit - (off - block * units);
    }
    // By a whole warp: units are summed a run of sequences per lane.
    __device__ __forceinline__ AxisWalk(const PagedParams& params, int cta, int grid) : p(params) {
        const int lane = threadIdx.x & 31;
        const int chunk = (p.nseq + 31) >> 5, b_lo = min(lane * chunk, p.nseq), b_hi = min(b_lo + chunk, p.nseq);
        int mine = 0;
#pragma unroll 4
        for (int k = b_lo; k < b_hi; ++k) mine += seq_units(key_len<PREFIX>(p, k), head_rows<PREFIX>(p, k));
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += v;
        }
        total = __shfl_sync(~0u, incl, 31);
        const int before = incl - mine;
        ctas = max(1, min(grid, total / A::kMinUnits));
        per = (int)((unsigned)total / (unsigned)ctas);
        more = total - per * ctas;
        const int lo = cta < ctas ? cta * per + min(cta, more) : total, hi = lo + per + (cta < more ? 1 : 0);
        // The sequence of a unit below `total`, and its first unit.
        auto find = [&](int unit, int& seq, int& first) {
            const int src = __ffs(__ballot_sync(~0u, unit >= before && unit < before + mine)) - 1;
            int at = before, k = b_lo;
            if (lane == src)
                for (;; ++k) {
                    const int n = seq_units(key_len<PREFIX>(p, k), head_rows<PREFIX>(p, k));
                    if (unit < at + n) break;
                    at += n;
                }
            seq = __shfl_sync(~0u, k, src);
            first = __shfl_sync(~0u, at, src);
        };
        auto snapped = [&](int unit, int seq, int first) {
            Stretch x;
            const int start = item_at(first, key_len<PREFIX>(p, seq), head_rows<PREFIX>(p, seq), unit, x);
            const int stop = start + item_units(x.n, x.keyed);
            return unit - start <= A::kItem + A::kSnap ? start : stop - unit <= A::kSnap ? stop : unit;
        };
        b = base = 0;
        u = end = total;
        if (lo < total) {
            find(lo, b, base);
            u = snapped(lo, b, base);
            if (hi < total) {
                int b_end, base_end;
                find(hi, b_end, base_end);
                end = snapped(hi, b_end, base_end);
            }
        }
        len = key_len<PREFIX>(p, b);
        nr = head_rows<PREFIX>(p, b);
    }
    // The next item of the stretch; false: none left.
    __device__ __forceinline__ bool next(Stretch& x) {
        if (u >= end) return false;
        for (int n; u >= base + (n = seq_units(len, nr));) {
            base += n;
            ++b;
            len = key_len<PREFIX>(p, b);
            nr = head_rows<PREFIX>(p, b);
        }
        const int start = item_at(base, len, nr, u, x), w = x.keyed ? A::kUnit : A::kUnitKeyless;
        x.b = b;
        x.len = len;
        x.n_rows = nr;
        // a tile belongs to the stretch that holds its first unit
        x.t0 = max(0, (u - start - A::kItem + w - 1) / w);
        x.t1 = min(x.n, (end - start - A::kItem + w - 1) / w);
        x.pieces = pieces_of(per, more, A::kItem, A::kSnap, start, x.n * w, x.c_first);
        u = start + A::kItem + x.n * w;  // (or past the stretch)
        if (u > end) u = end;
        // (the index-checked build) the item, its tiles within the keys that the table holds, its pieces' slots
        return SAF_CHECKED_OK(p.err,
                              b >= 0 && b < p.nseq && x.e >= 0 && x.e < p.entries && x.rb >= 0 && x.t0 >= 0 && x.t0 <= x.t1 &&
                                  x.t1 <= x.n && len <= (PREFIX ? p.prefix_len : p.max_len) && x.pieces >= 1 &&
                                  (x.pieces == 1 || (x.c_first >= 0 && x.c_first + x.pieces <= ctas)),
                              0x9402u);
    }
};

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

// The rows of an entry and the units of the longest axis must fit 31 bits, with room for a stretch's length and padding.
template <class A>
bool axis_fits(const PagedParams& p, bool prefix) {
    const int64_t n = prefix ? (int64_t)p.B * p.T : p.T, keys = prefix ? p.prefix_len : p.max_len;
    double units = 0;
    for (int keyless = 0; keyless < 2; ++keyless) {
        const int64_t rows = p.hp[keyless] * (keyless ? (n + p.pad - 1) / p.pad * p.pad : n), tile = keyless ? A::kTileKeyless : A::kTile;
        if (rows > INT_MAX - 256) return false;
        const double item = A::kItem + (double)std::max<int64_t>(1, (keys + tile - 1) / tile) * (keyless ? A::kUnitKeyless : A::kUnit);
        units += item * (double)((rows + p.block_rows - 1) / p.block_rows) * (keyless ? p.entries - p.keyed : p.keyed);
    }
    return units * p.nseq <= 2147483648.0 - (1 << 24);
}
// Entries of up to hp heads of one K/V head each, hp_replaced where none of them is ordinary; apart: of one kind each.
inline void make_entries(PagedParams& p, int hp, int hp_replaced, bool apart) {
    p.hp[0] = hp;
    p.hp[1] = hp_replaced;
    p.entries = 0;
    for (int want = 0; want < 2; ++want) {  // those that need keys, then those of replaced heads alone
        for (int g = 0; g < p.Hkv; ++g) {
            int ordinary = 0;
            while (ordinary < p.G && !p.replaced.get(p.heads[g * p.G + ordinary])) ++ordinary;
            const int split = apart || ordinary == 0 ? ordinary : p.G;  // heads of the keyed entries
            const int from = want ? split : 0, to = want ? p.G : split;
            const int most = p.hp[want];
            for (int u = from; u < to; u += most, ++p.entries) {
                p.e_g[p.entries] = (uint8_t)g;
                p.e_first[p.entries] = (uint8_t)u;
                p.e_heads[p.entries] = (uint16_t)std::min(most, to - u);
            }
        }
        if (want == 0) p.keyed = p.entries;
    }
}
constexpr long long kServingWaitLimit = 1ll << 31;  // about a second
void set_serving_wait_limit(long long cycles);      // 0: that

// CTAs of either kernel, two per SM; bounds the workspace (pieces: two per CTA).
constexpr int kMaxGrid = 320;
inline int paged_grid() { return std::min(kMaxGrid, 2 * sm_count()); }
// The tensor-core kernel (saf_paged_tc.cu): items of up to 128 rows.
cudaError_t launch_paged_tc(const saf_paged_kv& kv, PagedParams& p, bool prefix, cudaStream_t stream);

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len);
cudaError_t launch_rope_table(float* table, int max_pos, int rot_dim, double base, cudaStream_t stream);
cudaError_t launch_kv_append(AppendParams& p, cudaStream_t stream);
cudaError_t launch_paged_attn(const PagedCall& c, cudaStream_t stream);

}  // namespace saf
