// Attention of a few new tokens per sequence over the paged key/value cache.
//
// Work is a list of items (sequence b, K/V head g, row block): the rows of one
// item are the G = H / H_kv query heads of the group times the T new tokens,
// and share every key.  Keys come in tiles of 64.  The tiles of all items form
// one axis, weighted by the bytes they read (2 with K and V, 1 for a K/V head
// whose query heads are all replaced, which has no keys), and each CTA of a
// grid that fills the GPU takes an equal stretch of it, wherever that begins
// and ends: lengths are read on the device, so a captured call follows them.
// An item that one CTA holds whole is written at once; the others leave
// (m, l, O) pieces in the workspace, and the CTA that finishes an item's last
// piece joins them in key order (the result does not depend on which CTA that is).
//
// A CTA is one producer warp and four consumer warps.  The producer looks up
// the pages of a tile and fetches them by TMA (128-byte swizzle) into a ring;
// a tile of 64 keys is 64 / page_size boxes.  The consumers split the tile's
// keys (and, above 16 rows, the rows): S = Q K^T and O += P V as warp-level
// m16n8k16 MMAs with a running maximum and sum per row and warp,
//   ordinary row   s = q . k / 8
//   replaced row   s = a[j] + r[i - j]      (Eq. (3): its softmax is the pattern)
// joined over the warps at the end of an item.
//
// One new token makes this a stream of K and V at a few flops per byte: HBM
// bounds it, so the warp-level MMAs (a tile of 16 rows costs about 130 of the
// 700 cycles in which HBM delivers it to one SM) are enough, and the kernel is
// built for bytes in flight.
#include <limits.h>

#include <algorithm>

#include "mma_util.cuh"
#include "saf_paged.cuh"

namespace saf {
namespace {

using namespace tc;
using mma::load_b_frag_kn;
using mma::load_b_frag_nk;
using mma::mma_bf16;

constexpr int TK = 64;               // keys per tile
constexpr int NS = 3;                // ring stages
constexpr int NCONS = 128;           // consumer threads (four warps), then the producer warp
constexpr int CTAS_PER_SM = 3;
constexpr int kMaxGrid = 1024;       // bounds the workspace
constexpr uint32_t HALF = TK * 128;  // bytes of a tile's K or V
constexpr uint32_t STAGE = 2 * HALF;
constexpr int RED_PITCH = 72;        // floats per row of a warp's O: eight-byte stores of a quad row hit distinct banks
constexpr uint32_t SM_RED = NS * STAGE;
constexpr uint32_t SM_ML = SM_RED + 4 * 16 * RED_PITCH * 4;  // [4 warps][16 rows] m, then l
constexpr uint32_t SM_BAR = SM_ML + 2 * 4 * 16 * 4;
constexpr uint32_t SM_INFO = SM_BAR + 16 * NS;  // [NS] pages of a stage that are none; the scan's sums and results
constexpr uint32_t SM_TOTAL = SM_INFO + 4 * NS + 4 * 8;
constexpr uint32_t SM_ALLOC = SM_TOTAL + 1024;  // the ring starts on a 1024-byte boundary (swizzle atoms)
constexpr long long kWaitLimit = 1ll << 31;

struct SplitParams {
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;
    const float *a, *r;
    int pattern_len, prefix_len;
    HeadBits replaced, keyless;
    const int32_t *table, *seq_lens, *q_lens;
    int table_stride, num_pages, log_page, Hkv;
    int B, H, T, G, R, max_len;  // R = G T rows of one (b, g)
    int nseq, rows, nrb;         // key sequences, rows of one item list entry, row blocks
    int wsum;                    // sum of the K/V heads' weights
    uint8_t g_of_w[2 * kMaxHeads];  // K/V head of each weight unit
    unsigned int *err, *counters;
    float* slots;                // pieces: two per CTA
    float* part;                 // [Hkv * B * R][64] O, then [Hkv * B * R] m, then l, of the prefix (or null)
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
__device__ __forceinline__ float weight(float x, float m) { return ex2((x - (m == kNegInf ? 0.f : m)) * kLog2e); }

// A stretch [lo, hi) of the weighted tile axis, walked item by item.  The axis
// runs over sequences, their K/V heads, row blocks and tiles; a tile belongs to
// the CTA whose stretch holds its first unit.
struct Piece {
    int b, g, rb, t0, t1, n, len, w;  // tiles [t0, t1) of the item's n; len keys
    long long start;                  // unit of the item's tile 0
};
struct Walk {
    long long u, hi, base;  // next unit, end, first unit of sequence b
    int b, len, tiles;
};

template <bool PREFIX>
__device__ __forceinline__ int key_len(const SplitParams& p, int b) {
    return PREFIX ? p.prefix_len : min(max(p.seq_lens[b], 0), p.max_len);
}
// An item without keys still takes one (empty) tile: its rows are written.
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + TK - 1) / TK); }

template <bool PREFIX>
__device__ __forceinline__ bool next_piece(const SplitParams& p, Walk& w, Piece& x) {
    while (w.u < w.hi && w.b < p.nseq) {
        const int block = w.tiles * p.nrb;  // tiles of one weight unit
        const int off = (int)(w.u - w.base);
        if (off >= block * p.wsum) {
            w.base += (long long)block * p.wsum;
            if (++w.b < p.nseq) {
                w.len = key_len<PREFIX>(p, w.b);
                w.tiles = tiles_of(w.len);
            }
            continue;
        }
        int gw = off / block;
        x.g = p.g_of_w[gw];
        if (gw > 0 && p.g_of_w[gw - 1] == x.g) --gw;
        x.w = p.keyless.get(x.g) ? 1 : 2;
        const int in_g = off - gw * block, item = w.tiles * x.w;
        x.rb = in_g / item;
        const int in_item = in_g - x.rb * item;
        x.start = w.u - in_item;
        x.t0 = (in_item + x.w - 1) / x.w;
        x.t1 = (int)min((long long)w.tiles, (w.hi - x.start + x.w - 1) / x.w);
        x.b = w.b;
        x.n = w.tiles;
        x.len = w.len;
        w.u = x.start + item;
        if (x.t0 < x.t1) return true;
    }
    return false;
}

// One row of an item: rr counts the rows of the item list entry.
struct Row {
    int b, h, t;  // sequence, query head, new token
    int pos;      // position of the row, the prefix included
    bool valid;
};
template <bool PREFIX>
__device__ __forceinline__ Row row_of(const SplitParams& p, int b, int g, int rr) {
    Row x;
    x.b = PREFIX ? rr / p.R : b;
    const int rem = PREFIX ? rr - x.b * p.R : rr;
    x.valid = rr < p.rows;
    if (!x.valid) {
        x.b = x.h = x.t = x.pos = 0;
        return x;
    }
    const int u = rem / p.T;
    x.h = g * p.G + u;
    x.t = rem - u * p.T;
    const int n = p.q_lens ? min(max(p.q_lens[x.b], 0), p.T) : p.T;
    x.valid = x.t < n;
    x.pos = p.prefix_len + key_len<false>(p, x.b) - n + x.t;
    return x;
}

// A finished row (four columns from c): with PREFIX the part that the batch's
// own keys are joined to, else the output, after joining the prefix's part.
template <bool PREFIX>
__device__ __forceinline__ void finish_row(const SplitParams& p, int b, int g, int rr, int c, float4 o, float m, float l) {
    const Row x = row_of<PREFIX>(p, b, g, rr);
    if (!x.valid) return;
    const size_t nrow = (size_t)p.Hkv * p.B * p.R;
    const size_t pr = ((size_t)g * p.B + x.b) * p.R + (x.h - g * p.G) * p.T + x.t;
    if (PREFIX) {
        *reinterpret_cast<float4*>(p.part + pr * kHeadDim + c) = o;
        if (c == 0) {
            p.part[nrow * kHeadDim + pr] = m;
            p.part[nrow * (kHeadDim + 1) + pr] = l;
        }
        return;
    }
    if (p.part) {
        const float4 o2 = __ldcg(reinterpret_cast<const float4*>(p.part + pr * kHeadDim + c));
        const float m2 = __ldcg(p.part + nrow * kHeadDim + pr), l2 = __ldcg(p.part + nrow * (kHeadDim + 1) + pr);
        const float mm = fmaxf(m, m2), f = weight(m, mm), f2 = weight(m2, mm);
        o = make_float4(o.x * f + o2.x * f2, o.y * f + o2.y * f2, o.z * f + o2.z * f2, o.w * f + o2.w * f2);
        l = l * f + l2 * f2;
        m = mm;
    }
    const size_t row = ((size_t)x.b * p.H + x.h) * p.T + x.t;
    const bool some = !(l == 0.f);  // also a NaN
    const float s = some ? 1.f / l : 0.f;
    *reinterpret_cast<uint2*>(p.o + row * kHeadDim + c) = make_uint2(pack_bf16x2(o.x * s, o.y * s), pack_bf16x2(o.z * s, o.w * s));
    if (c == 0) p.lse[row] = some ? m + logf(l) : kNegInf;
}

// WR warps split the rows (16 each), WK = 4 / WR the keys of a tile.
template <int WR, bool PREFIX>
__global__ void __launch_bounds__(NCONS + 32, CTAS_PER_SM)
paged_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ SplitParams p) {
    constexpr int WK = 4 / WR, KW = TK / WK, NT = KW / 8, RT = 16 * WR;
    constexpr int SLOT = RT * (kHeadDim + 2);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bar_full = sbase + SM_BAR, bar_empty = bar_full + 8 * NS;
    uint32_t* meta = reinterpret_cast<uint32_t*>(smem + SM_INFO);
    int* scan_sums = reinterpret_cast<int*>(smem + SM_INFO) + NS;  // [5]
    int* first = scan_sums + 5;  // the stretch's first sequence, and the tiles before it
    int* last_flag = first + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 4);
        }
        fence_mbar_init();
    }
    // ---- this CTA's stretch: each thread sums the tiles of a run of sequences
    constexpr int NTH = NCONS + 32;
    const int chunk = (p.nseq + NTH - 1) / NTH, b_lo = min(tid * chunk, p.nseq), b_hi = min(b_lo + chunk, p.nseq);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(key_len<PREFIX>(p, b));
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan_sums[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int k = 0; k < NTH / 32; ++k) {
        if (k < warp) before += scan_sums[k];
        total += scan_sums[k];
    }
    const long long per_tile = (long long)p.nrb * p.wsum;
    const long long units = total * per_tile;
    // at least two units per CTA: then every stretch inside an item holds a tile
    const long long ctas = max(1ll, min((long long)gridDim.x, units / 2));
    if (blockIdx.x >= ctas) return;
    const long long lo = blockIdx.x * units / ctas, hi = (blockIdx.x + 1) * units / ctas;
    {
        long long at = before + incl - mine;  // tiles before this thread's run
        if (lo >= at * per_tile && lo < (at + mine) * per_tile) {
            int b = b_lo;
            for (; b < b_hi; ++b) {
                const int t = tiles_of(key_len<PREFIX>(p, b));
                if (lo < (at + t) * per_tile) break;
                at += t;
            }
            first[0] = b;
            first[1] = (int)at;
        }
    }
    __syncthreads();
    if (PREFIX) griddep_launch_dependents();  // the batch's own keys may start
    Walk wk;
    wk.u = lo;
    wk.hi = hi;
    wk.b = first[0];
    wk.base = first[1] * per_tile;
    wk.len = key_len<PREFIX>(p, wk.b);
    wk.tiles = tiles_of(wk.len);
    auto cta_of = [&](long long u) { return (int)(((u + 1) * ctas - 1) / units); };
    Piece x;

    if (warp == NCONS / 32) {
        // ------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        const int lp = p.log_page;
        const int boxes = max(1, TK >> lp);
        const uint32_t box_bytes = (uint32_t)min(TK, 1 << lp) * 128;
        int it = 0;
        bool ok = true;
        while (ok && next_piece<PREFIX>(p, wk, x)) {
            const bool keys = x.w == 2;
            const int32_t* table = p.table + (size_t)x.b * p.table_stride;
            const int npages = (x.len + (1 << lp) - 1) >> lp;
            int ids = -1, ids0 = -64;  // page ids [ids0, ids0 + 32), one per lane
            for (int t = x.t0; t < x.t1; ++t, ++it) {
                const int s = it % NS, pg0 = (t * TK) >> lp;
                if (pg0 >= ids0 + 32 || pg0 < ids0) {
                    ids0 = pg0;
                    ids = pg0 + lane < npages ? __ldg(table + pg0 + lane) : -1;
                }
                const int page = __shfl_sync(~0u, ids, (pg0 - ids0 + lane) & 31);
                const bool need = lane < boxes && pg0 + lane < npages;
                const bool good = need && page >= 0 && page < p.num_pages;
                const uint32_t bad = __ballot_sync(~0u, need && !good);
                const int loads = __popc(__ballot_sync(~0u, good));
                ok = mbar_wait_warp(bar_empty + 8 * s, ((it / NS) & 1) ^ 1, kWaitLimit);
                if (!ok) {
                    if (lane == 0) report(p.err, 0x401);
                    break;
                }
                if (lane == 0) {
                    meta[s] = bad;
                    mbar_expect_tx(bar_full + 8 * s, loads * box_bytes * (keys ? 2 : 1));
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = sbase + s * STAGE + lane * box_bytes;
                    const int y = (t * TK) & ((1 << lp) - 1);
                    if (keys) tma_load_4d(dst, &tmK, bar_full + 8 * s, 0, y, x.g, page);
                    tma_load_4d(dst + HALF, &tmV, bar_full + 8 * s, 0, y, x.g, page);
                }
            }
        }
        return;
    }

    // ---------------------------------------------------- consumers
    const int wr = warp / WK, wkey = warp % WK;
    float* red = reinterpret_cast<float*>(smem + SM_RED);
    float* red_m = reinterpret_cast<float*>(smem + SM_ML);
    float* red_l = red_m + 4 * 16;
    const int key_base = PREFIX ? 0 : p.prefix_len;  // position of local key 0
    int it = 0;
    bool ok = true, waited = false;
    while (next_piece<PREFIX>(p, wk, x)) {
        // this thread's two rows
        uint32_t qf[4][4];
        int vis[2];          // keys the row sees
        bool rep[2];
        const float *pa[2], *pr[2];  // a at local key j: pa[j]; r: pr[-j]
        int vmin = INT_MAX;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const Row row = row_of<PREFIX>(p, x.b, x.g, x.rb * RT + wr * 16 + (lane >> 2) + 8 * u);
            rep[u] = row.valid && p.replaced.get(row.h);
            vis[u] = row.valid ? max(0, min(x.len, row.pos - key_base + 1)) : 0;
            if (row.valid) vmin = min(vmin, vis[u]);
            const size_t ph = (size_t)row.h * p.pattern_len;
            pa[u] = p.a + ph + key_base;
            pr[u] = p.r + ph + (row.pos - key_base);
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                p.q + (((size_t)row.b * p.H + row.h) * p.T + row.t) * kHeadDim + (lane & 3) * 2);
            const bool read = row.valid && !rep[u];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                qf[k][u] = read ? __ldg(src + 8 * k) : 0u;
                qf[k][u + 2] = read ? __ldg(src + 8 * k + 4) : 0u;
            }
        }
        vmin = __reduce_min_sync(~0u, vmin);
        const bool any_rep = __any_sync(~0u, rep[0] || rep[1]);
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
        for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = 0.f;

        for (int t = x.t0; t < x.t1; ++t, ++it) {
            const int s = it % NS;
            const int j0 = t * TK + wkey * KW + (lane & 3) * 2;  // this thread's keys: j0 + 8 nt + {0, 1}
            float sc[NT][4];
            if (any_rep) {  // read while the tile is on its way
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = e >> 1, j = j0 + 8 * nt + (e & 1);
                        sc[nt][e] = rep[u] && j < vis[u] ? __ldg(pa[u] + j) + __ldg(pr[u] - j) : 0.f;
                    }
            }
            if (ok) {
                ok = mbar_wait_warp(bar_full + 8 * s, (it / NS) & 1, kWaitLimit);
                if (!ok && lane == 0) report(p.err, 0x402);
            }
            const uint32_t bad = meta[s];
            const uint32_t sk = sbase + s * STAGE, sv = sk + HALF;
            if (x.w == 2) {
                float dot[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) dot[nt][e] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; nt += 2)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b[4];
                        load_b_frag_nk(b, sk, wkey * KW + nt * 8, k * 16, lane);
                        mma_bf16(dot[nt], qf[k], b[0], b[1]);
                        mma_bf16(dot[nt + 1], qf[k], b[2], b[3]);
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!any_rep || !rep[e >> 1]) sc[nt][e] = dot[nt][e] * 0.125f;
            }
            // whole: every row of the warp sees every key of the tile
            const bool whole = t * TK + TK <= vmin && bad == 0;
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + 8 * nt + (e & 1);
                        if (j >= vis[e >> 1] || ((bad >> ((j & (TK - 1)) >> p.log_page)) & 1u)) sc[nt][e] = kNegInf;
                    }
            }
            float f[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float mx = m[u];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mx = max3(mx, sc[nt][2 * u], sc[nt][2 * u + 1]);
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                f[u] = mx > m[u] ? weight(m[u], mx) : 1.f;
                m[u] = mx;
                l[u] *= f[u];
                const float base = mx == kNegInf ? 0.f : mx;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sc[nt][2 * u] = ex2((sc[nt][2 * u] - base) * kLog2e);
                    sc[nt][2 * u + 1] = ex2((sc[nt][2 * u + 1] - base) * kLog2e);
                    l[u] += sc[nt][2 * u] + sc[nt][2 * u + 1];
                }
            }
            if (__any_sync(~0u, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    o[d][0] *= f[0];
                    o[d][1] *= f[0];
                    o[d][2] *= f[1];
                    o[d][3] *= f[1];
                }
            }
            // O += P V, P as a hi + lo bf16 pair: the tensor pipe has the room, and the
            // weights then carry 16 bits
#pragma unroll
            for (int kk = 0; kk < NT; kk += 2) {
                uint32_t ph[4], pl[4];
                mma::pack_bf16_split(sc[kk][0], sc[kk][1], ph[0], pl[0]);
                mma::pack_bf16_split(sc[kk][2], sc[kk][3], ph[1], pl[1]);
                mma::pack_bf16_split(sc[kk + 1][0], sc[kk + 1][1], ph[2], pl[2]);
                mma::pack_bf16_split(sc[kk + 1][2], sc[kk + 1][3], ph[3], pl[3]);
                uint32_t keep[2] = {~0u, ~0u};
                if (!whole) {  // a slot without a token may hold a NaN, and 0 times that is one
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = j0 + 8 * (kk + u);
                        const bool dead = (bad >> ((j & (TK - 1)) >> p.log_page)) & 1u;
                        keep[u] = dead ? 0u : (j < x.len ? 0xffffu : 0u) | (j + 1 < x.len ? 0xffff0000u : 0u);
                    }
                }
#pragma unroll
                for (int d = 0; d < 8; d += 2) {
                    uint32_t b[4];
                    load_b_frag_kn(b, sv, d * 8, wkey * KW + kk * 8, lane);
                    if (!whole) {
                        b[0] &= keep[0];
                        b[1] &= keep[1];
                        b[2] &= keep[0];
                        b[3] &= keep[1];
                    }
                    mma_bf16(o[d], ph, b[0], b[1]);
                    mma_bf16(o[d + 1], ph, b[2], b[3]);
                    mma_bf16(o[d], pl, b[0], b[1]);
                    mma_bf16(o[d + 1], pl, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
        }

        // ---- the warps' parts to shared memory, joined over the keys
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(~0u, l[u], 1);
            l[u] += __shfl_xor_sync(~0u, l[u], 2);
            const int row = (lane >> 2) + 8 * u;
            if ((lane & 3) == 0) {
                red_m[warp * 16 + row] = m[u];
                red_l[warp * 16 + row] = l[u];
            }
#pragma unroll
            for (int d = 0; d < 8; ++d)
                *reinterpret_cast<float2*>(red + (warp * 16 + row) * RED_PITCH + d * 8 + (lane & 3) * 2) =
                    make_float2(o[d][2 * u], o[d][2 * u + 1]);
        }
        named_sync(1, NCONS);
        const int c_first = cta_of(x.start), pieces = cta_of(x.start + (long long)(x.n - 1) * x.w) - c_first + 1;
        const int rows = min(RT, p.rows - x.rb * RT);
        const int c = (tid & 15) * 4;
        if (!PREFIX && p.part && !waited) {
            griddep_wait();
            waited = true;
        }
        float* slot = p.slots + ((size_t)blockIdx.x * 2 + (x.t0 == 0)) * SLOT;
        for (int row = tid >> 4; row < rows; row += NCONS / 16) {
            const int w0 = (row >> 4) * WK, rl = row & 15;
            float mm = kNegInf;
#pragma unroll
            for (int k = 0; k < WK; ++k) mm = fmaxf(mm, red_m[(w0 + k) * 16 + rl]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll
            for (int k = 0; k < WK; ++k) {
                const float f = weight(red_m[(w0 + k) * 16 + rl], mm);
                const float4 v = *reinterpret_cast<const float4*>(red + ((w0 + k) * 16 + rl) * RED_PITCH + c);
                acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
                ll += f * red_l[(w0 + k) * 16 + rl];
            }
            if (pieces == 1) {
                finish_row<PREFIX>(p, x.b, x.g, x.rb * RT + row, c, acc, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4*>(slot + row * kHeadDim + c), acc);
                if (c == 0) {
                    __stcg(slot + RT * kHeadDim + row, mm);
                    __stcg(slot + RT * (kHeadDim + 1) + row, ll);
                }
            }
        }
        if (pieces > 1) {
            __threadfence();
            named_sync(1, NCONS);
            if (tid == 0) *last_flag = atomicAdd(p.counters + c_first, 1u) == (unsigned)pieces - 1;
            named_sync(1, NCONS);
            if (*last_flag) {
                __threadfence();
                auto slot_of = [&](int k) { return p.slots + ((size_t)(c_first + k) * 2 + (k == 0)) * SLOT; };
                for (int row = tid >> 4; row < rows; row += NCONS / 16) {
                    float mm = kNegInf;
                    for (int k = tid & 15; k < pieces; k += 16) mm = fmaxf(mm, __ldcg(slot_of(k) + RT * kHeadDim + row));
                    // the sixteen threads of a row are a half-warp that runs this loop together
                    const uint32_t half = 0xffffu << (lane & 16);
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(half, mm, d));
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float ll = 0.f;
#pragma unroll 4
                    for (int k = 0; k < pieces; ++k) {
                        const float* sl = slot_of(k);
                        const float f = weight(__ldcg(sl + RT * kHeadDim + row), mm);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(sl + row * kHeadDim + c));
                        acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
                        ll += f * __ldcg(sl + RT * (kHeadDim + 1) + row);
                    }
                    finish_row<PREFIX>(p, x.b, x.g, x.rb * RT + row, c, acc, mm, ll);
                }
                if (tid == 0) atomicExch(p.counters + c_first, 0u);
            }
        }
        named_sync(1, NCONS);  // the shared parts have been read
    }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
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

// The cache as (d, slot, head, page), boxes of one page's rows (64 at most).
bool make_tmap_pages(const saf_paged_kv& kv, bool keys, CUtensorMap* out) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t st[3] = {keys ? kv.k_stride_slot : kv.v_stride_slot, keys ? kv.k_stride_head : kv.v_stride_head,
                           keys ? kv.k_stride_page : kv.v_stride_page};
    cuuint64_t dims[4] = {64, (cuuint64_t)kv.page_size, (cuuint64_t)kv.H_kv, (cuuint64_t)std::max(1, kv.num_pages)};
    cuuint64_t strides[3] = {(cuuint64_t)st[0] * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[2] * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)std::min(TK, kv.page_size), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, keys ? kv.k : kv.v, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: header, the two launches' piece counters, their pieces, the prefix's parts.
struct PagedWs {
    size_t counters[2], slots[2], part, total;
};
int row_warps(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
PagedWs paged_ws(int B, int H, int H_kv, int T, int prefix_len) {
    PagedWs w{};
    const int R = H / H_kv * T;
    size_t off = sizeof(WsHeader);
    for (int k = 0; k < 2; ++k) {
        w.counters[k] = off;
        off += kMaxGrid * sizeof(unsigned int);
    }
    for (int k = 0; k < (prefix_len > 0 ? 2 : 1); ++k) {
        w.slots[k] = off;
        const int rows = (int)std::min<int64_t>(64, k ? (int64_t)B * R : R);
        off = align256(off + sizeof(float) * 2 * kMaxGrid * 16 * row_warps(rows) * (kHeadDim + 2));
    }
    w.part = off;
    if (prefix_len > 0) off = align256(off + sizeof(float) * (size_t)B * H * T * (kHeadDim + 2));
    w.total = off;
    return w;
}

template <int WR, bool PREFIX>
cudaError_t launch_split(const CUtensorMap& mk, const CUtensorMap& mv, const SplitParams& p, bool overlap,
                         cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<WR, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)SM_ALLOC);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(kMaxGrid, CTAS_PER_SM * sm_count()));
    cfg.blockDim = dim3(NCONS + 32);
    cfg.dynamicSmemBytes = SM_ALLOC;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    const int kid = PREFIX ? KID_PAGED_PREFIX : KID_PAGED_ATTN;
    launch_begin(kid, stream);
    e = cudaLaunchKernelEx(&cfg, paged_split_kernel<WR, PREFIX>, mk, mv, p);
    launch_end(kid, stream);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <bool PREFIX>
cudaError_t launch_split_rows(const CUtensorMap& mk, const CUtensorMap& mv, SplitParams& p, bool overlap,
                              cudaStream_t stream) {
    const int wr = row_warps(p.rows);
    p.nrb = (p.rows + 16 * wr - 1) / (16 * wr);
    // the tile axis in the kernel's integers: a sequence's units and all tiles in 31 bits
    const double most = std::max(1, (std::max(p.max_len, p.prefix_len) + TK - 1) / TK);
    if (most * p.nrb * p.wsum >= 2147483648.0 || most * p.nseq >= 2147483648.0) return cudaErrorNotSupported;
    switch (wr) {
        case 1: return launch_split<1, PREFIX>(mk, mv, p, overlap, stream);
        case 2: return launch_split<2, PREFIX>(mk, mv, p, overlap, stream);
        default: return launch_split<4, PREFIX>(mk, mv, p, overlap, stream);
    }
}

}  // namespace

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len) {
    return paged_ws(B, H, H_kv, T, prefix_len).total;
}

cudaError_t launch_paged_attn(const PagedCall& c, cudaStream_t stream) {
    CUtensorMap mk, mv;
    if (!make_tmap_pages(c.kv, true, &mk) || !make_tmap_pages(c.kv, false, &mv)) return cudaErrorNotSupported;
    const PagedWs w = paged_ws(c.B, c.H, c.kv.H_kv, c.T, c.prefix_len);
    SplitParams p{};
    p.q = c.q;
    p.o = c.o;
    p.lse = c.lse;
    p.a = c.a;
    p.r = c.r;
    p.pattern_len = c.pattern_len;
    p.prefix_len = c.prefix_len;
    p.replaced = c.replaced;
    p.keyless = c.keyless;
    p.seq_lens = c.seq_lens;
    p.q_lens = c.q_lens;
    p.num_pages = c.kv.num_pages;
    p.Hkv = c.kv.H_kv;
    while ((1 << p.log_page) < c.kv.page_size) ++p.log_page;
    p.B = c.B;
    p.H = c.H;
    p.T = c.T;
    p.G = c.H / c.kv.H_kv;
    p.R = p.G * c.T;
    p.max_len = c.max_len;
    for (int g = 0; g < p.Hkv; ++g)
        for (int k = c.keyless.get(g) ? 1 : 2; k > 0; --k) p.g_of_w[p.wsum++] = (uint8_t)g;
    p.err = reinterpret_cast<unsigned int*>(c.ws);
    if (c.prefix_len > 0) {
        p.part = reinterpret_cast<float*>(c.ws + w.part);
        p.table = c.prefix_table;
        p.table_stride = 0;
        p.nseq = 1;
        p.rows = c.B * p.R;
        p.counters = reinterpret_cast<unsigned int*>(c.ws + w.counters[1]);
        p.slots = reinterpret_cast<float*>(c.ws + w.slots[1]);
        const cudaError_t e = launch_split_rows<true>(mk, mv, p, false, stream);
        if (e != cudaSuccess) return e;
    }
    p.table = c.page_table;
    p.table_stride = c.max_pages;
    p.nseq = c.B;
    p.rows = p.R;
    p.counters = reinterpret_cast<unsigned int*>(c.ws + w.counters[0]);
    p.slots = reinterpret_cast<float*>(c.ws + w.slots[0]);
    return launch_split_rows<false>(mk, mv, p, c.prefix_len > 0, stream);
}

}  // namespace saf
