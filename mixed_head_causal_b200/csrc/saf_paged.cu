// Attention of a few new tokens per sequence over the paged key/value cache.
//
// Work is a list of items (sequence b, K/V head g, row block): the rows of one
// item are the G = H / H_kv query heads of the group times the T new tokens,
// and share every key.  Keys come in tiles of 16 KB: 64 keys with K and V, or 128
// of V alone for a K/V head whose query heads are all replaced (it has no
// keys).  The tiles of all items form one axis, and each CTA of a grid that
// fills the GPU takes an equal stretch of it: lengths are read on the device,
// so a captured call follows them.  An item that one CTA holds whole is written
// at once; the others leave (m, l, O) pieces in the workspace, and the CTA that
// finishes an item's last piece joins them in key order (the result does not
// depend on which CTA that is).  An item costs a CTA about 2 us besides its
// tiles, and joining pieces 3 us of round trips, each a few tiles' worth of
// reading: an item begins with kItem units on the axis that stand for no tile, a CTA
// gets at least kMinUnits, and a stretch that would end within kSnap units of an
// item's ends ends there.
//
// A CTA is one producer warp and four or eight consumer warps.  The producer
// walks the items ahead of the others, works out their rows, fetches their
// queries, looks up the pages of a tile and fetches them by TMA (128-byte swizzle)
// into a ring, a box per page (64 rows at most).  The consumer warps take 64 keys
// in turn (a tile of V alone goes to two of them), so that one warp's chain of
// MMA, maximum, exponentials, MMA overlaps the others'.  The few rows are the N
// side of the warp-level m16n8k16 MMAs, eight to a block, and the keys (then the
// 64 columns of V) the M side:
//   S^T = K Q^T                    (M keys, N rows), a running maximum m and sum l per row
//   ordinary row   s = q . k / 8
//   replaced row   s = a[j] + r[i - j]      (Eq. (3): its softmax is the pattern)
//   O^T += V^T P^T                 (M columns, N rows), P = exp(s - m) as bf16
// The warps' (m, l, O) are joined at the end of an item.
//
// One new token makes this a stream of K and V at a few flops per byte: HBM
// bounds it, so the warp-level MMAs are enough, and the kernel is built for bytes
// in flight and short chains.  64 sequences of 16384 keys, 12 heads (3 replaced, no K):
// 2.82 GB in 416 to 425 us, 6.6 to 6.8 TB/s (a plain copy's rate).  Short work shows the
// latencies instead: 8 sequences of up to 4096 keys 22 us (10 at that rate), 512 keys
// of one sequence 8.7 us; five drafted tokens of 32 sequences (four heads to a K/V
// head: 20 rows, four warps for want of registers) 95 us against 52.
// Rows on the M side, sixteen at least, would leave most of an MMA to padding: with the
// keys there instead, 96 registers hold a warp's rows and eight warps fit (the first
// of these shapes 515 -> 418 us).
#include <atomic>

#include "mma_util.cuh"
#include "saf_paged.cuh"

namespace saf {
namespace {

using namespace tc;
using mma::mma_bf16;

constexpr int TK = 64;               // keys per tile with K and V (twice as many of V alone)
constexpr int CTAS_PER_SM = 2;
struct SplitAxis {
    static constexpr int kTile = TK, kTileKeyless = 2 * TK, kUnit = 1, kUnitKeyless = 1, kItem = 4, kSnap = 4, kMinUnits = 8;
};
constexpr uint32_t HALF = TK * 128;  // bytes of a tile's K or V
constexpr uint32_t STAGE = 2 * HALF;
constexpr int RED_PITCH = 68;        // floats per row of a warp's O: a warp's stores hit distinct banks
constexpr int Q_PITCH = 144;         // bytes per query row in shared memory: eight rows' words hit distinct banks

// What the consumers need of an item's stretch: tiles [t0, t1), pieces of the
// item in all, the CTA of its first one; vmin: keys that every row sees; replaced:
// bit per row (those that see a key).
struct Piece {
    int len, keyed, t0, t1, pieces, c_first, rows, vmin;
    uint32_t replaced;
};
// Shared memory of a CTA whose items hold up to 8 NB rows, two CTAs to an SM.
template <int NB>
struct Smem {
    static constexpr int ROWS = 8 * NB;
    static constexpr int NCW = NB == 1 ? 8 : 4;                     // consumer warps (their registers: see KC)
    static constexpr int NS = NB <= 2 ? 5 : 4;                      // ring stages
    static constexpr int NI = NB <= 2 ? 4 : 3;                      // items under way
    static constexpr int KC = NB <= 2 ? 64 : 32;                    // keys whose scores a warp holds at a time
    static constexpr uint32_t RED = NS * STAGE;                     // [NCW][ROWS][RED_PITCH] O of a warp
    static constexpr uint32_t ML = RED + NCW * ROWS * RED_PITCH * 4;  // [NCW][ROWS] m, then l
    static constexpr uint32_t ITEM = ML + 2 * NCW * ROWS * 4;       // [NI] Piece
    static constexpr uint32_t INFO = ITEM + NI * 48;                // [NI][ROWS] RowInfo
    static constexpr uint32_t Q = INFO + NI * ROWS * sizeof(RowInfo);  // [NI][ROWS][Q_PITCH]
    static constexpr uint32_t BAR = Q + NI * ROWS * Q_PITCH;        // ring full, empty; item full, free; join
    static constexpr uint32_t META = BAR + 16 * NS + 16 * NI + 8;   // [NS] boxes of a stage without a page; tiles issued; last
    static constexpr uint32_t TOTAL = META + 4 * NS + 8 + 1024;     // the ring starts on a 1024-byte boundary
};
static_assert(sizeof(Piece) <= 48 && sizeof(RowInfo) == 32, "shared memory slots");

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(n) : "memory");
}
// A packed 8 x 8 matrix of 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

template <int NB, bool PREFIX>
__global__ void __launch_bounds__(32 * (Smem<NB>::NCW + 1), CTAS_PER_SM)
paged_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ PagedParams p) {
    using L = Smem<NB>;
    constexpr int ROWS = L::ROWS, NCW = L::NCW, NS = L::NS, NI = L::NI, KB = L::KC / 16, NCONS = 32 * NCW;
    // P is rounded to one bf16 (half a step of 2^-8 off): as a hi + lo pair the second product takes 20.0 us instead of
    // 17.8 at 8 sequences of up to 4096 keys that are in L2 (416 instead of 413 at 64 of 16384).  O is divided by the sum
    // of the rounded weights, as the layer's forward divides a replaced head's: what all keys have in common comes
    // out exactly, and a dominant key's V is not scaled by its weight's rounding.  l, which lse and the joins
    // go by, is the sum of the weights before they are rounded.
    constexpr int SLOT = ROWS * (kHeadDim + 2);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bar_full = sbase + L::BAR, bar_empty = bar_full + 8 * NS;
    const uint32_t bar_item = bar_empty + 8 * NS, bar_taken = bar_item + 8 * NI, bar_join = bar_taken + 8 * NI;
    uint32_t* meta = reinterpret_cast<uint32_t*>(smem + L::META);
    volatile int* issued = reinterpret_cast<int*>(smem + L::META) + NS;  // tiles whose loads the producer has issued
    volatile int* last_flag = issued + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 2);
        }
        for (int s = 0; s < NI; ++s) {
            mbar_init(bar_item + 8 * s, 1);
            mbar_init(bar_taken + 8 * s, NCW);
        }
        mbar_init(bar_join, NCW);
        *issued = 0;
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    // The launch may overlap the one before it on the stream, whose results are awaited before any is read.  After a
    // prefix's launch, which has waited for what came before both, only its results are (see below).
    if (PREFIX || !p.part) griddep_wait();
    griddep_launch_dependents();
    __syncthreads();

    if (warp == NCW) {
        // ------------------------------------------------ producer
        AxisWalk<SplitAxis, PREFIX> walk(p, blockIdx.x, gridDim.x);
        const int lp = p.log_page, lb = min(lp, 6);  // page and box rows
        const uint32_t box_bytes = 128u << lb;
        int it = 0, ni = 0;  // tiles whose loads have been issued, items whose queries have
        unsigned gave_up = 0;
        // What the producer waits for comes from warps that stop for a prefix's launch before they leave their first
        // item, for as long as it takes.  Past that item it awaits that launch itself, once there is something to wait
        // for, and only then is the wait bounded.
        bool behind = !PREFIX && p.part;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (behind && ni > 0 && !__all_sync(~0u, mbar_try_wait(bar, parity))) {
                griddep_wait();
                behind = false;
            }
            return mbar_wait_warp(bar, parity, p.wait_limit);
        };
        for (; !gave_up; ++ni) {
            Piece x;
            Stretch w;
            x.t1 = -1;  // no more
            if (walk.next(w)) {
                x.len = w.len;
                x.keyed = w.keyed;
                x.t0 = w.t0;
                x.t1 = w.t1;
                x.pieces = w.pieces;
                x.c_first = w.c_first;
            }
            const int slot = ni % NI;
            if (!wait(bar_taken + 8 * slot, ((ni / NI) & 1) ^ 1)) {
                gave_up = 0x403;
                break;
            }
            if (x.t1 < 0) {
                if (lane == 0) {
                    reinterpret_cast<Piece*>(smem + L::ITEM + 48 * slot)->t1 = -1;
                    mbar_arrive(bar_item + 8 * slot);
                }
                break;
            }
            const int g = p.e_g[w.e], row0 = w.rb * ROWS;
            x.rows = min(ROWS, max(0, p.e_heads[w.e] * w.n_rows - row0));
            int out;
            {  // a lane per row
                const RowInfo row = row_info<PREFIX>(p, w.b, w.e, w.len, w.n_rows, row0 + lane);
                x.replaced = __ballot_sync(~0u, lane < x.rows && row.replaced && row.vis > 0);
                x.vmin = __reduce_min_sync(~0u, lane < x.rows && row.out >= 0 ? row.vis : INT_MAX);
                out = row.out;
                if (lane < ROWS) *reinterpret_cast<RowInfo*>(smem + L::INFO + (slot * ROWS + lane) * sizeof(RowInfo)) = row;
            }
            if (lane == 0) *reinterpret_cast<Piece*>(smem + L::ITEM + 48 * slot) = x;
            __syncwarp();
            if (lane == 0) mbar_expect_tx(bar_item + 8 * slot, x.rows * 128);
            __syncwarp();
            if (lane < x.rows) {  // the queries, a row that has no token taking row 0's
                bulk_load(sbase + L::Q + (slot * ROWS + lane) * Q_PITCH, p.q + (size_t)max(out, 0) * kHeadDim, 128,
                          bar_item + 8 * slot);
            }
            const int tk = w.keyed ? TK : 2 * TK, boxes = tk >> lb;
            const int32_t* table = p.table + (size_t)w.b * p.table_stride;
            const int npages = (x.len + (1 << lp) - 1) >> lp;
            int ids = -1, ids0 = -64;  // page ids [ids0, ids0 + 32), one per lane
            for (int t = x.t1 - 1; t >= x.t0; --t, ++it) {  // last tile first (see the consumers)
                const int s = it % NS, key = t * tk + (lane << lb);  // this lane's box
                const int pg_lo = (t * tk) >> lp, pg_hi = (t * tk + tk - 1) >> lp;
                if (pg_lo < ids0 || pg_hi >= ids0 + 32) {
                    ids0 = max(0, pg_hi - 31);
                    ids = ids0 + lane < npages ? __ldg(table + ids0 + lane) : -1;
                }
                const int page = __shfl_sync(~0u, ids, ((key >> lp) - ids0) & 31);
                const bool need = lane < boxes && key < x.len;
                const bool good = need && page >= 0 && page < p.num_pages;
                const uint32_t bad = __ballot_sync(~0u, need && !good);
                const int loads = __popc(__ballot_sync(~0u, good));
                if (!wait(bar_empty + 8 * s, ((it / NS) & 1) ^ 1)) {
                    gave_up = 0x401;
                    break;
                }
                if (lane == 0) {
                    meta[s] = bad;
                    mbar_expect_tx(bar_full + 8 * s, loads * box_bytes * (w.keyed ? 2 : 1));
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = sbase + s * STAGE + lane * box_bytes;
                    const int y = key & ((1 << lp) - 1);
                    if (w.keyed) tma_load_4d(dst, &tmK, bar_full + 8 * s, 0, y, g, page);
                    tma_load_4d(dst + (w.keyed ? HALF : 0), &tmV, bar_full + 8 * s, 0, y, g, page);
                }
                if (lane == 0) *issued = it + 1;
            }
        }
        if (gave_up && lane == 0) report(p.err, gave_up);
        if (lane == 0) {  // the loads in flight land before the shared memory is let go, whether a consumer still wants them or not
            for (int k = max(0, it - NS); k < it; ++k) mbar_wait(bar_full + 8 * (k % NS), (k / NS) & 1, kDrainLimit);
            // (the mark of the end stands in the place of item ni - NI, which the consumers have taken)
            for (int k = max(0, gave_up ? ni - NI : ni - NI + 1); k < ni; ++k)
                mbar_wait(bar_item + 8 * (k % NI), (k / NI) & 1, kDrainLimit);
        }
        // A grid in which none has waited may end before the one ahead of it, and the next would start too soon.
        if (!PREFIX && p.part) griddep_wait();
        return;
    }

    // ---------------------------------------------------- consumers
    float* red = reinterpret_cast<float*>(smem + L::RED);
    float* red_m = reinterpret_cast<float*>(smem + L::ML);
    float* red_l = red_m + NCW * ROWS;
    float* mine = red + warp * ROWS * RED_PITCH;
    const int lb = min(p.log_page, 6);
    const int r0 = (lane & 3) * 2;  // this thread's rows of a block: r0, r0 + 1; its keys of a 16-key step: lane / 4, + 8
    int it = 0;                     // tiles of the CTA before this item
    uint32_t joins = 0;
    bool ok = true, waited = false;  // a wait that gave up: no more waits, and the warp leaves at its next item
    // A barrier of the consumer warps, bounded like every wait.
    auto join_warps = [&] {
        mbar_arrive_warp(bar_join);
        if (ok) {
            ok = mbar_wait_warp(bar_join, joins & 1, p.wait_limit);
            if (!ok && lane == 0) report(p.err, 0x405);
        }
        ++joins;
    };
    for (int ni = 0;; ++ni) {
        if (ok) {
            ok = mbar_wait_warp(bar_item + 8 * (ni % NI), (ni / NI) & 1, p.wait_limit);
            if (!ok && lane == 0) report(p.err, 0x404);
        }
        const Piece x = *reinterpret_cast<const Piece*>(smem + L::ITEM + 48 * (ni % NI));
        const RowInfo* info = reinterpret_cast<const RowInfo*>(smem + L::INFO) + (ni % NI) * ROWS;
        if (x.t1 < 0 || !ok) break;
        uint32_t qf[NB][4][2];  // Q^T fragments; a replaced row's queries are not used
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int row = nb * 8 + (lane >> 2);
            const bool read = row < x.rows && !((x.replaced >> row) & 1u);
            const uint32_t src = sbase + L::Q + ((ni % NI) * ROWS + row) * Q_PITCH + (lane & 3) * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                qf[nb][k][0] = read ? ld_shared_u32(src + 32 * k) : 0u;
                qf[nb][k][1] = read ? ld_shared_u32(src + 32 * k + 16) : 0u;
            }
        }
        // Running maximum (in units of the row's scores: dot products for an ordinary row), its log2(e) per unit, the sum
        // (of this thread's keys) and O^T (columns 16 db + lane / 4, + 8), for this thread's two rows of each block.
        float m[NB][2], o[4][NB][4];
        uint64_t unit2[NB], l2[NB], lr2[NB];  // lr2: the sum of the rounded weights
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float un[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nb][e] = kNegInf;
                un[e] = ((x.replaced >> (nb * 8 + r0 + e)) & 1u) ? kLog2e : 0.125f * kLog2e;
            }
            unit2[nb] = f32x2(un[0], un[1]);
            l2[nb] = lr2[nb] = 0;
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][nb][e] = 0.f;
        }
        // The warps' turns: a tile with K and V goes to one warp, one of V alone to two.
        const int turns = x.keyed ? NCW : NCW / 2, turn = x.keyed ? warp : warp >> 1, sub = x.keyed ? 0 : warp & 1;
        const int tk = x.keyed ? TK : 2 * TK;
        // Last tile first: patterns tend to favour near keys, so that the running maximum starts near where it ends.
        int t = x.t1 - 1 - ((turn - it) & (turns - 1));
        // A replaced row's scores of 64 keys are summed lane by lane (two each) into the warp's part of `red`, and
        // read back in the fragment's order.  The first such row's are loaded a step ahead; the others of the same
        // head then find theirs in L1.
        float ahead[4];
        auto load_ahead = [&](int key) {
            const RowInfo& w = info[__ffs(x.replaced) - 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = max(0, min(key + lane + 32 * e, w.vis - 1));
                ahead[e] = __ldg(p.a + w.a0 + j);
                ahead[2 + e] = __ldg(p.r + w.r0 - j);
            }
        };
        if (x.replaced) load_ahead(t * tk + sub * TK);

        for (; t >= x.t0; t -= turns) {
            const unsigned at = (unsigned)(it + x.t1 - 1 - t), s = at % NS;
            const int k0 = t * tk + sub * TK;
            const uint32_t sk = sbase + s * STAGE, sv = sk + (x.keyed || sub ? HALF : 0);
            if (x.replaced) {
                const int first = __ffs(x.replaced) - 1;
                mine[first * RED_PITCH + lane] = ahead[0] + ahead[2];
                mine[first * RED_PITCH + lane + 32] = ahead[1] + ahead[3];
                load_ahead(k0 - turns * tk);
                for (uint32_t left = x.replaced & (x.replaced - 1); left;) {  // four rows' loads at a time
                    float v[4][4];
                    int rows[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        rows[u] = left ? __ffs(left) - 1 : rows[0];
                        left &= left - 1;
                        const RowInfo& w = info[rows[u]];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = min(k0 + lane + 32 * e, w.vis - 1);
                            v[u][e] = __ldg(p.a + w.a0 + j);
                            v[u][2 + e] = __ldg(p.r + w.r0 - j);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        mine[rows[u] * RED_PITCH + lane] = v[u][0] + v[u][2];
                        mine[rows[u] * RED_PITCH + lane + 32] = v[u][1] + v[u][3];
                    }
                }
                __syncwarp();
            }
            // The stages are handed round, so a warp meets a stage's fills now and then.  Once the producer has issued this
            // tile, the stage's fill before has been used up, and its barrier's parity can only tell of this one.
            if (ok && *issued <= (int)at) {
                const long long began = clock64();
                while (*issued <= (int)at && ok) ok = clock64() - began < p.wait_limit;
            }
            ok = __all_sync(~0u, ok);
            if (ok) ok = mbar_wait_warp(bar_full + 8 * s, (at / NS) & 1, p.wait_limit);
            if (!ok && lane == 0) report(p.err, 0x402);
            const uint32_t bad = meta[s] >> (sub ? TK >> lb : 0);
            const bool whole = k0 + TK <= x.vmin && bad == 0;  // every row sees every key
            if (!whole) {  // a slot without a token may hold a NaN, and 0 times that is one: its V becomes zeros
#pragma unroll 1
                for (int j = lane; j < TK; j += 32) {
                    if (k0 + j < x.len && !((bad >> (j >> lb)) & 1u)) continue;
                    // a row per lane, the lanes' 16 bytes in distinct banks (unrolled where there are registers: 20 rows
                    // lose 13 us of 97 to spills otherwise)
#pragma unroll(NB == 1 ? 8 : 1)
                    for (int c = 0; c < 8; ++c) st_shared_v4(sv + 128 * j + 16 * ((c + lane) & 7), 0, 0, 0, 0);
                }
                fence_proxy_async_smem();  // (before the stage's next load)
                __syncwarp();
            }
#pragma unroll
            for (int kc = 0; kc < TK; kc += L::KC) {
                float st[KB][NB][4];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) st[kb][nb][e] = 0.f;
                if (x.keyed) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            uint32_t a[4];
                            mma::load_a_frag(a, sk, kc + kb * 16, k * 16, lane);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) mma_bf16(st[kb][nb], a, qf[nb][k][0], qf[nb][k][1]);
                        }
                }
                if (x.replaced) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if ((x.replaced >> (nb * 8 + r0 + e)) & 1u) {
                                const float* src = mine + (nb * 8 + r0 + e) * RED_PITCH + kc + (lane >> 2);
#pragma unroll
                                for (int kb = 0; kb < KB; ++kb) {
                                    st[kb][nb][e] = src[kb * 16];
                                    st[kb][nb][2 + e] = src[kb * 16 + 8];
                                }
                            }
                }
                if (!whole) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        // this thread's keys are kb * 16 + 8 * (e >> 1) past the first of them
                        const int first = k0 + kc + (lane >> 2), v0 = info[nb * 8 + r0].vis - first, v1 = info[nb * 8 + r0 + 1].vis - first;
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (kb * 16 + 8 * (e >> 1) >= ((e & 1) ? v1 : v0)) st[kb][nb][e] = kNegInf;
                    }
                    if (bad) {
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int jl = kc + kb * 16 + (lane >> 2) + 8 * u;
                                if (!((bad >> (jl >> lb)) & 1u)) continue;
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) st[kb][nb][2 * u] = st[kb][nb][2 * u + 1] = kNegInf;
                            }
                    }
                }
                // The maximum moves only when a score passes it by more than 2^8: P and the sums stay far from fp32's limits,
                // and most steps need no reduction across the lanes and no rescaling.
                bool grow = false;
                float mx[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float2 un = split_f32x2(unit2[nb]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(st[0][nb][e], st[0][nb][2 + e]);
#pragma unroll
                        for (int kb = 1; kb < KB; ++kb) v = max3(v, st[kb][nb][e], st[kb][nb][2 + e]);
                        mx[nb][e] = v;
                        grow |= (v - m[nb][e]) * (e ? un.y : un.x) > 8.f;
                    }
                }
                if (__any_sync(~0u, grow)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const float2 un = split_f32x2(unit2[nb]);
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = mx[nb][e];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
                            const float u = e ? un.y : un.x;
                            const bool up = (v - m[nb][e]) * u > 8.f;
                            f[e] = up ? ex2((m[nb][e] - v) * u) : 1.f;
                            if (up) m[nb][e] = v;
                        }
                        l2[nb] = mul_f32x2(l2[nb], f32x2(f[0], f[1]));
                        lr2[nb] = mul_f32x2(lr2[nb], f32x2(f[0], f[1]));
#pragma unroll
                        for (int d = 0; d < 4; ++d)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[d][nb][e] *= f[e & 1];
                    }
                }
                // P^T, rounded, turned into the second product's B fragments
                uint32_t pt[KB][NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // (x - m) * unit, not x * unit - m * unit: the products may overflow where the difference is small
                    const uint64_t base2 = f32x2(m[nb][0] == kNegInf ? 0.f : m[nb][0], m[nb][1] == kNegInf ? 0.f : m[nb][1]);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 e =
                                split_f32x2(mul_f32x2(sub_f32x2(f32x2(st[kb][nb][2 * u], st[kb][nb][2 * u + 1]), base2), unit2[nb]));
                            const float p0 = ex2(e.x), p1 = ex2(e.y);
                            l2[nb] = add_f32x2(l2[nb], f32x2(p0, p1));
                            const uint32_t pr = pack_bf16x2(p0, p1);
                            lr2[nb] = add_f32x2(lr2[nb], pair_of(pr));
                            pt[kb][nb][u] = transpose8(pr);
                        }
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        // V^T: 16 columns x 16 keys, from V stored [key][column]
                        uint32_t a[4];
                        const int key = kc + kb * 16 + (lane & 7) + (lane >> 4) * 8, col = d * 16 + ((lane >> 3) & 1) * 8;
                        mma::ldsm_x4_t(a[0], a[1], a[2], a[3], sv + mma::swz(key, col));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_bf16(o[d][nb], a, pt[kb][nb][0], pt[kb][nb][1]);
                    }
                }
            }
            __syncwarp();
            // (a stage that this warp has given up on may still be landing, and is not filled again)
            if (lane == 0 && ok) mbar_arrive_n(bar_empty + 8 * s, x.keyed ? 2 : 1);
        }
        it += x.t1 - x.t0;

        // ---- the warps' parts to shared memory, joined over the keys
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float2 ll = split_f32x2(l2[nb]), lr = split_f32x2(lr2[nb]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nb * 8 + r0 + e;
                float l = e ? ll.y : ll.x, rounded = e ? lr.y : lr.x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l += __shfl_xor_sync(~0u, l, d);
                    rounded += __shfl_xor_sync(~0u, rounded, d);
                }
                const float f = by_rounded(l, rounded);
                if (lane < 4) {
                    red_m[warp * ROWS + row] = ((x.replaced >> row) & 1u) ? m[nb][e] : 0.125f * m[nb][e];
                    red_l[warp * ROWS + row] = l;
                }
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    mine[row * RED_PITCH + d * 16 + (lane >> 2)] = o[d][nb][e] * f;
                    mine[row * RED_PITCH + d * 16 + (lane >> 2) + 8] = o[d][nb][2 + e] * f;
                }
            }
        }
        join_warps();
        const int c = (tid & 15) * 4;
        if (!PREFIX && p.part && !waited) {
            griddep_wait();
            waited = true;
        }
        float* slot = p.slots + ((size_t)blockIdx.x * 2 + (x.t0 == 0)) * SLOT;
        for (int row = tid >> 4; row < x.rows; row += NCONS / 16) {
            float mm = kNegInf;
#pragma unroll
            for (int k = 0; k < NCW; ++k) mm = fmaxf(mm, red_m[k * ROWS + row]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll
            for (int k = 0; k < NCW; ++k) {
                const float f = weight(red_m[k * ROWS + row], mm);
                const float4 v = *reinterpret_cast<const float4*>(red + (k * ROWS + row) * RED_PITCH + c);
                acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
                ll += f * red_l[k * ROWS + row];
            }
            if (x.pieces == 1) {
                finish_row<PREFIX>(p, info[row], c, acc, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4*>(slot + row * kHeadDim + c), acc);
                if (c == 0) {
                    __stcg(slot + ROWS * kHeadDim + row, mm);
                    __stcg(slot + ROWS * (kHeadDim + 1) + row, ll);
                }
            }
        }
        if (x.pieces > 1) {
            __threadfence();
            join_warps();
            if (tid == 0) *last_flag = atomicAdd(p.counters + x.c_first, 1u) == (unsigned)x.pieces - 1;
            join_warps();
            if (*last_flag && ok) {
                __threadfence();
                auto slot_of = [&](int k) { return p.slots + ((size_t)(x.c_first + k) * 2 + (k == 0)) * SLOT; };
                for (int row = tid >> 4; row < x.rows; row += NCONS / 16) {
                    float mm = kNegInf;
                    for (int k = tid & 15; k < x.pieces; k += 16) mm = fmaxf(mm, __ldcg(slot_of(k) + ROWS * kHeadDim + row));
                    // the sixteen threads of a row are a half-warp that runs this loop together
                    const uint32_t half = 0xffffu << (lane & 16);
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(half, mm, d));
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float ll = 0.f;
#pragma unroll 4
                    for (int k = 0; k < x.pieces; ++k) {
                        const float* sl = slot_of(k);
                        const float f = weight(__ldcg(sl + ROWS * kHeadDim + row), mm);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(sl + row * kHeadDim + c));
                        acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
                        ll += f * __ldcg(sl + ROWS * (kHeadDim + 1) + row);
                    }
                    finish_row<PREFIX>(p, info[row], c, acc, mm, ll);
                }
                if (tid == 0) atomicExch(p.counters + x.c_first, 0u);
            }
        }
        join_warps();  // the shared parts have been read
        if (lane == 0) mbar_arrive(bar_taken + 8 * (ni % NI));
    }
}

// ------------------------------------------------------------------ host side
// Items of more rows than this go to the tensor-core kernel.  Measured, this kernel's us against that one's: 16 rows (a
// prefix of 2048 keys) 30 against 40, 24 of them 39 against 35; 20 rows (32 sequences of up to 8192 keys, 4 heads to a
// K/V head) 95 against 185, 24 of them 101 against 187; 32 rows of the same two kinds 67 against 38, 200 against 193
// (a fourth block of eight spills).
constexpr int kTcRows = 24;

// Workspace: header, the two launches' piece counters, shared items and pieces,
// the prefix's parts.  Sizes grow with each argument.
struct PagedWs {
    size_t counters[2], shared[2], slots[2], part, total;
};
PagedWs paged_ws(int B, int H, int H_kv, int T, int prefix_len) {
    PagedWs w{};
    const int R = H / H_kv * T;
    size_t off = sizeof(WsHeader);
    for (int k = 0; k < 2; ++k) {
        w.counters[k] = off;
        off += kMaxGrid * sizeof(unsigned int);
    }
    for (int k = 0; k < 2; ++k) {
        w.shared[k] = off = align256(off);
        off += kMaxGrid * sizeof(SharedItem);
    }
    off = align256(off);
    for (int k = 0; k < (prefix_len > 0 ? 2 : 1); ++k) {
        const int rows = k ? B * R : R, most = rows > kTcRows ? 128 : (rows + 7) & ~7;
        w.slots[k] = off;
        off = align256(off + sizeof(float) * 2 * kMaxGrid * most * (kHeadDim + 2));
    }
    w.part = off;
    if (prefix_len > 0) off = align256(off + sizeof(float) * (size_t)B * H * T * (kHeadDim + 2));
    w.total = off;
    return w;
}

template <int NB, bool PREFIX>
cudaError_t launch_split(const CUtensorMap& mk, const CUtensorMap& mv, const PagedParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<NB, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Smem<NB>::TOTAL);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)paged_grid());
    cfg.blockDim = dim3(32 * (Smem<NB>::NCW + 1));
    cfg.dynamicSmemBytes = Smem<NB>::TOTAL;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int kid = PREFIX ? KID_PAGED_PREFIX : KID_PAGED_ATTN;
    launch_begin(kid, stream);
    e = cudaLaunchKernelEx(&cfg, paged_split_kernel<NB, PREFIX>, mk, mv, p);
    launch_end(kid, stream);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <bool PREFIX>
cudaError_t launch_split_rows(const saf_paged_kv& kv, PagedParams& p, cudaStream_t stream) {
    CUtensorMap mk, mv;
    if (!make_tmap_pages(kv, true, TK, &mk) || !make_tmap_pages(kv, false, TK, &mv)) return cudaErrorNotSupported;
    p.pad = 1;
    static_assert(kTcRows == 24, "three blocks of eight rows");
    make_entries(p, p.G, p.G, false);
    p.block_rows = ((PREFIX ? p.B * p.R : p.R) + 7) & ~7;  // (all in one block)
    p.by_block = divisor(p.block_rows);
    if (!axis_fits<SplitAxis>(p, PREFIX)) return cudaErrorNotSupported;
    switch (p.block_rows / 8) {
        case 1: return launch_split<1, PREFIX>(mk, mv, p, stream);
        case 2: return launch_split<2, PREFIX>(mk, mv, p, stream);
        default: return launch_split<3, PREFIX>(mk, mv, p, stream);
    }
}

}  // namespace

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len) {
    return paged_ws(B, H, H_kv, T, prefix_len).total;
}

namespace {
std::atomic<long long> g_wait_limit{kServingWaitLimit};
}
void set_serving_wait_limit(long long cycles) { g_wait_limit = cycles ? cycles : kServingWaitLimit; }

cudaError_t launch_paged_attn(const PagedCall& c, cudaStream_t stream) {
    const PagedWs w = paged_ws(c.B, c.H, c.kv.H_kv, c.T, c.prefix_len);
    PagedParams p{};
    p.q = c.q;
    p.o = c.o;
    p.lse = c.lse;
    p.a = c.a;
    p.r = c.r;
    p.pattern_len = c.pattern_len;
    p.prefix_len = c.prefix_len;
    p.replaced = c.replaced;
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
    for (int g = 0, at = 0; g < p.Hkv; ++g)
        for (int want = 0; want < 2; ++want)
            for (int h = g * p.G; h < (g + 1) * p.G; ++h)
                if (c.replaced.get(h) == (want == 1)) p.heads[at++] = (uint8_t)h;
    p.by_T = divisor(p.T);
    p.by_BT = p.by_BT_pad = divisor(p.B * p.T);
    p.err = reinterpret_cast<unsigned int*>(c.ws);
    p.wait_limit = g_wait_limit;
    if (c.prefix_len > 0) {
        p.part = reinterpret_cast<float*>(c.ws + w.part);
        p.part_rows = c.B * c.H * c.T;
        p.table = c.prefix_table;
        p.table_stride = 0;
        p.nseq = 1;
        p.counters = reinterpret_cast<unsigned int*>(c.ws + w.counters[1]);
        p.slots = reinterpret_cast<float*>(c.ws + w.slots[1]);
        p.shared = reinterpret_cast<SharedItem*>(c.ws + w.shared[1]);
        const cudaError_t e = c.B * p.R > kTcRows ? launch_paged_tc(c.kv, p, true, stream)
                                               : launch_split_rows<true>(c.kv, p, stream);
        if (e != cudaSuccess) return e;
    }
    p.table = c.page_table;
    p.table_stride = c.max_pages;
    p.nseq = c.B;
    p.counters = reinterpret_cast<unsigned int*>(c.ws + w.counters[0]);
    p.slots = reinterpret_cast<float*>(c.ws + w.slots[0]);
    p.shared = reinterpret_cast<SharedItem*>(c.ws + w.shared[0]);
    if (p.R <= kTcRows) return launch_split_rows<false>(c.kv, p, stream);
    return launch_paged_tc(c.kv, p, false, stream);
}

}  // namespace saf
