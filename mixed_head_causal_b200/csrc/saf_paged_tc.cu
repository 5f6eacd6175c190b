// Attention of many rows over the paged key/value cache on the 5th-generation
// tensor cores: prompt chunks, and a shared prefix seen by a whole batch.
//
// An item is 128 rows of one K/V head (its query heads times the new tokens, and
// with a shared prefix times the sequences), its keys in blocks of 128, last block
// first (patterns tend to favour near keys: the running maximum then starts near
// where it ends).  The blocks of all items form one axis, of which every CTA of two
// per SM takes an equal stretch, as in the kernel for few rows (saf_paged.cu).  The
// pieces of an item that several share are joined by a launch of its own, with a
// thread per four columns of every row: the CTA that finishes an item's last piece
// took 13 us over 4 pieces of 128 rows, 50 us over 18.  Six warps:
//   warp 0      producer: walks the stretch, page look-up and TMA loads, a box per
//               page, two stages each of K and V (no K where all rows are replaced)
//   warp 1      TMEM owner and MMA issuer (one elected lane):
//               S = Q K^T  (tcgen05 SS, 128x128x64), O += P V  (TS, 128x64x128)
//   warps 2..5  one row per thread: its queries to shared memory, then per block the
//               scores out of TMEM, the running maximum (moved only when a score
//               passes it by 2^8), P = exp(s - m) as bf16 into TMEM (half a step of
//               2^-8 off), the sum of what is rounded there in fp32
// O is divided as in the layer's forward: a replaced row's by the sum of the rounded weights (an MMA against a tile of
// ones, into columns that hold S where there are keys: eight MMAs of N = 16 a block, no time that shows), so that a dominant key's V is
// not scaled by its weight's rounding; an ordinary row's by the sum of the weights before that (256 columns a CTA leave
// no room beside S, and summing the rounded ones in the row warps took the chunks below from 91 to 99 us).
// S_{j+1} is issued as soon as the rows have copied S_j to registers, before P V_j.
//   ordinary row   s = q . k / 8
//   replaced row   s = a[j] + r[i - j], 32 keys at a time, from shared memory: one stretch
//                  of r for the whole warp where its rows' stretches lie within NEAR_SPAN of
//                  each other (a chunk's tokens, sequences of like lengths), else one per row
//                  (which L2 bounds: a row's own stretch is twice the bytes of a K row)
// Rows come head by head, ordinary and replaced heads in items of their own (those of
// replaced rows need no K), and a replaced head begins with a warp: a warp of two
// heads' rows looks every score up by itself, which took 25 us a block.
// Per block and row: 128 exponentials against 2 x 128 x 64 multiply-adds, so the exp
// unit (16 a cycle and SM: 2048 cycles, 1.1 us, for the two CTAs' blocks) bounds it
// before the tensor pipe (about 770 cycles a block).  Measured per block: 1.8 us of
// ordinary rows, 3.6 of replaced ones near each other, 5.4 far apart.  The row warps
// wait for nothing meanwhile: with two of them to a scheduler (registers and shared
// memory allow no more) the latencies of their own chain of load, maximum, exponential
// and store show.
// 4 sequences of up to 8192 keys, chunks of 500, 12 heads (3 replaced): 92 us, of which
// about 80 this kernel; prefix of 16384 under 256 sequences, 32 heads (8 replaced) on 8: 86 us.
#include "saf_paged.cuh"

namespace saf {
namespace {

using namespace tc;

constexpr int BM = 128, BN = 128;  // rows per CTA, keys per block
constexpr int NST = 2;             // K and V stages
constexpr int NTHREADS = 192;
constexpr uint32_t TILE_BYTES = 128 * 64 * 2;
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t TO_COL = 128, TP_COL = 192;  // S in 0..127, O, P
constexpr uint32_t TSUM_COL = 0;                // the rows' sums of rounded weights, of items without keys (and without S)

// shared memory map (offsets from a 1024-aligned base)
constexpr uint32_t SM_Q = 0;                           // of an item without keys: 16 rows x 128 bytes of ones
constexpr uint32_t SM_K = SM_Q + TILE_BYTES;
constexpr uint32_t SM_V = SM_K + NST * TILE_BYTES;
constexpr int PAT_PITCH = 33;                          // floats: a warp's reads of its 32 rows hit distinct banks
// A staging area holds three buffers of 16 keys: the stretches of 32 rows of r, from the 16-byte boundary at or
// before them on (20 floats a row), and a; or two of 128 keys: a, and one stretch of r that serves all rows, from the
// 16-byte boundary on; or (mixed blocks) the scores of 32 keys of 32 rows.
constexpr int FAR_PITCH = 20, FAR_A = 32 * FAR_PITCH, FAR_BUF = FAR_A + 16, FAR_BUFS = 3;
constexpr int NEAR_SPAN = 720, NEAR_BUF = 128 + 128 + NEAR_SPAN + 4;  // floats; rows at most NEAR_SPAN apart
constexpr uint32_t PAT_BYTES = FAR_BUFS * FAR_BUF * 4;  // a warp's staging area
static_assert(PAT_BYTES >= 32 * PAT_PITCH * 4 && PAT_BYTES >= 2 * NEAR_BUF * 4 && NEAR_BUF % 4 == 0, "all uses fit");
constexpr uint32_t SM_PAT = SM_V + NST * TILE_BYTES;   // [4 warps] staging area
constexpr uint32_t SM_ROW = SM_PAT + 4 * PAT_BYTES;  // [128] {head, r at local key 0 within the head's} of a row
constexpr uint32_t SM_BAR = SM_ROW + 128 * 8;
constexpr uint32_t SM_ITEM = SM_BAR + 20 * 8;       // [2] TcPiece
constexpr uint32_t SM_WARP = SM_ITEM + 2 * 48;      // [4] WarpRows
constexpr uint32_t SM_MISC = SM_WARP + 4 * 80;      // TMEM address, [4] boxes of a K load without a page, [4] of a V load
constexpr uint32_t SM_LIMIT = SM_MISC + 40;         // PagedParams::wait_limit, for the row loops
constexpr uint32_t SM_TOTAL = SM_LIMIT + 8;

struct TcAxis {
    // (a block of replaced rows takes about twice as long as one of ordinary rows: 3.6 us against 1.8, two CTAs per SM)
    static constexpr int kTile = BN, kTileKeyless = BN, kUnit = 2, kUnitKeyless = 4, kItem = 4, kSnap = 4, kMinUnits = 16;
};
// An item's stretch as the other warps need it: nt blocks from t0 (those that some
// row sees; nt < 0: no more items), keyed: some row is ordinary.
struct TcPiece {
    int b, e, rb, len, n_rows, t0, nt, keyed, pieces, c_first, lb;  // lb: log2 of the rows of a box
};
static_assert(sizeof(TcPiece) <= 48, "item slot");
// What the rows of a warp have in common.  It and the item stay in shared memory
// and are read where they are wanted: the row loops below are functions of their
// own, with a handful of scalar arguments, so that little crowds the 128 scores of
// a row out of the registers or goes through the stack (with two CTAs' shared
// memory taken, L1 is too small to hold one: spilled, the loops took twice as long;
// what is left is about 50 to 70 bytes a call of a loop, and 160 in the kernel
// around them).
struct WarpRows {
    const float *a, *r;    // of the head of the first row that looks scores up, at local key 0 (r: at its own position, r[-j])
    const float *a0, *r0;  // the arrays, a0 at local key 0 of head 0
    int pattern_len;
    uint32_t reps;         // the rows that look their scores up
    int one_head;          // all of these are of one head
    int pure;              // all rows with a token look up, by one head's vectors
    int low, span;         // from r on: the lowest of their stretches, and from there to the highest
    int low_edge;          // the 16-byte boundary at or before the lowest's entry of local key 127
    int room, before;      // floats of the array from r on (2^31 - 9 at most), and before it (2^31 - 1 at most)
    int last;              // the last key
    int vmin;              // keys that every row sees
};
static_assert(sizeof(WarpRows) <= 80, "warp slot");
struct RowResult {
    float m, l;
    int ok;
};

__device__ __forceinline__ uint8_t* smem_base() {
    extern __shared__ __align__(1024) uint8_t smem[];
    return smem;
}
__device__ __forceinline__ int quarter_of() { return (threadIdx.x >> 5) & 3; }
__device__ __forceinline__ const volatile TcPiece& item_of(int ni) {
    return reinterpret_cast<volatile TcPiece*>(smem_base() + SM_ITEM)[ni & 1];
}
__device__ __forceinline__ const WarpRows& warp_rows() { return reinterpret_cast<WarpRows*>(smem_base() + SM_WARP)[quarter_of()]; }
// A wait of the row loops (mbar_wait_warp, the limit looked up only where there is something to wait for).
__device__ __forceinline__ bool row_wait(uint32_t bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const long long began = clock64();
        do ok = mbar_try_wait(bar, parity);
        while (!ok && clock64() - began <= *reinterpret_cast<const volatile long long*>(smem_base() + SM_LIMIT));
    }
    return __all_sync(~0u, ok);
}
__device__ __forceinline__ float* staging() { return reinterpret_cast<float*>(smem_base() + SM_PAT + quarter_of() * PAT_BYTES); }

// The values of a TMEM load pass through here once the load has been waited for, so
// that nothing made of them moves ahead of the wait.
__device__ __forceinline__ void loaded(uint32_t (&v)[32]) {
    asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
    asm volatile("" : "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]));
}
// Maxima of 32 raw scores into two independent chains of three-input max.
__device__ __forceinline__ void quarter_max(const uint32_t (&v)[32], float (&mx)[2]) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
}

// P = exp2(s * unit - m * unit) of keys [32 Q, 32 Q + 32) as 16 bf16 pairs, their sum added to l2.
template <int Q>
__device__ __forceinline__ void exp_quarter(const uint32_t (&v)[32], uint64_t unit2, uint64_t nm2, uint64_t (&l2)[4],
                                            uint32_t tP) {
    uint32_t pw[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 x =
            split_f32x2(fma_f32x2(f32x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), unit2, nm2));
        const float p0 = ex2(x.x), p1 = ex2(x.y);
        l2[(e >> 1) & 3] = add_f32x2(l2[(e >> 1) & 3], f32x2(p0, p1));
        pw[e >> 1] = pack_bf16x2(p0, p1);
    }
    tmem_st16(tP + 16 * Q, pw);
}

// This warp's 32 O rows times f, with `sums` the sums of their rounded weights too.
__device__ __forceinline__ void rescale_o(uint32_t tmem, float f, bool sums) {
    const uint32_t tO = tmem + TO_COL;
    if (sums) {
        const float x = __uint_as_float(tmem_ld1(tmem + TSUM_COL));
        tmem_wait_ld();
        tmem_st1(tmem + TSUM_COL, __float_as_uint(x * f));
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t ov[32];
        tmem_ld32(tO + 32 * c, ov);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
        tmem_st32(tO + 32 * c, ov);
    }
}

// Scores of 32 keys, chunk c of a block (which goes from 3 to 0), of a row each:
// the maximum moves if it must (then what the block has written of P so far is
// scaled along with O and l, and rounded to bf16 once more: another half step of 2^-8
// on weights that are at most as large as the new maximum's), P goes to TMEM and
// its sum to l.  first: O holds nothing yet.
__device__ __forceinline__ void chunk_out(const float (&v)[32], int c, bool first, float unit, float& m, float& l,
                                          uint32_t tmem, bool sums) {
    const uint32_t tP = tmem + TP_COL;
    float mx2[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int e = 0; e < 32; e += 2) mx2[(e >> 1) & 1] = max3(mx2[(e >> 1) & 1], v[e], v[e + 1]);
    const float mx = fmaxf(mx2[0], mx2[1]);
    const bool grow = (mx - m) * unit > 8.f;
    if (__any_sync(~0u, grow)) {
        const float f = grow ? ex2((m - mx) * unit) : 1.f;
        if (grow) m = mx;
        l *= f;
        tmem_wait_st();
        if (!first) rescale_o(tmem, f, sums);
#pragma unroll 1
        for (int d = c + 1; d < 4; ++d) {
            uint32_t pw[16];
            tmem_ld16(tP + 16 * d, pw);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                pw[e] = pack_bf16x2(__uint_as_float(pw[e] << 16) * f, __uint_as_float(pw[e] & 0xffff0000u) * f);
            tmem_st16(tP + 16 * d, pw);
        }
        tmem_wait_st();
    }
    // (x - m) * unit, not x * unit - m * unit: a pattern's products may overflow where the difference is small
    const float base = m == kNegInf ? 0.f : m;
    const uint64_t base2 = f32x2(base, base), unit2 = f32x2(unit, unit);
    uint64_t l2[2] = {0, 0};
    uint32_t pw[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 x = split_f32x2(mul_f32x2(sub_f32x2(f32x2(v[e], v[e + 1]), base2), unit2));
        const float p0 = ex2(x.x), p1 = ex2(x.y);
        l2[(e >> 1) & 1] = add_f32x2(l2[(e >> 1) & 1], f32x2(p0, p1));
        pw[e >> 1] = pack_bf16x2(p0, p1);
    }
    tmem_st16(tP + 16 * c, pw);
    const float2 s2 = split_f32x2(add_f32x2(l2[0], l2[1]));
    l += s2.x + s2.y;
}

__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// v[e] += a[e], read by all lanes alike
template <int N>
__device__ __forceinline__ void add_a(float* v, const float* a) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 av = *reinterpret_cast<const float4*>(a + e);
        v[e] += av.x;
        v[e + 1] += av.y;
        v[e + 2] += av.z;
        v[e + 3] += av.w;
    }
}

// A block of a warp whose rows are all replaced and of one head, their stretches of
// r at most NEAR_SPAN apart (a chunk's tokens, sequences of like lengths): one
// stretch serves them all, copied a block ahead.  off: this row's against the
// first's.  primed: the block's copies are under way; next: there is a block after
// it, and its copies are started.  masked: not every row sees every key (vis, and
// boxes without a page in `bad`); what lies before the array or past the last key is
// then not copied.  Returns (m, l).
__device__ __forceinline__ void near_copy(int k0) {
    const WarpRows& w = warp_rows();
    const int lane = threadIdx.x & 31;
    const uint32_t buf = smem_addr(staging()) + (uint32_t)((k0 / BN) & 1) * NEAR_BUF * 4;
    const float* r = w.r - k0;
#pragma unroll
    for (int i = 0; i < 4; ++i) copy4(buf + (32 * i + lane) * 4, w.a + min(k0 + 32 * i + lane, w.last));
    // from the boundary at or before the lowest row's last key to the highest row's first key
    const int edge = w.low_edge, stop = w.low + w.span + 1;
    for (int at = edge + 4 * lane; at < stop; at += 128) {
        const int rel = at - k0;  // (sums of these stay within 31 bits: positions come near that far)
        const bool in = rel >= -w.before;
        const int bytes = in ? min(4, w.room - max(rel, -4)) * 4 : 0;  // (the last may reach past the array)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(buf + (128 + at - edge) * 4),
                     "l"(in ? r + at : w.r0), "r"(bytes));
    }
    copies_commit();
}
__device__ __noinline__ float2 near_block(float m, float l, bool primed, bool next, bool first, int off, uint32_t tmem, int k0,
                                          bool masked, int vis, uint32_t bad, int lb) {
    if (!primed) near_copy(k0);
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncwarp();
    if (next) near_copy(k0 - BN);
    const float *a = staging() + ((k0 / BN) & 1) * NEAR_BUF, *r = a + 128 + off - warp_rows().low_edge;
#pragma unroll 1
    for (int c = 3; c >= 0; --c) {
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = r[-32 * c - e];
        add_a<32>(v, a + 32 * c);
        if (masked) {
            const int left = vis - k0 - 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e >= left || ((bad >> ((32 * c + e) >> lb)) & 1u)) v[e] = kNegInf;
        }
        chunk_out(v, c, first, kLog2e, m, l, tmem, true);
    }
    __syncwarp();  // the buffer has been read
    return make_float2(m, l);
}

// The same where they lie anywhere: 16 keys at a time, three under way.  The 16
// bytes i = 0..3 that a lane copies are of the rows 8 i + lane / 4, the fifth of its
// own row.  off: this row's stretch against the warp's first, edge: the 16-byte
// boundary at or before its 16 entries from local key 15 down to key 0.
__device__ __forceinline__ void far_copy(int edge, int key) {  // the 16 keys from `key` on
    const WarpRows& w = warp_rows();
    const int lane = threadIdx.x & 31;
    const uint32_t buf = smem_addr(staging()) + (uint32_t)((key >> 4) % FAR_BUFS) * FAR_BUF * 4;
    const float *r = w.r - key, *a = w.a + key;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        const uint32_t dst = buf + (i < 4 ? (8 * i + (lane >> 2)) * FAR_PITCH + 4 * (lane & 3) : lane * FAR_PITCH + 16) * 4;
        const int src = i < 4 ? __shfl_sync(~0u, edge, 8 * i + (lane >> 2)) + 4 * (lane & 3) : edge + 16;
        // the fifth may end past the array's last float, or begin there (a stretch that starts on a boundary needs none)
        const int bytes = i < 4 ? 16 : min(4, max(0, w.room - max(src - key, -4))) * 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(r + src), "r"(bytes));
    }
    if (lane < 16) copy4(buf + (FAR_A + lane) * 4, a + lane);
    copies_commit();
}
__device__ __noinline__ float2 far_block(float m, float l, bool primed, bool next, bool first, int off, int edge,
                                         uint32_t tmem, int k0) {
    const int lane = threadIdx.x & 31;
    if (!primed) {
#pragma unroll 1
        for (int n = 7; n > 7 - FAR_BUFS; --n) far_copy(edge, k0 + 16 * n);
    }
    const float* rows = staging() + lane * FAR_PITCH + (off - edge);
#pragma unroll 1
    for (int c = 3; c >= 0; --c) {
        float v[32];
#pragma unroll
        for (int h = 1; h >= 0; --h) {
            const int n = 2 * c + h, key = k0 + 16 * n, buf = ((key >> 4) % FAR_BUFS) * FAR_BUF;
            asm volatile("cp.async.wait_group %0;\n" ::"n"(FAR_BUFS - 1) : "memory");
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[16 * h + e] = rows[buf - e];
            add_a<16>(v + 16 * h, staging() + buf + FAR_A);
            __syncwarp();
            if (n >= FAR_BUFS || next) far_copy(edge, key - 16 * FAR_BUFS);
            else copies_commit();
        }
        chunk_out(v, c, first, kLog2e, m, l, tmem, true);
    }
    return make_float2(m, l);
}

// A block of a warp that is none of these: several heads' rows, both kinds, or keys
// that a row does not see.  32 keys at a time, in a loop (a cold unrolled
// copy would cost more to fetch than to run).  Returns (m, l).
__device__ __noinline__ float2 mixed_block(float m, float l, float unit, int vis, bool first, uint32_t tmem, int ni, int k0,
                                           uint32_t bad) {
    const WarpRows& w = warp_rows();
    const int lane = threadIdx.x & 31, len = item_of(ni).len, lb = item_of(ni).lb;
    const bool keyed = item_of(ni).keyed;
    const uint32_t reps = w.reps;
    const int vis_last = max(vis, 1) - 1;
    float* pat = staging();
    const int2* rows = reinterpret_cast<const int2*>(smem_base() + SM_ROW) + quarter_of() * 32;
#pragma unroll 1
    for (int c = 3; c >= 0; --c) {
        uint32_t raw[32];
        float v[32];
        if (keyed) {
            tmem_ld32(tmem + 32 * c, raw);
            tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
        if (reps) {
            const int key = k0 + 32 * c + lane;
            const bool one = w.one_head;
            const float av = one ? __ldg(w.a + min(key, len - 1)) : 0.f;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
                if (!((reps >> r0) & 0xffu)) continue;
                float x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {  // (a row that looks nothing up reads entry 0)
                    const int j = min(key, __shfl_sync(~0u, vis_last, r0 + u));
                    const int2 at = rows[r0 + u];
                    const bool read = (reps >> (r0 + u)) & 1u;
                    const long long ph = (long long)at.x * w.pattern_len;
                    x[u] = (one ? av : __ldg(read ? w.a0 + ph + j : w.a)) + __ldg(read ? w.r0 + ph + at.y - j : w.r);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) pat[(r0 + u) * PAT_PITCH + lane] = x[u];
            }
            __syncwarp();
            if ((reps >> lane) & 1u) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = pat[lane * PAT_PITCH + e];
            }
            __syncwarp();
        }
        const int left = vis - k0 - 32 * c;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e >= left || ((bad >> ((32 * c + e) >> lb)) & 1u)) v[e] = kNegInf;
        chunk_out(v, c, first, unit, m, l, tmem, !keyed);
    }
    return make_float2(m, l);
}

// The barriers and per-load words, by the offsets that the kernel lays them out at.
constexpr uint32_t BAR_KF = SM_BAR, BAR_KE = BAR_KF + 8 * NST;      // [NST] K stage full, free (S MMA done)
constexpr uint32_t BAR_VF = BAR_KE + 8 * NST, BAR_VE = BAR_VF + 8 * NST;  // [NST] V stage full, free (P V MMA done)
constexpr uint32_t BAR_ITEM = BAR_VE + 8 * NST, BAR_TAKEN = BAR_ITEM + 16;  // [2] item slot full, free (MMA and row warps)
constexpr uint32_t BAR_Q = BAR_TAKEN + 16;                          // queries in place (4 warp arrivals)
constexpr uint32_t BAR_S = BAR_Q + 8;                               // S ready
constexpr uint32_t BAR_SF = BAR_S + 8;                              // S copied out by the rows (4 warp arrivals)
constexpr uint32_t BAR_P = BAR_SF + 8;                              // P written (4 warp arrivals)
constexpr uint32_t BAR_O = BAR_P + 8;                               // P V done
static_assert(BAR_O + 8 <= SM_ITEM, "barrier area");
constexpr uint32_t SM_KMETA = SM_MISC + 8, SM_VMETA = SM_MISC + 24;

// Block i of item ni has landed, with its scores where it has some; boxes without a
// page in `bad`.  nk, nv: S and P V products before it.
__device__ __forceinline__ bool block_arrived(bool keyed, int nk, int nv, uint32_t& bad) {
    const uint32_t sbase = smem_addr(smem_base());
    bool ok;
    if (keyed) {
        // (not the K stage's barrier: it may be a fill ahead by now; what the producer wrote before the load was
        // seen by the MMA warp before it issued S)
        ok = row_wait(sbase + BAR_S, nk & 1);
        bad = ld_shared_u32(sbase + SM_KMETA + 4 * (nk & 3));
    } else {
        ok = row_wait(sbase + BAR_VF + 8 * (nv & 1), (nv >> 1) & 1);
        bad = ld_shared_u32(sbase + SM_VMETA + 4 * (nv & 3));
    }
    tc_fence_after();
    return ok;
}
// P V of the block before has read P and added to O (an item's first: waited for by the item before).
__device__ __forceinline__ bool p_free(bool first, int nv) {
    if (first) return true;
    const bool ok = row_wait(smem_addr(smem_base()) + BAR_O, (nv - 1) & 1);
    tc_fence_after();
    return ok;
}
__device__ __forceinline__ void s_copied(bool keyed) {  // the MMA warp may now overwrite S
    tc_fence_before();
    if (keyed) mbar_arrive_warp(smem_addr(smem_base()) + BAR_SF);
}
__device__ __forceinline__ void hand_over() {
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive_warp(smem_addr(smem_base()) + BAR_P);
}
// Slots without a token may hold a NaN, and 0 times that is one: their V rows become
// zeros before P V reads them.
__device__ __forceinline__ bool clear_dead(int ni, int nv, int k0, uint32_t bad) {
    const int len = item_of(ni).len;
    if (k0 + BN <= len && !bad) return true;
    const uint32_t sbase = smem_addr(smem_base());
    const int row = quarter_of() * 32 + (threadIdx.x & 31);
    const bool ok = row_wait(sbase + BAR_VF + 8 * (nv & 1), (nv >> 1) & 1);
    if (k0 + row >= len || ((bad >> (row >> item_of(ni).lb)) & 1u)) {
#pragma unroll
        for (int c = 0; c < 8; ++c) st_shared_v4(sbase + SM_V + (nv & 1) * TILE_BYTES + row * 128 + 16 * c, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    return ok;
}

// The blocks of a warp without rows that look scores up.  tmem: of this warp's lanes.
__device__ __noinline__ RowResult plain_rows(float unit, int vis, uint32_t tmem, int ni, int nk, int nv) {
    float m = kNegInf, l = 0.f;
    const int nt = item_of(ni).nt, vmin = warp_rows().vmin;
    const bool keyed = item_of(ni).keyed;
    int k0 = (item_of(ni).t0 + nt) * BN;
    for (int i = 0; i < nt; ++i, ++nk, ++nv) {
        k0 -= BN;
        uint32_t bad;
        if (!block_arrived(keyed, nk, nv, bad)) return {m, l, 0};
        if (k0 + BN > vmin || bad) {
            if (!p_free(i == 0, nv)) return {m, l, 0};
            const float2 ml = mixed_block(m, l, unit, vis, i == 0, tmem, ni, k0, bad);
            m = ml.x;
            l = ml.y;
            s_copied(keyed);
            if (!clear_dead(ni, nv, k0, bad)) return {m, l, 0};
        } else {
            // The scores of keys 64..127 stay in registers, the others are loaded again for their exponentials: all
            // 128 with what the exponentials need would not fit 168 registers.
            uint32_t v[2][32], w[2][32];
            tmem_ld32(tmem, w[0]);
            tmem_ld32(tmem + 32, w[1]);
            tmem_ld32(tmem + 64, v[0]);
            tmem_ld32(tmem + 96, v[1]);
            tmem_wait_ld();
            loaded(w[0]);
            loaded(w[1]);
            loaded(v[0]);
            loaded(v[1]);
            float ma[2] = {kNegInf, kNegInf}, mb[2] = {kNegInf, kNegInf};
            quarter_max(w[0], ma);
            quarter_max(w[1], mb);
            quarter_max(v[0], ma);
            quarter_max(v[1], mb);
            const float mx = fmaxf(fmaxf(ma[0], ma[1]), fmaxf(mb[0], mb[1]));
            float f = 1.f;
            if ((mx - m) * unit > 8.f) {
                f = ex2((m - mx) * unit);
                l *= f;
                m = mx;
            }
            if (!p_free(i == 0, nv)) return {m, l, 0};
            const float nm = m == kNegInf ? 0.f : -m * unit;
            const uint64_t unit2 = f32x2(unit, unit), nm2 = f32x2(nm, nm);
            uint64_t l2[4] = {0, 0, 0, 0};
            tmem_ld32(tmem, w[0]);
            exp_quarter<2>(v[0], unit2, nm2, l2, tmem + TP_COL);
            tmem_ld32(tmem + 32, w[1]);
            exp_quarter<3>(v[1], unit2, nm2, l2, tmem + TP_COL);
            tmem_wait_ld();
            loaded(w[0]);
            loaded(w[1]);
            s_copied(keyed);
            exp_quarter<0>(w[0], unit2, nm2, l2, tmem + TP_COL);
            exp_quarter<1>(w[1], unit2, nm2, l2, tmem + TP_COL);
            const float2 s2 = split_f32x2(add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3])));
            l += s2.x + s2.y;
            if (i > 0 && __any_sync(~0u, f != 1.f)) rescale_o(tmem, f, false);
        }
        hand_over();
    }
    return {m, l, 1};
}

// The blocks of a warp without a row that has a token, in an item without keys: there is no S to read, and no one reads
// what its rows come to.
__device__ __noinline__ RowResult idle_rows(int ni, int nk, int nv) {
    const int nt = item_of(ni).nt;
    int k0 = (item_of(ni).t0 + nt) * BN;
    for (int i = 0; i < nt; ++i, ++nv) {
        k0 -= BN;
        uint32_t bad;
        if (!block_arrived(false, nk, nv, bad) || !p_free(i == 0, nv) || !clear_dead(ni, nv, k0, bad)) return {kNegInf, 0.f, 0};
        hand_over();
    }
    return {kNegInf, 0.f, 1};
}

// The blocks of a warp with replaced rows (off, edge: see near_block and far_block).
__device__ __noinline__ RowResult pattern_rows(float unit, int vis, uint32_t tmem, int ni, int nk, int nv, int off, int edge) {
    float m = kNegInf, l = 0.f;
    bool primed = false, ok = true;
    const int nt = item_of(ni).nt;
    const bool keyed = item_of(ni).keyed;
    int k0 = (item_of(ni).t0 + nt) * BN;
    for (int i = 0; ok && i < nt; ++i, ++nk, ++nv) {
        k0 -= BN;
        uint32_t bad;
        ok = block_arrived(keyed, nk, nv, bad) && p_free(i == 0, nv);
        if (!ok) break;
        const WarpRows& w = warp_rows();
        float2 ml;
        const bool next = i + 1 < nt, masked = k0 + BN > w.vmin || bad;
        if (w.pure && w.span <= NEAR_SPAN) {
            ml = near_block(m, l, primed, next, i == 0, off, tmem, k0, masked, vis, bad, item_of(ni).lb);
            primed = next;
        } else if (w.pure && !masked) {
            ml = far_block(m, l, primed, next, i == 0, off, edge, tmem, k0);
            primed = next;
        } else {
            if (primed) {  // copies begun for this block: its staging area is wanted
                asm volatile("cp.async.wait_all;\n" ::: "memory");
                __syncwarp();
                primed = false;
            }
            ml = mixed_block(m, l, unit, vis, i == 0, tmem, ni, k0, bad);
        }
        m = ml.x;
        l = ml.y;
        s_copied(keyed);
        ok = clear_dead(ni, nv, k0, bad);
        hand_over();
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncwarp();
    return {m, l, ok};
}

template <bool PREFIX>
__global__ void __launch_bounds__(NTHREADS, 2)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ PagedParams p) {
    uint8_t* const smem = smem_base();
    const uint32_t sbase = smem_addr(smem);
    const uint32_t bar_kf = sbase + BAR_KF, bar_ke = sbase + BAR_KE, bar_vf = sbase + BAR_VF, bar_ve = sbase + BAR_VE;
    const uint32_t bar_item = sbase + BAR_ITEM, bar_taken = sbase + BAR_TAKEN, bar_q = sbase + BAR_Q, bar_s = sbase + BAR_S;
    const uint32_t bar_sf = sbase + BAR_SF, bar_p = sbase + BAR_P, bar_o = sbase + BAR_O;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + SM_MISC);
    volatile uint32_t *kmeta = reinterpret_cast<uint32_t*>(smem + SM_KMETA),
                      *vmeta = reinterpret_cast<uint32_t*>(smem + SM_VMETA);
    TcPiece* items = reinterpret_cast<TcPiece*>(smem + SM_ITEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (sbase & 1023u) {  // the swizzled tiles need what the declaration asks for
        griddep_wait();
        if (threadIdx.x == 0) {
            p.shared[blockIdx.x].pieces = 0;
            report(p.err, 0x504);
        }
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar_kf + 8 * s, 1);
            mbar_init(bar_ke + 8 * s, 1);
            mbar_init(bar_vf + 8 * s, 1);
            mbar_init(bar_ve + 8 * s, 1);
            mbar_init(bar_item + 8 * s, 1);
            mbar_init(bar_taken + 8 * s, 5);
        }
        mbar_init(bar_q, 4);
        mbar_init(bar_s, 1);
        mbar_init(bar_sf, 4);
        mbar_init(bar_p, 4);
        mbar_init(bar_o, 1);
        *reinterpret_cast<long long*>(smem + SM_LIMIT) = p.wait_limit;
        fence_mbar_init();
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_holder), TMEM_COLS);
        tmem_relinquish();
    }
    // The launch may overlap the one before it on the stream, whose results are awaited before any is read.  After a
    // prefix's launch, which has waited for what came before both, only its results are (see below).
    if (PREFIX || !p.part) griddep_wait();
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------ producer
        const int lp = p.log_page, lb = min(lp, 7);  // page and box rows
        const uint32_t box_bytes = 128u << lb;
        const int boxes = BN >> lb;
        AxisWalk<TcAxis, PREFIX> walk(p, blockIdx.x, gridDim.x);
        int nk = 0, nv = 0;  // K and V loads so far
        bool ok = true;
        for (int ni = 0; ok; ++ni) {
            // The rows stop for a prefix's launch before they leave their first item, for as long as it takes: past that
            // item no bounded wait for them (or, by way of them, for the MMA warp) begins before it has ended.
            if (!PREFIX && p.part && ni == 1) griddep_wait();
            Stretch w;
            TcPiece x;
            x.nt = -1;
            if (walk.next(w)) {
                x.b = w.b;
                x.e = w.e;
                x.n_rows = w.n_rows;
                x.rb = w.rb;
                x.len = w.len;
                x.t0 = w.t0;
                x.pieces = w.pieces;
                x.c_first = w.c_first;
                x.lb = lb;
                int most = 0, ordinary = 0;
#pragma unroll 1
                for (int r = lane; r < BM; r += 32) {
                    const RowInfo row = row_info<PREFIX>(p, w.b, w.e, w.len, w.n_rows, w.rb * BM + r);
                    most = max(most, row.vis);
                    ordinary |= row.out >= 0 && !row.replaced;
                }
                most = __reduce_max_sync(~0u, most);
                x.keyed = __any_sync(~0u, ordinary);
                x.nt = max(0, min(w.t1, (most + BN - 1) / BN) - w.t0);
            }
            const int slot = ni & 1;
            ok = mbar_wait_warp(bar_taken + 8 * slot, ((ni >> 1) & 1) ^ 1, p.wait_limit);
            if (!ok) break;
            if (lane == 0) {
                items[slot] = x;
                mbar_arrive(bar_item + 8 * slot);
            }
            if (x.nt < 0) break;
            const int32_t* table = p.table + (size_t)x.b * p.table_stride;
            const int g = p.e_g[w.e];
            // pages of this lane's boxes of the last two blocks looked up (block i in entry i & 1)
            int pages[2] = {-1, -1}, looked = 0;
            auto load = [&](int i, bool keys) {
                const int key = (x.t0 + x.nt - 1 - i) * BN + (lane << lb);
                const bool need = lane < boxes && key < x.len;
                if (i >= looked) {
                    const int page = need ? __ldg(table + (key >> lp)) : -1;
                    if (i & 1) pages[1] = page;
                    else pages[0] = page;
                    looked = i + 1;
                }
                const int page = (i & 1) ? pages[1] : pages[0];
                const int at = keys ? nk++ : nv++, s = at & 1;
                const uint32_t full = (keys ? bar_kf : bar_vf) + 8 * s, empty = (keys ? bar_ke : bar_ve) + 8 * s;
                const bool good = need && page >= 0 && page < p.num_pages;
                const uint32_t bad = __ballot_sync(~0u, lane < boxes && !good);
                const int loads = __popc(__ballot_sync(~0u, good));
                if (!mbar_wait_warp(empty, ((at >> 1) & 1) ^ 1, p.wait_limit)) {
                    --(keys ? nk : nv);
                    return false;
                }
                if (lane == 0) {
                    // four entries: the rows may still be two loads behind the stage that is being filled
                    (keys ? kmeta : vmeta)[at & 3] = bad;
                    mbar_expect_tx(full, loads * box_bytes);
                }
                __syncwarp();
                if (good)
                    tma_load_4d(sbase + (keys ? SM_K : SM_V) + s * TILE_BYTES + lane * box_bytes, keys ? &tmK : &tmV, full, 0,
                                key & ((1 << lp) - 1), g, page);
                return true;
            };
            // K_{i+1} before V_i, whose stage frees later: S runs ahead of P V
            if (x.keyed && x.nt > 0) ok = load(0, true);
            for (int i = 0; ok && i < x.nt; ++i) {
                if (x.keyed && i + 1 < x.nt) ok = load(i + 1, true);
                if (ok) ok = load(i, false);
            }
        }
        if (!ok && lane == 0) report(p.err, 0x501);
        if (lane == 0) {  // the loads in flight land before the shared memory is let go, whether anyone still wants them or not
            for (int i = max(0, nk - 2); i < nk; ++i) mbar_wait(bar_kf + 8 * (i & 1), (i >> 1) & 1, kDrainLimit);
            for (int i = max(0, nv - 2); i < nv; ++i) mbar_wait(bar_vf + 8 * (i & 1), (i >> 1) & 1, kDrainLimit);
        }
        // A grid in which none has waited may end before the one ahead of it, and the next would start too soon.
        if (!PREFIX && p.part) griddep_wait();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (one elected lane, as in the layer's kernels)
        const uint32_t idS = idesc_bf16(128, 128, 0, 0);  // Q (K-major) x K (K-major)
        const uint32_t idO = idesc_bf16(128, 64, 0, 1);   // P (TMEM) x V (MN-major)
        const uint32_t idSum = idesc_bf16(128, 16, 0, 0); // P (TMEM) x ones (K-major)
        constexpr uint64_t kStage = TILE_BYTES >> 4;
        const uint64_t dQ = sw128_desc(sbase + SM_Q), dK0 = sw128_desc(sbase + SM_K), dV0 = sw128_desc(sbase + SM_V);
        int nk = 0, nv = 0, nq = 0;  // S and P V products issued, items with queries
        bool ok = true;
        for (int ni = 0; ok; ++ni) {
            if (!PREFIX && p.part && ni == 1) griddep_wait();  // (as the producer does)
            ok = mbar_wait_warp(bar_item + 8 * (ni & 1), (ni >> 1) & 1, p.wait_limit);
            if (!ok) break;
            const int nt = items[ni & 1].nt;
            const bool keyed = items[ni & 1].keyed && nt > 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_taken + 8 * (ni & 1));
            if (nt < 0) break;
            auto issue_s = [&] {
                const int s = nk & 1;
                // the rows have copied the S before (an item's first: that item's last)
                if (nk > 0 && !mbar_wait_warp(bar_sf, (nk - 1) & 1, p.wait_limit)) return false;
                if (!mbar_wait_warp(bar_kf + 8 * s, (nk >> 1) & 1, p.wait_limit)) return false;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem, dQ + 2 * k, dK0 + s * kStage + 2 * k, idS, k > 0 ? 1u : 0u);
                    mma_commit(bar_s);
                    mma_commit(bar_ke + 8 * s);
                }
                __syncwarp();
                ++nk;
                return true;
            };
            if (keyed) {
                ok = mbar_wait_warp(bar_q, nq & 1, p.wait_limit) && issue_s();
                ++nq;
            }
            for (int i = 0; ok && i < nt; ++i) {
                if (keyed && i + 1 < nt) ok = issue_s();
                const int s = nv & 1;
                ok = ok && mbar_wait_warp(bar_vf + 8 * s, (nv >> 1) & 1, p.wait_limit) && mbar_wait_warp(bar_p, nv & 1, p.wait_limit);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + TO_COL, tmem + TP_COL + 8 * k, dV0 + s * kStage + 128 * k, idO, (i > 0 || k > 0) ? 1u : 0u);
                    if (!keyed) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(tmem + TSUM_COL, tmem + TP_COL + 8 * k, dQ + 2 * (k & 3), idSum, (i > 0 || k > 0) ? 1u : 0u);
                    }
                    mma_commit(bar_o);
                    mma_commit(bar_ve + 8 * s);
                }
                __syncwarp();
                ++nv;
            }
        }
        if (!ok && lane == 0) report(p.err, 0x502);
        // the products in flight end before the operands and TMEM are let go, whether the rows still want them or not
        if (lane == 0 && nk > 0) mbar_wait(bar_s, (nk - 1) & 1, kDrainLimit);
        if (lane == 0 && nv > 0) mbar_wait(bar_o, (nv - 1) & 1, kDrainLimit);
    } else {
        // ------------------------------------------------ row threads
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t tmem_rows = tmem + ((uint32_t)(quarter * 32) << 16), tO = tmem_rows + TO_COL;
        int nk = 0, nv = 0;  // S and P V products so far
        bool ok = true, waited = false;
        if (row == 0) p.shared[blockIdx.x].pieces = 0;  // until there is one
        for (int ni = 0; ok; ++ni) {
            ok = mbar_wait_warp(bar_item + 8 * (ni & 1), (ni >> 1) & 1, p.wait_limit);
            if (!ok) break;
            const TcPiece x = items[ni & 1];
            if (x.nt < 0) break;
            const RowInfo info = row_info<PREFIX>(p, x.b, x.e, x.len, x.n_rows, x.rb * BM + row);
            const bool keyed = x.keyed && x.nt > 0;
            if (keyed) {  // the row's queries (zeros where there are none) in the 128-byte swizzle
                const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)max(info.out, 0) * kHeadDim);
                const bool read = info.out >= 0 && !info.replaced;
                uint4 w[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) w[c] = read ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared_v4(sbase + SM_Q + row * 128 + ((c ^ (row & 7)) << 4), w[c].x, w[c].y, w[c].z, w[c].w);
                fence_proxy_async_smem();
                mbar_arrive_warp(bar_q);
            } else if (x.nt > 0) {  // ones, which the first P V waits for along with P
                const uint32_t one2 = 0x3f803f80u;
                st_shared_v4(sbase + SM_Q + row * 16, one2, one2, one2, one2);
                fence_proxy_async_smem();
            }
            const bool rep = info.out >= 0 && info.replaced;
            const uint32_t reps = __ballot_sync(~0u, rep && info.vis > 0);
            const float unit = rep ? kLog2e : 0.125f * kLog2e;  // log2(e) per unit of the row's scores (dot products: 1/8)
            const bool looks = (reps >> lane) & 1u;
            const int from = reps ? __ffs(reps) - 1 : 0;
            const long long a_first = __shfl_sync(~0u, info.a0, from), r_first = __shfl_sync(~0u, info.r0, from);
            const bool one_head = __all_sync(~0u, !looks || info.a0 == a_first);
            // rows without a token ride along on the first one's stretch
            const int off = looks && one_head ? (int)(info.r0 - r_first) : 0;
            const int low = __reduce_min_sync(~0u, off), span = __reduce_max_sync(~0u, off) - low;
            const int pure = reps && one_head && __all_sync(~0u, info.out < 0 || looks);
            // (a warp without rows still clears its share of the dead slots)
            const int vmin = __reduce_min_sync(~0u, info.out >= 0 ? info.vis : x.len);
            const int head = max(info.replaced - 1, 0);
            reinterpret_cast<int2*>(smem + SM_ROW)[row] = make_int2(head, (int)(info.r0 - (long long)head * p.pattern_len));
            if (lane == 0) {
                WarpRows& w = reinterpret_cast<WarpRows*>(smem + SM_WARP)[quarter];
                w.a = p.a + a_first;
                w.r = p.r + r_first;
                w.a0 = p.a + (PREFIX ? 0 : p.prefix_len);
                w.r0 = p.r;
                w.pattern_len = p.pattern_len;
                w.reps = reps;
                w.one_head = one_head;
                w.pure = pure;
                w.low = low;
                w.low_edge = (int)(((r_first + low - 127) & ~3ll) - r_first);
                w.span = span;
                w.room = (int)min((long long)p.H * p.pattern_len - r_first, (long long)INT_MAX - 8);
                w.before = (int)min(r_first, (long long)INT_MAX);
                w.last = max(x.len, 1) - 1;
                w.vmin = vmin;
            }
            __syncwarp();
            RowResult res;  // running maximum (in the row's units), sum
            if (!reps && !x.keyed && vmin >= x.len) {
                res = idle_rows(ni, nk, nv);
            } else if (!reps) {
                res = plain_rows(unit, info.vis, tmem_rows, ni, nk, nv);
            } else {
                const int edge = (int)(((r_first + off - 15) & ~3ll) - r_first);
                res = pattern_rows(unit, info.vis, tmem_rows, ni, nk, nv, off, edge);
            }
            ok = res.ok;
            nv += x.nt;
            if (keyed) nk += x.nt;
            const float m = rep ? res.m : 0.125f * res.m, l = res.l;
            if (ok && x.nt > 0) ok = mbar_wait_warp(bar_o, (nv - 1) & 1, p.wait_limit);
            tc_fence_after();
            if (!ok) break;
            if (!PREFIX && p.part && !waited) {
                griddep_wait();
                waited = true;
            }
            // ---- the rows out, or a piece of them
            // A replaced row is divided by the sum of its rounded weights (see the kernel for few rows), an ordinary one, as in
            // the layer's forward, by that of the weights: a column of sums has no room beside S.
            float f = 1.f;
            if (!keyed && x.nt > 0) {
                f = __uint_as_float(tmem_ld1(tmem_rows + TSUM_COL));
                tmem_wait_ld();
                f = by_rounded(l, f);
            }
            constexpr int SLOT = BM * (kHeadDim + 2);
            float* slot = p.slots + ((size_t)blockIdx.x * 2 + (x.t0 == 0)) * SLOT;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t ov[32];
                if (x.nt > 0) {
                    tmem_ld32(tO + 32 * c, ov);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 o = make_float4(__uint_as_float(ov[e]) * f, __uint_as_float(ov[e + 1]) * f,
                                                 __uint_as_float(ov[e + 2]) * f, __uint_as_float(ov[e + 3]) * f);
                    if (x.pieces > 1) __stcg(reinterpret_cast<float4*>(slot + row * kHeadDim + 32 * c + e), o);
                    else finish_row<PREFIX>(p, info, 32 * c + e, o, m, l);
                }
            }
            tc_fence_before();  // (O is read before the next item's first P V, which waits for this thread's P)
            if (x.pieces > 1) {
                __stcg(slot + BM * kHeadDim + row, m);
                __stcg(slot + BM * (kHeadDim + 1) + row, l);
            }
            if (row == 0 && x.pieces > 1 && x.c_first == blockIdx.x)
                p.shared[blockIdx.x] = SharedItem{x.pieces, x.b, x.e, x.rb, x.len, x.n_rows, {0, 0}};
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_taken + 8 * (ni & 1));
        }
        if (!ok) {
            if (lane == 0) report(p.err, 0x503);
            tmem_wait_st();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the pieces of the items that several CTAs shared, in key order: eight
// blocks per CTA of the launch before, sixteen threads per row.
template <bool PREFIX>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p) {
    griddep_launch_dependents();  // (what comes after reads nothing of this call's before it waits in turn)
    griddep_wait();
    constexpr int SLOT = BM * (kHeadDim + 2);
    const int first = blockIdx.x >> 3, in_block = (blockIdx.x & 7) * 16 + (threadIdx.x >> 4), c = (threadIdx.x & 15) * 4;
    const SharedItem it = p.shared[first];
    if (it.pieces == 0) return;
    const RowInfo x = row_info<PREFIX>(p, it.b, it.e, it.len, it.n_rows, it.rb * BM + in_block);
    if (x.out < 0) return;
    auto slot_of = [&](int k) { return p.slots + ((size_t)(first + k) * 2 + (k == 0)) * SLOT; };
    float mm = kNegInf;
#pragma unroll 8
    for (int k = 0; k < it.pieces; ++k) mm = fmaxf(mm, slot_of(k)[BM * kHeadDim + in_block]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 8
    for (int k = 0; k < it.pieces; ++k) {
        const float* sl = slot_of(k);
        const float f = weight(sl[BM * kHeadDim + in_block], mm);
        const float4 v = *reinterpret_cast<const float4*>(sl + in_block * kHeadDim + c);
        o = make_float4(o.x + f * v.x, o.y + f * v.y, o.z + f * v.z, o.w + f * v.w);
        l += f * sl[BM * (kHeadDim + 1) + in_block];
    }
    finish_row<PREFIX>(p, x, c, o, mm, l);
}

template <bool PREFIX>
cudaError_t launch(const saf_paged_kv& kv, PagedParams& p, cudaStream_t stream) {
    CUtensorMap mk, mv;
    if (!make_tmap_pages(kv, true, BN, &mk) || !make_tmap_pages(kv, false, BN, &mv)) return cudaErrorNotSupported;
    // as many heads to an entry as a block has room for; replaced heads begin with a warp (see near_block)
    const int rows = PREFIX ? p.B * p.T : p.T;
    p.pad = 32;
    auto heads = [&](int n) { return std::max(1, std::min(p.G, BM / n)); };
    make_entries(p, heads(rows), heads(padded(rows, p.pad)), true);
    p.by_BT_pad = divisor(padded(p.B * p.T, p.pad));
    p.block_rows = BM;
    p.by_block = divisor(BM);
    if (!axis_fits<TcAxis>(p, PREFIX)) return cudaErrorNotSupported;
    const int smem = SM_TOTAL;
    cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)paged_grid());
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int kid = PREFIX ? KID_PAGED_PREFIX_TC : KID_PAGED_TC;
    launch_begin(kid, stream);
    e = cudaLaunchKernelEx(&cfg, paged_tc_kernel<PREFIX>, mk, mv, p);
    launch_end(kid, stream);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(paged_grid() * 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    launch_begin(KID_PAGED_JOIN, stream);
    e = cudaLaunchKernelEx(&cfg, paged_join_kernel<PREFIX>, p);
    launch_end(KID_PAGED_JOIN, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const saf_paged_kv& kv, PagedParams& p, bool prefix, cudaStream_t stream) {
    return prefix ? launch<true>(kv, p, stream) : launch<false>(kv, p, stream);
}

}  // namespace saf
