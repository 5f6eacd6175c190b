// Appending new tokens to the paged key/value cache, with the rotation of
// queries and keys by position, and the table of angles.
//
// A row (one head of one token, 64 bf16) is eight 16-byte chunks, one per
// lane of an eight-lane group.  Rotated pairs (i, i + rot/2) lie rot/16 chunks
// apart, in another lane of the group (exchanged by shuffles); interleaved
// pairs (2i, 2i+1) lie inside a chunk.  Rows q, k, v of a token form one axis of
// H + 2 H_kv rows.
//
// Long appends: 8 x 4096 tokens of 12 heads (3 replaced), with the rotated keys beside
// the cache, 290 MB in 59 us, 4.9 TB/s (44 us at a plain copy's rate): HBM half busy by
// its counters, issue slots two thirds, 26 warps an SM that each wait for four rows
// of 128 bytes and end.  A step's few rows take 2 to 5 us, a launch's latency.
#include <algorithm>

#include "saf_paged.cuh"

namespace saf {
namespace {

__global__ void rope_table_kernel(float* table, int max_pos, int rot_dim, double base) {
    const int half = rot_dim >> 1;
    const int64_t n = (int64_t)max_pos * half;
    for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
        const int i = (int)(x % half);
        const int64_t p = x / half;
        double s, c;
        sincos((double)p * pow(base, -2.0 * i / rot_dim), &s, &c);
        table[p * rot_dim + i] = (float)c;
        table[p * rot_dim + half + i] = (float)s;
    }
}

// x cos + y sin of a pair, rounded to bf16 (the products and their sum in fp32).
__device__ __forceinline__ uint32_t turn(uint32_t x, uint32_t y, uint64_t cs, uint64_t sn) {
    const float2 v = tc::split_f32x2(tc::fma_f32x2(pair_of(x), cs, tc::mul_f32x2(pair_of(y), sn)));
    return tc::pack_bf16x2(v.x, v.y);
}

// U rows of one token per eight lanes: their loads are in flight together, and the
// token's position, page and angles are looked up once.  Neighbouring groups of
// lanes take the same rows of neighbouring tokens, eight at a time: the outputs of a
// head are then written 1 KB at a stretch.
template <int U>
__global__ void __launch_bounds__(256, U == 1 ? 6 : 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
    tc::griddep_wait();  // (the launch may overlap the one before it on the stream)
    tc::griddep_launch_dependents();
    const int unit = blockIdx.x * 4 + (threadIdx.x >> 6), c = threadIdx.x & 7;
    const int tok8 = p.by_units.div(unit), r0 = (unit - tok8 * p.units) * U;
    const int tok = tok8 * 8 + ((threadIdx.x >> 3) & 7);
    const int b = p.by_T.div(tok), t = tok - b * p.T;
    // the lanes of a group agree on every row and branch below, and the shuffles name the group's lanes alone
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    if (b >= p.B) return;
    const int n = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
    const long long pos = (long long)p.seq_lens[b] - n + t;
    if (t >= n || pos < 0 || pos >= p.max_len) return;
    // rows [0, H) are q, [H, H + H_kv) k, then v; skipped ones become row -1
    const int Hkv = p.kv.H_kv;
    uint4 w[U];
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int rr = r0 + u, h = rr < p.H ? rr : rr - p.H;
        const bool skip = rr >= p.H + 2 * Hkv || (rr < p.H ? p.q == nullptr || p.replaced.get(h) : h < Hkv && p.keyless.get(h));
        row[u] = skip ? -1 : rr;
        const __nv_bfloat16* src = rr < p.H   ? p.q + b * p.qs[0] + t * p.qs[2] + h * p.qs[1]
                                   : h < Hkv ? p.k + b * p.ks[0] + t * p.ks[2] + h * p.ks[1]
                                             : p.v + b * p.vs[0] + t * p.vs[2] + (h - Hkv) * p.vs[1];
        if (!skip) w[u] = *reinterpret_cast<const uint4*>(src + 8 * c);
    }
    const int page = p.page_table[(long long)b * p.max_pages + (pos >> p.log_page)];
    const int slot = (int)pos & (p.kv.page_size - 1);
    const bool paged = page >= 0 && page < p.kv.num_pages;
    const int nc = p.rot_dim >> 3, hc = nc >> 1;  // chunks rotated; half of them
    // the pairs' angles: y' = x cos + partner sin, with the sine's sign in it
    uint64_t cs[4], sn[4];
    int other = c;  // the chunk of the partners (a chunk's own where they lie inside it)
    if (c < nc) {
        const float sign = c < hc ? -1.f : 1.f;
        if (!p.interleaved) other = c < hc ? c + hc : c - hc;
        const float* tab = p.rope + (pos + p.pos_offset) * p.rot_dim + (p.interleaved ? 4 * c : 8 * (c < hc ? c : other));
        const float* tab_sin = tab + (p.rot_dim >> 1);
        if (p.interleaved) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(tab)), y = __ldg(reinterpret_cast<const float4*>(tab_sin));
            cs[0] = tc::f32x2(x.x, x.x), cs[1] = tc::f32x2(x.y, x.y), cs[2] = tc::f32x2(x.z, x.z), cs[3] = tc::f32x2(x.w, x.w);
            sn[0] = tc::f32x2(-y.x, y.x), sn[1] = tc::f32x2(-y.y, y.y), sn[2] = tc::f32x2(-y.z, y.z), sn[3] = tc::f32x2(-y.w, y.w);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(tab) + i);
                const float4 y = __ldg(reinterpret_cast<const float4*>(tab_sin) + i);
                cs[2 * i] = tc::f32x2(x.x, x.y), cs[2 * i + 1] = tc::f32x2(x.z, x.w);
                sn[2 * i] = tc::f32x2(sign * y.x, sign * y.y), sn[2 * i + 1] = tc::f32x2(sign * y.z, sign * y.w);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (row[u] < 0) continue;
        const int rr = row[u], h = rr < p.H ? rr : rr - p.H;
        if (nc && (rr < p.H || h < Hkv)) {
            uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = p.interleaved ? __byte_perm(x[i], 0, 0x1032) : __shfl_sync(group, x[i], other, 8);
            if (c < nc)
                w[u] = make_uint4(turn(x[0], y[0], cs[0], sn[0]), turn(x[1], y[1], cs[1], sn[1]),
                                  turn(x[2], y[2], cs[2], sn[2]), turn(x[3], y[3], cs[3], sn[3]));
        }
        if (rr < p.H) {
            *reinterpret_cast<uint4*>(p.q_out + (((long long)b * p.H + h) * p.T + t) * kHeadDim + 8 * c) = w[u];
        } else if (h < Hkv) {
            if (p.k_out) *reinterpret_cast<uint4*>(p.k_out + (((long long)b * Hkv + h) * p.T + t) * kHeadDim + 8 * c) = w[u];
            if (paged)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.kv.k) + page * p.kv.k_stride_page +
                                          slot * p.kv.k_stride_slot + h * p.kv.k_stride_head + 8 * c) = w[u];
        } else if (paged) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.kv.v) + page * p.kv.v_stride_page +
                                      slot * p.kv.v_stride_slot + (h - Hkv) * p.kv.v_stride_head + 8 * c) = w[u];
        }
    }
}

template <int U>
cudaError_t launch(AppendParams& p, cudaStream_t stream) {
    p.units = (p.H + 2 * p.kv.H_kv + U - 1) / U;
    p.by_units = divisor(p.units);
    const int64_t units = ((int64_t)p.B * p.T + 7) / 8 * p.units;  // four to a block
    launch_begin(KID_KV_APPEND, stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units + 3) / 4));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_append_kernel<U>, p);
    launch_end(KID_KV_APPEND, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(float* table, int max_pos, int rot_dim, double base, cudaStream_t stream) {
    const int64_t n = (int64_t)max_pos * (rot_dim >> 1);
    launch_begin(KID_ROPE_TABLE, stream);
    rope_table_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, stream>>>(table, max_pos, rot_dim, base);
    launch_end(KID_ROPE_TABLE, stream);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(AppendParams& p, cudaStream_t stream) {
    p.by_T = divisor(p.T);
    p.log_page = 0;
    while ((1 << p.log_page) < p.kv.page_size) ++p.log_page;
    // Few rows: one per eight lanes, for the most of them at once.  With 1 and 4 rows of a token per eight lanes: 12,288
    // rows 2.5 and 3.2 us, 25,200 3.1 and 3.5, 64,890 5.0 and 4.2, 1.2 million 85 and 58 (2: 73, 6 and 8: 65).
    return (int64_t)p.B * p.T * (p.H + 2 * p.kv.H_kv) < 32768 ? launch<1>(p, stream) : launch<4>(p, stream);
}

}  // namespace saf
