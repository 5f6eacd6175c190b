// Appending new tokens to the paged key/value cache, with the rotation of
// queries and keys by position, and the table of angles.
//
// A row (one head of one token, 64 bf16) is eight 16-byte chunks, one per
// lane of an eight-lane group.  Rotated pairs (i, i + rot/2) lie rot/16 chunks
// apart, in another lane of the group (exchanged by shuffles); interleaved
// pairs (2i, 2i+1) lie inside a chunk.  Rows q, k, v of a token form one axis of
// H + 2 H_kv rows.
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

// Eight bf16 as fp32, and back (rounded to nearest even).
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendParams p) {
    const int R = p.H + 2 * p.kv.H_kv;
    const int64_t row = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 3;
    const int c = threadIdx.x & 7;
    const int64_t tok = row / R;
    const int rr = (int)(row - tok * R);
    const int b = (int)(tok / p.T), t = (int)(tok - (int64_t)b * p.T);
    // lanes of a group agree on everything below, and the shuffle names the group's lanes alone
    const uint32_t group = 0xffu << (threadIdx.x & 24);
    if (b >= p.B) return;
    const int n = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
    const int64_t pos = (int64_t)p.seq_lens[b] - n + t;
    if (t >= n || pos < 0 || pos >= p.max_len) return;
    const bool isq = rr < p.H, isk = !isq && rr < p.H + p.kv.H_kv;
    const int h = isq ? rr : isk ? rr - p.H : rr - p.H - p.kv.H_kv;
    if (isq ? (p.q == nullptr || p.replaced.get(h)) : (isk && p.keyless.get(h))) return;
    const __nv_bfloat16* src = isq ? p.q + b * p.qs[0] + h * p.qs[1] + t * p.qs[2]
                               : isk ? p.k + b * p.ks[0] + h * p.ks[1] + t * p.ks[2]
                                     : p.v + b * p.vs[0] + h * p.vs[1] + t * p.vs[2];
    uint4 w = *reinterpret_cast<const uint4*>(src + 8 * c);
    if ((isq || isk) && p.rope) {
        const int nc = p.rot_dim >> 3, hc = nc >> 1;  // chunks rotated; half of them
        const float* tab = p.rope + (pos + p.pos_offset) * p.rot_dim;
        float x[8];
        unpack8(w, x);
        if (p.interleaved) {
            if (c < nc) {
                const float4 cs = *reinterpret_cast<const float4*>(tab + 4 * c);
                const float4 sn = *reinterpret_cast<const float4*>(tab + (p.rot_dim >> 1) + 4 * c);
                const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = x[2 * i], x1 = x[2 * i + 1];
                    x[2 * i] = x0 * cc[i] - x1 * ss[i];
                    x[2 * i + 1] = x1 * cc[i] + x0 * ss[i];
                }
            }
        } else {
            const int other = c < hc ? c + hc : c < nc ? c - hc : c;  // the chunk of the pairs' other halves
            uint4 ow;
            ow.x = __shfl_sync(group, w.x, other, 8);
            ow.y = __shfl_sync(group, w.y, other, 8);
            ow.z = __shfl_sync(group, w.z, other, 8);
            ow.w = __shfl_sync(group, w.w, other, 8);
            if (c < nc) {
                float y[8];
                unpack8(ow, y);
                const int i0 = 8 * (c < hc ? c : c - hc);
                const float sign = c < hc ? -1.f : 1.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 cs = *reinterpret_cast<const float4*>(tab + i0 + 4 * u);
                    const float4 sn = *reinterpret_cast<const float4*>(tab + (p.rot_dim >> 1) + i0 + 4 * u);
                    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[4 * u + i] = x[4 * u + i] * cc[i] + sign * y[4 * u + i] * ss[i];
                }
            }
        }
        if (c < nc) w = pack8(x);
    }
    if (isq) {
        *reinterpret_cast<uint4*>(p.q_out + (((int64_t)b * p.H + h) * p.T + t) * kHeadDim + 8 * c) = w;
        return;
    }
    if (isk && p.k_out)
        *reinterpret_cast<uint4*>(p.k_out + (((int64_t)b * p.kv.H_kv + h) * p.T + t) * kHeadDim + 8 * c) = w;
    const int page = p.page_table[(int64_t)b * p.max_pages + pos / p.kv.page_size];
    if (page < 0 || page >= p.kv.num_pages) return;
    const int slot = (int)(pos % p.kv.page_size);
    __nv_bfloat16* dst =
        isk ? static_cast<__nv_bfloat16*>(p.kv.k) + page * p.kv.k_stride_page + h * p.kv.k_stride_head + slot * p.kv.k_stride_slot
            : static_cast<__nv_bfloat16*>(p.kv.v) + page * p.kv.v_stride_page + h * p.kv.v_stride_head + slot * p.kv.v_stride_slot;
    *reinterpret_cast<uint4*>(dst + 8 * c) = w;
}

}  // namespace

cudaError_t launch_rope_table(float* table, int max_pos, int rot_dim, double base, cudaStream_t stream) {
    const int64_t n = (int64_t)max_pos * (rot_dim >> 1);
    launch_begin(KID_ROPE_TABLE, stream);
    rope_table_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, stream>>>(table, max_pos, rot_dim, base);
    launch_end(KID_ROPE_TABLE, stream);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
    const int64_t threads = (int64_t)p.B * p.T * (p.H + 2 * p.kv.H_kv) * 8;
    launch_begin(KID_KV_APPEND, stream);
    kv_append_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(p);
    launch_end(KID_KV_APPEND, stream);
    return cudaGetLastError();
}

}  // namespace saf
