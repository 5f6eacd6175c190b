// Attention of new tokens over the paged key/value cache: the plain first
// form, one block per row (head h, new token t of sequence b), keys in tiles of
// 128, one key per thread for the scores and one column per thread for P V.
#include "saf_paged.cuh"

namespace saf {
namespace {

__global__ void __launch_bounds__(128) paged_row_kernel(const __grid_constant__ PagedParams p) {
    __shared__ float qs[64], ps[128], red[8], part[128];
    __shared__ const __nv_bfloat16* vrow[128];
    const int t = blockIdx.x % p.T, h = (blockIdx.x / p.T) % p.H, b = blockIdx.x / p.T / p.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
    if (t >= n) return;
    const int len = min(max(p.seq_lens[b], 0), p.max_len);
    const int i = p.prefix_len + len - n + t;  // position of the row; it sees keys j <= i
    const int g = h / (p.H / p.kv.H_kv);
    const bool rep = p.replaced.get(h);
    const int64_t row = ((int64_t)b * p.H + h) * p.T + t;
    if (tid < 64) qs[tid] = rep ? 0.f : __bfloat162float(p.q[row * kHeadDim + tid]);
    __syncthreads();
    float m = kNegInf, l = 0.f, acc = 0.f;
    const int nk = min(i + 1, p.prefix_len + len);
    for (int j0 = 0; j0 < nk; j0 += 128) {
        const int j = j0 + tid;
        float s = kNegInf;
        vrow[tid] = nullptr;
        if (j < nk) {
            const int at = j < p.prefix_len ? j : j - p.prefix_len;
            const int32_t* table = j < p.prefix_len ? p.prefix_table : p.page_table + (int64_t)b * p.max_pages;
            const int page = table[at / p.kv.page_size], slot = at % p.kv.page_size;
            if (page >= 0 && page < p.kv.num_pages) {
                vrow[tid] = static_cast<const __nv_bfloat16*>(p.kv.v) + page * p.kv.v_stride_page + g * p.kv.v_stride_head +
                            slot * p.kv.v_stride_slot;
                if (rep) {
                    s = p.a[(int64_t)h * p.pattern_len + j] + p.r[(int64_t)h * p.pattern_len + (i - j)];
                } else {
                    const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.kv.k) + page * p.kv.k_stride_page +
                                              g * p.kv.k_stride_head + slot * p.kv.k_stride_slot;
                    float dot = 0.f;
                    for (int c = 0; c < 64; ++c) dot = fmaf(qs[c], __bfloat162float(kr[c]), dot);
                    s = dot * 0.125f;
                }
            }
        }
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float f = mn == kNegInf ? 1.f : expf(m - mn);
        const float e = s == kNegInf ? 0.f : expf(s - mn);
        ps[tid] = e;
        float sum = e;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) red[4 + warp] = sum;
        __syncthreads();
        l = l * f + (red[4] + red[5] + red[6] + red[7]);
        acc *= f;
        m = mn;
        for (int u = 0; u < 64; ++u) {
            const int key = (tid >> 6) * 64 + u;
            if (vrow[key]) acc = fmaf(ps[key], __bfloat162float(vrow[key][tid & 63]), acc);
        }
        __syncthreads();
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < 64) p.o[row * kHeadDim + tid] = __float2bfloat16(l > 0.f || l != l ? (part[tid] + part[tid + 64]) / l : 0.f);
    if (tid == 0) p.lse[row] = l > 0.f || l != l ? m + logf(l) : kNegInf;
}

}  // namespace

size_t paged_workspace_bytes(int B, int H, int H_kv, int T, int prefix_len) {
    (void)B, (void)H, (void)H_kv, (void)T, (void)prefix_len;
    return 256;
}

cudaError_t launch_paged_attn(const PagedParams& p, cudaStream_t stream) {
    launch_begin(KID_PAGED_ATTN, stream);
    paged_row_kernel<<<(unsigned)((int64_t)p.B * p.H * p.T), 128, 0, stream>>>(p);
    launch_end(KID_PAGED_ATTN, stream);
    return cudaGetLastError();
}

}  // namespace saf
