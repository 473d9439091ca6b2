// Attention of new tokens over a paged key/value cache, one warp per (row, query head): each lane
// holds d / 32 elements of q and o, and the row's keys are visited one by one with a running
// maximum and sum.
#include <algorithm>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

namespace {

struct PagedParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* o;
    float* lse;
    const int32_t *cu_q, *kv_lens, *table;
    int64_t q_stride, table_stride, page_stride, token_stride, head_stride;
    int B, T, H, G, max_pages, num_pages, page_shift, window;
    int causal;
    float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(128) paged_attn_simple_kernel(const PagedParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y, hk = h / p.G;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= p.T) return;
    // the request that owns the row (row starts may be damaged: they are clamped)
    int b = -1, start = 0, end = 0;
    for (int i = 0; i < p.B; ++i) {
        const int s = min(max(p.cu_q[i], 0), p.T), e = min(max(p.cu_q[i + 1], s), p.T);
        if (row >= s && row < e) {
            b = i;
            start = s;
            end = e;
            break;
        }
    }
    if (b < 0) return;
    const int len = min(max(p.kv_lens[b], 0), kPagedMaxLen);
    const int kv = min(len, p.max_pages << p.page_shift);
    const int pos = len - (end - start) + (row - start);
    int lo = 0, hi = kv;
    if (p.causal) {
        hi = min(kv, pos + 1);
        if (p.window > 0) lo = max(0, pos - p.window + 1);
    }
    float q[E], o[E];
    const __nv_bfloat16* qr = p.q + row * p.q_stride + h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(qr[e]) * p.scale_log2;
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int s = lo; s < hi; ++s) {
        const int page = p.table[b * p.table_stride + (s >> p.page_shift)];
        if (unsigned(page) >= unsigned(p.num_pages)) continue;
        const int64_t off = page * p.page_stride + (s & ((1 << p.page_shift) - 1)) * p.token_stride +
                            hk * p.head_stride + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(p.k[off + e]);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        const float mn = fmaxf(m, x);
        const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = mn == -INFINITY ? 0.f : exp2f(x - mn);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(p.v[off + e]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* orow = p.o + (int64_t(row) * p.H + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0) p.lse[int64_t(h) * p.T + row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace_bytes(int, int, int, int) { return 256; }

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
    PagedParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = static_cast<const __nv_bfloat16*>(a.cache.k);
    p.v = static_cast<const __nv_bfloat16*>(a.cache.v);
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.cu_q = a.cu_q; p.kv_lens = a.kv_lens; p.table = a.table;
    p.q_stride = a.q_stride; p.table_stride = a.table_stride;
    p.page_stride = a.cache.page_stride; p.token_stride = a.cache.token_stride; p.head_stride = a.cache.head_stride;
    p.B = a.B; p.T = a.T; p.H = a.H; p.G = a.H / a.cache.H_kv;
    p.max_pages = a.max_pages; p.num_pages = a.cache.num_pages;
    p.page_shift = __builtin_ctz(unsigned(a.cache.page_size));
    p.window = a.window; p.causal = a.causal;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (a.H > 65535) return ULYSSES_ERR_UNSUPPORTED;
    const dim3 grid((a.T + 3) / 4, a.H);
    if (a.cache.d_h == 128) paged_attn_simple_kernel<128><<<grid, 128, 0, stream>>>(p);
    else paged_attn_simple_kernel<64><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace ulysses
