// Attention of new tokens over a paged key/value cache, one warp per (row, query head): each lane
// holds d / 32 elements of q and o, and the row's keys are visited one by one with a running
// maximum and sum.
#include <algorithm>

#include "paged_common.cuh"

namespace ulysses {

namespace {

template <int D>
__global__ void __launch_bounds__(128) paged_attn_simple_kernel(const PagedParams p, const ulysses_kv_cache_t c) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y, hk = h / p.G;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= p.T) return;
    PagedSeq sq{};
    int b = -1;
    for (int i = 0; i < p.B && b < 0; ++i) {
        sq = paged_seq(p, i);
        if (row >= sq.start && row < sq.start + sq.n) b = i;
    }
    if (b < 0) return;
    const int kv = sq.kv, pos = sq.base + (row - sq.start);
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16*>(c.k), *vp = static_cast<const __nv_bfloat16*>(c.v);
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
        const int64_t off = page * c.page_stride + (s & ((1 << p.page_shift) - 1)) * c.token_stride +
                            hk * c.head_stride + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(kp[off + e]);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        const float mn = fmaxf(m, x);
        const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = mn == -INFINITY ? 0.f : exp2f(x - mn);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(vp[off + e]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* orow = p.o + (int64_t(row) * p.H + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) orow[e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0) p.lse[int64_t(h) * p.T + row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

// Requests whose rows (new tokens x grouped heads) fit the decode kernel's tile go there: all of them
// when the caller's bound on new tokens says so, else those that do.
static bool decode_only(int G, int max_q) {
    return G <= paged_decode_rows() && max_q > 0 && int64_t(max_q) * G <= paged_decode_rows();
}

size_t paged_attn_workspace_bytes(int, int, int d_h, int) { return paged_decode_workspace_bytes(d_h); }

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
    PagedParams p{};
    p.B = a.B; p.T = a.T; p.H = a.H; p.Hkv = a.cache.H_kv; p.G = a.H / a.cache.H_kv;
    p.max_pages = a.max_pages; p.num_pages = a.cache.num_pages;
    p.page_shift = __builtin_ctz(unsigned(a.cache.page_size));
    p.causal = a.causal; p.window = a.window;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.q_stride = a.q_stride; p.table_stride = a.table_stride;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.cu_q = a.cu_q; p.kv_lens = a.kv_lens; p.table = a.table;
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.err = device_error_word();
    if (!p.err) return ULYSSES_ERR_CUDA;
    if (a.H > 65535) return ULYSSES_ERR_UNSUPPORTED;
    const bool only = decode_only(p.G, a.max_q);
    if (p.G <= paged_decode_rows()) {
        p.min_rows = 1;
        p.max_rows = only ? 0x7fffffff : paged_decode_rows();
        const int rc = launch_paged_decode(a, p, a.workspace, stream);
        if (rc != ULYSSES_OK || only) return rc;
        p.min_rows = paged_decode_rows() + 1;
    } else {
        p.min_rows = 1;
    }
    p.max_rows = 0x7fffffff;
    const dim3 grid((a.T + 3) / 4, a.H);
    if (a.cache.d_h == 128) paged_attn_simple_kernel<128><<<grid, 128, 0, stream>>>(p, a.cache);
    else paged_attn_simple_kernel<64><<<grid, 128, 0, stream>>>(p, a.cache);
    return cudaGetLastError() == cudaSuccess ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace ulysses
