// Host side of the paged-cache calls of include/ulysses.h: argument validation and dispatch.
#include <cmath>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool page_size_ok(int page_size) {
    return page_size >= 16 && page_size <= 4096 && (page_size & (page_size - 1)) == 0;
}

// A stride is used only where its dimension has more than one entry; others are set to a valid
// value, so that the kernels and tensor maps need no special case.
int normalise_cache(const ulysses_kv_cache_t* in, ulysses_kv_cache_t& c) {
    if (!in) return ULYSSES_ERR_INVALID_ARG;
    c = *in;
    if (c.num_pages < 1 || c.H_kv < 1 || c.d_h < 1 || !page_size_ok(c.page_size)) return ULYSSES_ERR_INVALID_ARG;
    if (int64_t(c.num_pages) * c.page_size > 0x7fffffffll) return ULYSSES_ERR_INVALID_ARG;
    if (c.d_h % 8 != 0 || int64_t(c.H_kv) * c.d_h > (1 << 24)) return ULYSSES_ERR_UNSUPPORTED;
    if (!c.k || !c.v || c.k == c.v) return ULYSSES_ERR_INVALID_ARG;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return ULYSSES_ERR_MISALIGNED;
    const int64_t whole = int64_t(c.page_size) * c.H_kv * c.d_h;
    if (c.H_kv == 1) c.head_stride = c.d_h;
    if (c.num_pages == 1) c.page_stride = whole;
    const int64_t strides[3] = {c.page_stride, c.token_stride, c.head_stride};
    for (int64_t s : strides) {
        if (s < c.d_h || s > (int64_t(1) << 38)) return ULYSSES_ERR_INVALID_ARG;
        if (s % 8 != 0) return ULYSSES_ERR_MISALIGNED;
    }
    return ULYSSES_OK;
}

int mask_ok(int mask_kind, int window) {
    if (mask_kind == ULYSSES_MASK_BLOCK_SPARSE) return ULYSSES_ERR_UNSUPPORTED;
    if (mask_kind != ULYSSES_MASK_NONE && mask_kind != ULYSSES_MASK_CAUSAL) return ULYSSES_ERR_INVALID_ARG;
    if (window < 0 || (window > 0 && mask_kind != ULYSSES_MASK_CAUSAL)) return ULYSSES_ERR_INVALID_ARG;
    return ULYSSES_OK;
}

int heads_ok(int H, int H_kv, int d_h, int max_q) {
    if (H < 1 || H_kv < 1 || d_h < 1 || max_q < 0 || H % H_kv != 0) return ULYSSES_ERR_INVALID_ARG;
    if ((d_h != 64 && d_h != 128) || H / H_kv > kPagedMaxGroup) return ULYSSES_ERR_UNSUPPORTED;
    return ULYSSES_OK;
}

}  // namespace
}  // namespace ulysses

using namespace ulysses;

extern "C" {

int ulysses_page_plan(int B, int T, int page_size, int max_pages, int64_t table_stride, int num_pages,
                      const int32_t* cached_lens, const int32_t* new_lens, const int32_t* free_pages,
                      int free_capacity, const int32_t* n_free, int32_t* block_table, int32_t* cu_q,
                      int32_t* kv_lens, int32_t* slot_map, int32_t* info, void* stream) {
    if (B < 0 || T < 0 || max_pages < 0 || num_pages < 1 || free_capacity < 0 || !page_size_ok(page_size))
        return ULYSSES_ERR_INVALID_ARG;
    if (int64_t(num_pages) * page_size > 0x7fffffffll || int64_t(max_pages) * page_size + T > 0x7fffffffll)
        return ULYSSES_ERR_INVALID_ARG;
    if (B > kPlanMaxB) return ULYSSES_ERR_UNSUPPORTED;
    if (B > 1 && table_stride < max_pages) return ULYSSES_ERR_INVALID_ARG;
    if (!n_free || !cu_q || !info) return ULYSSES_ERR_INVALID_ARG;
    if (B > 0 && (!cached_lens || !new_lens || !kv_lens || (!block_table && max_pages > 0))) return ULYSSES_ERR_INVALID_ARG;
    if ((T > 0 && !slot_map) || (free_capacity > 0 && !free_pages)) return ULYSSES_ERR_INVALID_ARG;
    const void* ins[] = {cached_lens, new_lens, free_pages, n_free};
    const void* outs[] = {block_table, cu_q, kv_lens, slot_map, info};
    for (int i = 0; i < 5; ++i) {
        if (!aligned(outs[i], 4)) return ULYSSES_ERR_MISALIGNED;
        for (const void* b : ins)
            if (outs[i] && outs[i] == b) return ULYSSES_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return ULYSSES_ERR_INVALID_ARG;
    }
    for (const void* a : ins)
        if (!aligned(a, 4)) return ULYSSES_ERR_MISALIGNED;
    return launch_page_plan(B, T, __builtin_ctz(unsigned(page_size)), max_pages, table_stride, num_pages, cached_lens,
                            new_lens, free_pages, free_capacity, n_free, block_table, cu_q, kv_lens, slot_map, info,
                            static_cast<cudaStream_t>(stream));
}

int ulysses_kv_append(const ulysses_kv_cache_t* cache, int T, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const int32_t* slot_map, void* stream) {
    ulysses_kv_cache_t c;
    const int rc = normalise_cache(cache, c);
    if (rc != ULYSSES_OK) return rc;
    if (T < 0) return ULYSSES_ERR_INVALID_ARG;
    if (T == 0) return ULYSSES_OK;
    if (!k || !v || !slot_map) return ULYSSES_ERR_INVALID_ARG;
    const void* ins[] = {k, v, slot_map};
    for (const void* a : ins)
        if (a == c.k || a == c.v) return ULYSSES_ERR_INVALID_ARG;
    const int64_t row = int64_t(c.H_kv) * c.d_h;
    if (T == 1) k_stride = v_stride = row;
    if (k_stride < row || v_stride < row) return ULYSSES_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4))
        return ULYSSES_ERR_MISALIGNED;
    return launch_kv_append(c, T, k, k_stride, v, v_stride, slot_map, static_cast<cudaStream_t>(stream));
}

size_t ulysses_paged_attn_workspace_size(int H, int H_kv, int d_h, int max_q) {
    if (heads_ok(H, H_kv, d_h, max_q) != ULYSSES_OK) return 0;
    return paged_attn_workspace_bytes(H, H_kv, d_h, max_q);
}

int ulysses_paged_attn_fwd(const ulysses_kv_cache_t* cache, int B, int T, int H, int max_q, int mask_kind, int window,
                           float softmax_scale, const void* q, int64_t q_stride, const int32_t* cu_q,
                           const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride, int max_pages,
                           void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    PagedAttnArgs a{};
    int rc = normalise_cache(cache, a.cache);
    if (rc != ULYSSES_OK) return rc;
    if (B < 0 || T < 0 || max_pages < 0) return ULYSSES_ERR_INVALID_ARG;
    if ((rc = heads_ok(H, a.cache.H_kv, a.cache.d_h, max_q)) != ULYSSES_OK) return rc;
    if ((rc = mask_ok(mask_kind, window)) != ULYSSES_OK) return rc;
    if (B > 1 && table_stride < max_pages) return ULYSSES_ERR_INVALID_ARG;
    if (int64_t(max_pages) * a.cache.page_size > kPagedMaxLen || T > kPagedMaxLen) return ULYSSES_ERR_UNSUPPORTED;
    if (int64_t(H) * a.cache.d_h > (1 << 24)) return ULYSSES_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return ULYSSES_OK;
    if (!q || !cu_q || !kv_lens || (!block_table && max_pages > 0) || !o || !lse || !workspace) return ULYSSES_ERR_INVALID_ARG;
    const void* ins[] = {q, cu_q, kv_lens, block_table, a.cache.k, a.cache.v};
    const void* outs[] = {o, lse, workspace};
    for (const void* x : outs)
        for (const void* y : ins)
            if (x == y) return ULYSSES_ERR_INVALID_ARG;
    if (o == lse || o == workspace || lse == workspace) return ULYSSES_ERR_INVALID_ARG;
    if (workspace_bytes < paged_attn_workspace_bytes(H, a.cache.H_kv, a.cache.d_h, max_q)) return ULYSSES_ERR_INVALID_ARG;
    const int64_t row = int64_t(H) * a.cache.d_h;
    if (T == 1) q_stride = row;
    if (q_stride < row || q_stride > (int64_t(1) << 38)) return ULYSSES_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256) ||
        !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4))
        return ULYSSES_ERR_MISALIGNED;
    a.B = B; a.T = T; a.H = H; a.max_q = max_q;
    a.window = window < kPagedMaxLen ? window : kPagedMaxLen;  // positions and keys stay below it
    a.causal = mask_kind == ULYSSES_MASK_CAUSAL;
    a.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(float(a.cache.d_h));
    a.q = q; a.q_stride = q_stride;
    a.cu_q = cu_q; a.kv_lens = kv_lens; a.table = block_table; a.table_stride = table_stride; a.max_pages = max_pages;
    a.o = o; a.lse = lse; a.workspace = workspace;
    return launch_paged_attn(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
