// Host side of the rotary calls of include/ulysses.h: argument validation and dispatch.
#include <cmath>

#include "ulysses_internal.h"

namespace ulysses {
namespace {

// Elements of a row: the parts of its heads, 512 elements at the least, are rows of a grid.
constexpr int64_t kRopeMaxRow = 1 << 23;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int rope_ok(const ulysses_rope_t* rope, int d_h) {
    if (!rope || rope->rot < 0 || rope->rot > d_h || (rope->rot > 0 && !rope->turns)) return ULYSSES_ERR_INVALID_ARG;
    if (!std::isfinite(rope->amplitude)) return ULYSSES_ERR_INVALID_ARG;
    if ((d_h != 64 && d_h != 128) || rope->rot % 16 != 0) return ULYSSES_ERR_UNSUPPORTED;
    return aligned(rope->turns, 8) ? ULYSSES_OK : ULYSSES_ERR_MISALIGNED;
}

int norm_ok(const void* w_q, const void* w_k, bool wide, float eps) {
    if (!w_q != !w_k) return ULYSSES_ERR_INVALID_ARG;
    if (w_q && !(eps >= 0.f && std::isfinite(eps))) return ULYSSES_ERR_INVALID_ARG;
    return aligned(w_q, wide ? 4 : 2) && aligned(w_k, wide ? 4 : 2) ? ULYSSES_OK : ULYSSES_ERR_MISALIGNED;
}

// Heads of a row and the rows' places, for a sharded layout.
int place(const ulysses_shape_t& s, int layout, RopeArgs& a) {
    if (s.B < 0 || s.L < 0 || s.H <= 0 || s.d_h <= 0 || s.P <= 0 || s.H_kv < 0) return ULYSSES_ERR_INVALID_ARG;
    if (layout != ULYSSES_LAYOUT_TOKEN_SHARDED && layout != ULYSSES_LAYOUT_HEAD_SHARDED) return ULYSSES_ERR_INVALID_ARG;
    const int hkv = shape_hkv(s);
    if (s.L % s.P != 0 || s.H % hkv != 0) return ULYSSES_ERR_INVALID_ARG;
    const bool head = layout == ULYSSES_LAYOUT_HEAD_SHARDED;
    if (head && (s.H % s.P != 0 || (hkv % s.P != 0 && s.P % hkv != 0))) return ULYSSES_ERR_INVALID_ARG;
    const int64_t rows = int64_t(s.B) * s.L;
    if (rows > 0x7fffffffll / (head ? s.P : 1)) return ULYSSES_ERR_UNSUPPORTED;
    a.q.heads = head ? s.H / s.P : s.H;
    a.k.heads = head ? kv_info(s).Hkvp : hkv;
    if (int64_t(a.q.heads) * s.d_h > kRopeMaxRow) return ULYSSES_ERR_UNSUPPORTED;
    a.d = s.d_h;
    a.rows = int(head ? rows * s.P : rows);
    a.seg = head ? s.L : s.L / s.P;
    a.shard_rows = head ? a.rows : s.B * a.seg;
    a.shard_step = head ? 0 : a.seg;
    a.q.x_stride = a.q.out_stride = int64_t(a.q.heads) * s.d_h;
    a.k.x_stride = a.k.out_stride = int64_t(a.k.heads) * s.d_h;
    return ULYSSES_OK;
}

// The tensors of a call: every one there and 16-byte aligned, none written that is another.
int tensors_ok(const RopeArgs& a) {
    const void* ins[] = {a.q.x, a.k.x, a.q.dy, a.k.dy, a.q.w, a.k.w, a.rope.turns, a.positions, a.cu_q, a.kv_lens};
    const void* outs[] = {a.q.out, a.k.out, a.q.dw, a.k.dw, a.workspace};
    if (!a.q.out || !a.k.out) return ULYSSES_ERR_INVALID_ARG;
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < i; ++j)
            if (outs[i] && outs[i] == outs[j]) return ULYSSES_ERR_INVALID_ARG;
        for (const void* in : ins) {
            if (!outs[i] || outs[i] != in) continue;
            const RopeTensors &t = i == 0 ? a.q : a.k, &other = i == 0 ? a.k : a.q;  // in place, element by element
            if (i > 1 || (in != t.x && in != t.dy) || t.x_stride != t.out_stride) return ULYSSES_ERR_INVALID_ARG;
            if (in == other.x || in == other.dy) return ULYSSES_ERR_INVALID_ARG;  // blocks of the other side still read it
        }
    }
    const RopeTensors* sides[] = {&a.q, &a.k};
    for (const RopeTensors* t : sides) {
        if (!aligned(t->x, 16) || !aligned(t->dy, 16) || !aligned(t->out, 16) || !aligned(t->dw, 4)) return ULYSSES_ERR_MISALIGNED;
        if (t->x_stride % 8 != 0 || t->out_stride % 8 != 0) return ULYSSES_ERR_MISALIGNED;
    }
    return ULYSSES_OK;
}

}  // namespace
}  // namespace ulysses

using namespace ulysses;

extern "C" {

int ulysses_qk_rope_fwd(ulysses_shape_t shape, int io_layout, const ulysses_rope_t* rope, int64_t pos0, const void* q,
                        const void* k, const void* w_q, const void* w_k, int w_fp32, float eps, void* q_out, void* k_out,
                        void* stream) {
    RopeArgs a{};
    int rc = place(shape, io_layout, a);
    if (rc != ULYSSES_OK || (rc = rope_ok(rope, shape.d_h)) != ULYSSES_OK) return rc;
    if ((rc = norm_ok(w_q, w_k, w_fp32 != 0, eps)) != ULYSSES_OK) return rc;
    if (a.rows == 0) return ULYSSES_OK;
    if (!q || !k) return ULYSSES_ERR_INVALID_ARG;
    a.q.x = q; a.q.out = q_out; a.q.w = w_q;
    a.k.x = k; a.k.out = k_out; a.k.w = w_k;
    a.rope = *rope; a.wide = w_fp32 != 0; a.eps = eps; a.pos0 = pos0;
    if ((rc = tensors_ok(a)) != ULYSSES_OK) return rc;
    return launch_rope(a, static_cast<cudaStream_t>(stream));
}

size_t ulysses_qk_rope_bwd_workspace_size(ulysses_shape_t shape) {
    RopeArgs a{};
    if (place(shape, ULYSSES_LAYOUT_TOKEN_SHARDED, a) != ULYSSES_OK || (a.d != 64 && a.d != 128)) return 0;
    return rope_bwd_workspace_bytes(a.q.heads, a.k.heads, a.d);  // the head layout's rows have fewer heads
}

int ulysses_qk_rope_bwd(ulysses_shape_t shape, int io_layout, const ulysses_rope_t* rope, int64_t pos0, const void* dq_out,
                        const void* dk_out, const void* q, const void* k, const void* w_q, const void* w_k, int w_fp32,
                        float eps, void* dq, void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
                        void* stream) {
    RopeArgs a{};
    int rc = place(shape, io_layout, a);
    if (rc != ULYSSES_OK || (rc = rope_ok(rope, shape.d_h)) != ULYSSES_OK) return rc;
    if ((rc = norm_ok(w_q, w_k, w_fp32 != 0, eps)) != ULYSSES_OK) return rc;
    a.rope = *rope; a.wide = w_fp32 != 0; a.eps = eps; a.pos0 = pos0; a.back = true;
    if (w_q) {
        if (!dw_q || !dw_k || !workspace) return ULYSSES_ERR_INVALID_ARG;
        if (workspace_bytes < rope_bwd_workspace_bytes(a.q.heads, a.k.heads, a.d)) return ULYSSES_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return ULYSSES_ERR_MISALIGNED;
        a.q.dw = dw_q; a.k.dw = dw_k; a.q.w = w_q; a.k.w = w_k;
        a.workspace = workspace;
    }
    if (a.rows > 0) {
        if (!dq_out || !dk_out || (w_q && (!q || !k))) return ULYSSES_ERR_INVALID_ARG;
        a.q.dy = dq_out; a.q.out = dq;
        a.k.dy = dk_out; a.k.out = dk;
        if (w_q) {
            a.q.x = q;
            a.k.x = k;
        }
        if ((rc = tensors_ok(a)) != ULYSSES_OK) return rc;
    } else if (dw_q == dw_k || !aligned(dw_q, 4) || !aligned(dw_k, 4)) {
        if (w_q) return dw_q == dw_k ? ULYSSES_ERR_INVALID_ARG : ULYSSES_ERR_MISALIGNED;
    }
    return launch_rope(a, static_cast<cudaStream_t>(stream));
}

int ulysses_qk_rope_rows(int T, int H, int H_kv, int d_h, const ulysses_rope_t* rope, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const int32_t* positions, int B, const int32_t* cu_q,
                         const int32_t* kv_lens, const void* w_q, const void* w_k, int w_fp32, float eps, void* q_out,
                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    if (T < 0 || H < 1 || H_kv < 1 || d_h < 1 || B < 0) return ULYSSES_ERR_INVALID_ARG;
    RopeArgs a{};
    int rc = rope_ok(rope, d_h);
    if (rc != ULYSSES_OK || (rc = norm_ok(w_q, w_k, w_fp32 != 0, eps)) != ULYSSES_OK) return rc;
    if (int64_t(H) * d_h > kRopeMaxRow || int64_t(H_kv) * d_h > kRopeMaxRow) return ULYSSES_ERR_UNSUPPORTED;
    if (T == 0 || (!positions && B == 0)) return ULYSSES_OK;
    if (!q || !k || (!positions && (!cu_q || !kv_lens))) return ULYSSES_ERR_INVALID_ARG;
    const int64_t q_row = int64_t(H) * d_h, k_row = int64_t(H_kv) * d_h;
    if (T == 1) {
        q_stride = q_out_stride = q_row;
        k_stride = k_out_stride = k_row;
    }
    const int64_t most = int64_t(1) << 31;
    if (q_stride < q_row || q_out_stride < q_row || k_stride < k_row || k_out_stride < k_row) return ULYSSES_ERR_INVALID_ARG;
    if (q_stride > most || q_out_stride > most || k_stride > most || k_out_stride > most) return ULYSSES_ERR_UNSUPPORTED;
    if (!aligned(positions, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4)) return ULYSSES_ERR_MISALIGNED;
    a.q.x = q; a.q.out = q_out; a.q.w = w_q; a.q.heads = H; a.q.x_stride = q_stride; a.q.out_stride = q_out_stride;
    a.k.x = k; a.k.out = k_out; a.k.w = w_k; a.k.heads = H_kv; a.k.x_stride = k_stride; a.k.out_stride = k_out_stride;
    a.rope = *rope; a.wide = w_fp32 != 0; a.eps = eps; a.d = d_h; a.rows = T;
    a.positions = positions;
    if (!positions) {
        a.B = B; a.cu_q = cu_q; a.kv_lens = kv_lens;
    }
    if ((rc = tensors_ok(a)) != ULYSSES_OK) return rc;
    return launch_rope(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
