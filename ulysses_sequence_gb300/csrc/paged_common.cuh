// What the two paged attention kernels share: how a ragged batch whose lengths are known only
// on the device is cut into equal shares of work, without a plan made on the host.
//
// A unit is one tile of a request's new rows with one key/value head; its rows are the unit's
// tokens times the G query heads of that key/value head, so grouped heads read each key once. A
// unit's work is its number of key tiles (at least one). All units, in the order request, head,
// row tile, form one line of W key tiles, and CTA c of n takes [c W / n, (c + 1) W / n) of it:
// every CTA gets the same number of key tiles whatever the lengths. A unit that a CTA boundary
// cuts is finished by a second kernel, which joins its pieces by the online-softmax rule
// (m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i, in fp32 and in the pieces' order). A
// CTA leaves at most two pieces, so the workspace depends on the grid alone.
#pragma once

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

struct PagedParams {
    int B, T, H, Hkv, G;
    int max_pages, num_pages, page_shift;
    int causal, window;
    int min_rows;            // requests with fewer rows (new tokens x G) than this are left to the other kernel
    int max_rows;            // and those with more
    float scale_log2;
    int64_t q_stride, table_stride;
    const __nv_bfloat16* q;
    const int32_t *cu_q, *kv_lens, *table;
    __nv_bfloat16* o;
    float* lse;
    float* part_o;           // [2 * CTAs][rows][d] fp32 pieces of cut units, not normalised
    float2* part_ml;         // [2 * CTAs][rows] (m in the log2 domain, l)
    struct PagedMeta* meta;  // [CTAs]
    uint32_t* err;
};

// What the joining kernel knows of CTA c: a first piece that continues a unit is in slot 2 c, a last
// piece that opens one in slot 2 c + 1.
struct PagedMeta {
    int cont;    // the first piece continues a unit begun by an earlier CTA
    int ends;    // ... and finishes it
    int opens;   // the last piece begins a unit that a later CTA continues
    int head;    // of the unit opened
    int row0;    // its first row of q
    int rows;    // its rows (tokens x G)
};

// The new rows [start, start + n) of request i, its keys [0, kv), and the position of row 0.
struct PagedSeq {
    int start, n, kv, base;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int i) {
    PagedSeq s;
    const int a = p.cu_q[i], e = p.cu_q[i + 1], len = min(max(p.kv_lens[i], 0), kPagedMaxLen);
    s.start = min(max(a, 0), p.T);
    s.n = min(max(e, s.start), p.T) - s.start;
    s.kv = min(len, p.max_pages << p.page_shift);
    s.base = len - s.n;
    const int64_t rows = int64_t(s.n) * p.G;
    if (rows < p.min_rows || rows > p.max_rows) s.n = 0;
    return s;
}

// Keys [lo, hi) that some row of tokens [t0, t1) may see.
__device__ __forceinline__ void paged_range(const PagedParams& p, const PagedSeq& s, int t0, int t1, int& lo, int& hi) {
    lo = 0;
    hi = s.kv;
    if (p.causal) {
        hi = min(s.kv, max(0, s.base + t1));
        if (p.window > 0) lo = min(hi, max(0, s.base + t0 - p.window + 1));
    }
}

// Key tiles of a unit: the first one and how many (one, all masked, where no row sees a key).
template <int KT>
__device__ __forceinline__ void paged_tiles(const PagedParams& p, const PagedSeq& s, int t0, int t1, int& first, int& count) {
    int lo, hi;
    paged_range(p, s, t0, t1, lo, hi);
    first = lo / KT;
    count = max(1, (hi + KT - 1) / KT - first);
}

// Key tiles of one head of a request, over its row tiles of TQ tokens.
template <int KT>
__device__ __forceinline__ int64_t paged_head_cost(const PagedParams& p, const PagedSeq& s, int TQ) {
    int64_t sum = 0;
    for (int t0 = 0; t0 < s.n; t0 += TQ) {
        int first, count;
        paged_tiles<KT>(p, s, t0, min(s.n, t0 + TQ), first, count);
        sum += count;
    }
    return sum;
}

// One CTA's walk along the line of key tiles; the whole warp holds the same state.
template <int KT>
struct PagedWalk {
    int i, head, t0, t1;     // unit: request, key/value head, tokens [t0, t1)
    PagedSeq s;
    int first, count, off;   // its key tiles, and the next one's offset among them
    int64_t left;            // key tiles that this CTA still has to do

    __device__ __forceinline__ void unit(const PagedParams& p, int TQ) {
        t1 = min(s.n, t0 + TQ);
        paged_tiles<KT>(p, s, t0, t1, first, count);
    }
    // The next request that has rows, 32 looked at at a time; only called while there is one.
    __device__ __forceinline__ void next_request(const PagedParams& p) {
        const int lane = int(lane_id());
        for (int a = i + 1; a < p.B; a += 32) {
            PagedSeq c{};
            if (a + lane < p.B) c = paged_seq(p, a + lane);
            const unsigned has = __ballot_sync(0xffffffffu, c.n > 0);
            if (has) {
                const int src = __ffs(has) - 1;
                i = a + src;
                s.start = __shfl_sync(0xffffffffu, c.start, src);
                s.n = __shfl_sync(0xffffffffu, c.n, src);
                s.kv = __shfl_sync(0xffffffffu, c.kv, src);
                s.base = __shfl_sync(0xffffffffu, c.base, src);
                return;
            }
        }
        s.n = 0;
    }
    __device__ __forceinline__ void next_unit(const PagedParams& p, int TQ) {
        off = 0;
        t0 += TQ;
        if (t0 >= s.n) {
            t0 = 0;
            if (++head == p.Hkv) {
                head = 0;
                next_request(p);
            }
        }
        unit(p, TQ);
    }
};

// Where this CTA's share of the line begins. All threads of the block call it (NT threads, a whole
// number of warps); every warp leaves with the same walk. Returns the number of CTAs that have work
// (the first ones); a CTA at or past it has none.
template <int KT, int NT>
__device__ __forceinline__ int paged_share(const PagedParams& p, int TQ, int min_tiles, int64_t* sh /* [NT / 32 + 4] */,
                                           PagedWalk<KT>& w) {
    constexpr int NW = NT / 32;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0, cost0 = 0;
    for (int i = tid; i < p.B; i += NT) {
        const PagedSeq s = paged_seq(p, i);
        const int64_t c = s.n > 0 ? paged_head_cost<KT>(p, s, TQ) * p.Hkv : 0;
        if (i == tid) cost0 = c;
        mine += c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh[warp] = mine;
    if (tid == 0) sh[NW] = -1;
    __syncthreads();
    int64_t W = 0;
    for (int k = 0; k < NW; ++k) W += sh[k];
    const int n = int(min(int64_t(gridDim.x), (W + min_tiles - 1) / min_tiles));
    const int c = int(blockIdx.x);
    if (c >= n) return n;
    const int64_t begin = W * c / n;
    w.left = W * (c + 1) / n - begin;
    // the request that holds tile `begin`: a running prefix, NT requests at a time
    int64_t run = 0;
    for (int a = 0; a < p.B; a += NT) {
        int64_t cost = cost0;
        if (a > 0) {
            cost = 0;
            if (a + tid < p.B) {
                const PagedSeq s = paged_seq(p, a + tid);
                if (s.n > 0) cost = paged_head_cost<KT>(p, s, TQ) * p.Hkv;
            }
        }
        int64_t incl = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) sh[warp] = incl;
        __syncthreads();
        int64_t before = run, total = 0;
        for (int k = 0; k < NW; ++k) {
            if (k < warp) before += sh[k];
            total += sh[k];
        }
        if (begin >= before + incl - cost && begin < before + incl) {
            sh[NW] = a + tid;
            sh[NW + 1] = begin - (before + incl - cost);
        }
        run += total;
        if (begin < run) break;  // the same in all threads
    }
    __syncthreads();
    w.i = int(sh[NW]);
    int64_t rem = sh[NW + 1];
    w.s = paged_seq(p, w.i);
    // the head, then the row tile, 32 looked at at a time
    int64_t per_head = 0;
    for (int t = lane * TQ; t < w.s.n; t += 32 * TQ) {
        int first, count;
        paged_tiles<KT>(p, w.s, t, min(w.s.n, t + TQ), first, count);
        per_head += count;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) per_head += __shfl_xor_sync(0xffffffffu, per_head, o);
    w.head = int(rem / per_head);
    rem -= per_head * w.head;
    for (int64_t a = 0; a < w.s.n; a += int64_t(32) * TQ) {
        const int64_t t = a + int64_t(lane) * TQ;
        int first = 0, count = 0;
        if (t < w.s.n) paged_tiles<KT>(p, w.s, int(t), int(min(int64_t(w.s.n), t + TQ)), first, count);
        int64_t incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, rem >= incl - count && rem < incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            w.t0 = int(a) + src * TQ;
            w.off = int(rem - __shfl_sync(0xffffffffu, incl - count, src));
            break;
        }
        rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    w.unit(p, TQ);
    return n;
}

// Joins the pieces of cut units: block (c, y) takes columns [y D / NY, (y + 1) D / NY) of the unit that
// CTA c - 1 opened and CTA c continues. ROWS is the row pitch of a slot.
template <int D, int ROWS, int NY>
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedParams p, int ctas) {
    constexpr int COLS = D / NY, V = COLS / 4;  // float4 columns of this block
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = int(blockIdx.x) + 1;
    const PagedMeta open = p.meta[c - 1];
    if (!open.opens || !p.meta[c].cont) return;
    int last = c;
    while (!p.meta[last].ends && last + 1 < ctas) ++last;
    // pieces: slot 2 (c - 1) + 1, then slots 2 c, 2 (c + 1), ... 2 last
    const int pieces = last - c + 2;
    auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i); };
    for (int x = int(threadIdx.x); x < open.rows * V; x += 128) {
        const int r = x / V, col = int(blockIdx.y) * COLS + (x % V) * 4;
        float m = -INFINITY;
        for (int i = 0; i < pieces; ++i) m = fmaxf(m, p.part_ml[int64_t(slot(i)) * ROWS + r].x);
        const float neg = m == -INFINITY ? 0.f : -m;
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < pieces; ++i) {
            const int64_t at = int64_t(slot(i)) * ROWS + r;
            const float2 ml = p.part_ml[at];
            const float4 y = *reinterpret_cast<const float4*>(p.part_o + at * D + col);
            const float e = ex2(ml.x + neg);  // 2^-inf = 0: a piece that saw no key has l = 0 and O = 0
            l += e * ml.y;
            o.x += e * y.x;
            o.y += e * y.y;
            o.z += e * y.z;
            o.w += e * y.w;
        }
        const float inv = l > 0.f ? 1.0f / l : 0.f;
        const int row = open.row0 + r / p.G, h = open.head * p.G + r % p.G;
        *reinterpret_cast<uint2*>(p.o + (int64_t(row) * p.H + h) * D + col) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (col == 0) p.lse[int64_t(h) * p.T + row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

// Launches the joining kernel behind the kernel that wrote the pieces, its start overlapped with that
// kernel's end (it waits for it before its first read).
template <int D, int ROWS, int NY>
inline int launch_paged_join(const PagedParams& p, int ctas, cudaStream_t stream) {
    if (ctas < 2) return ULYSSES_OK;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(ctas - 1), NY);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, ROWS, NY>, p, ctas) == cudaSuccess ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

// Tensor map of a pool's keys or values, (64 elements, token, head, page, 64-element chunk), for copies
// of `rows` tokens of one page and head by `chunks` chunks (chunk after chunk), 128-byte swizzle.
bool encode_pages(CUtensorMap* map, const ulysses_kv_cache_t& c, const void* base, int rows, int chunks);

// Requests of few rows (paged_decode.cu), and the others (paged_chunk.cu).
int paged_decode_rows();
size_t paged_decode_workspace_bytes(int d_h);
int launch_paged_decode(const PagedAttnArgs& a, const PagedParams& p, void* workspace, cudaStream_t stream);
size_t paged_chunk_workspace_bytes(int d_h);
int launch_paged_chunk(const PagedAttnArgs& a, const PagedParams& p, void* workspace, cudaStream_t stream);

}  // namespace ulysses
