// What the two paged attention kernels share: how a ragged batch whose lengths are known only
// on the device is cut into equal shares of work, without a plan made on the host.
//
// A unit is one tile of a request's new rows with one key/value head; its rows are the unit's
// tokens times the G query heads of that key/value head, so grouped heads read each key once. A
// unit costs its number of key tiles (at least one) plus a fixed part for its queries and its rows'
// way out, counted in key tiles. All units, in the order request, head, row tile, form one line of cost
// W, and CTA c of n takes [c W / n, (c + 1) W / n) of it: every CTA gets the same cost whatever the
// lengths. A unit that a CTA boundary cuts is finished by a second kernel, which joins its pieces by the
// online-softmax rule (m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i, in fp32 and in the
// pieces' order). A CTA leaves at most two pieces, so the workspace depends on the grid alone.
#pragma once

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

// What the joining kernel knows of CTA c: the unit that its last piece opens and later CTAs go on with. The
// opening piece is in slot 2 c + 1, those of CTAs c + 1, ... in slots 2 (c + 1), ...
struct PagedMeta {
    int pieces;  // of the unit, 0 where there is none
    int head, row0, rows;
};

// The pieces that one kernel's CTAs leave, in the workspace.
struct PagedParts {
    float* o;         // [2 * CTAs][rows][d] fp32, not normalised
    float2* ml;       // [2 * CTAs][rows] (m in the log2 domain, l)
    PagedMeta* meta;  // [CTAs]
    int rows;         // pitch of a slot: the rows of a unit
    int ctas;         // of the launch; 0 where the kernel is not launched
};

struct PagedParams {
    int B, T, H, Hkv, G;
    int max_pages, num_pages, page_shift;
    int causal, window;
    int min_rows;            // requests with fewer rows (new tokens x G) than this are left to the other kernel
    int max_rows;            // and those with more
    int unit_tokens;         // new tokens of a unit
    float scale_log2;
    int64_t q_stride, table_stride;
    const __nv_bfloat16* q;
    const int32_t *cu_q, *kv_lens, *table;
    __nv_bfloat16* o;
    float* lse;
    PagedParts parts;        // of the kernel that gets these parameters
    uint32_t* err;
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

// Cost of one head of a request, over its row tiles of TQ tokens; OVH is a unit's fixed part.
template <int KT, int OVH>
__device__ __forceinline__ int64_t paged_head_cost(const PagedParams& p, const PagedSeq& s) {
    const int TQ = p.unit_tokens;
    int64_t sum = 0;
#pragma unroll 1
    for (int t0 = 0; t0 < s.n; t0 += TQ) {
        int first, count;
        paged_tiles<KT>(p, s, t0, min(s.n, t0 + TQ), first, count);
        sum += count + OVH;
    }
    return sum;
}

// One CTA's walk along the line; the whole warp holds the same state.
template <int KT, int OVH>
struct PagedWalk {
    int i, head, t0, t1;     // unit: request, key/value head, tokens [t0, t1)
    PagedSeq s;
    int first, count;        // its key tiles
    int pos;                 // cost of it that lies behind
    int64_t left;            // cost that this CTA still has to do
    int64_t W;               // the line's cost
    int n;                   // CTAs with work (the first ones)

    __device__ __forceinline__ void unit(const PagedParams& p) {
        t1 = min(s.n, t0 + p.unit_tokens);
        paged_tiles<KT>(p, s, t0, t1, first, count);
    }
    // This CTA's part of the unit, key tiles [off, off + tiles), possibly none.
    __device__ __forceinline__ void take(int& off, int& tiles) {
        const int end = int(min(int64_t(pos) + left, int64_t(OVH) + count));
        off = max(0, pos - OVH);
        tiles = max(0, end - OVH) - off;
        left -= end - pos;
        pos = end;
    }
    // Pieces of the unit from CTA c, which has just taken its end of the line and left some of the unit.
    __device__ __forceinline__ int pieces(int c) const {
        const int64_t unit_end = W * (c + 1) / n + (OVH + count - pos);
        return int((unit_end * n + W - 1) / W) - c;  // the CTA whose end reaches the unit's, as an index past c
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
        left = 0;  // not reached while the lengths stand still: the share ends where the requests do
    }
    __device__ __forceinline__ void next_unit(const PagedParams& p) {
        pos = 0;
        t0 += p.unit_tokens;
        if (t0 >= s.n) {
            t0 = 0;
            if (++head == p.Hkv) {
                head = 0;
                next_request(p);
            }
        }
        unit(p);
    }
};

// Inclusive prefix over the block's NT threads, and the block's sum. sh: NT / 32 entries.
template <int NT>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* sh, int64_t& total) {
    constexpr int NW = NT / 32;
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();  // sh may still be read from the call before
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        if (k < warp) before += sh[k];
        total += sh[k];
    }
    return v + before;
}

// The CTA's end of the line, once its cost is known: false for a CTA without work.
template <int KT, int OVH>
__device__ __forceinline__ bool paged_cut(PagedWalk<KT, OVH>& w, int min_cost, int64_t& begin) {
    w.n = int(min(int64_t(gridDim.x), (w.W + min_cost - 1) / min_cost));
    const int c = int(blockIdx.x);
    w.left = 0;
    if (c >= w.n) return false;
    int64_t end;
    if (w.W < (int64_t(1) << 31)) {  // 32-bit divisions where they do
        const uint32_t W = uint32_t(w.W), n = uint32_t(w.n), q = W / n, r = W - q * n;
        begin = q * uint32_t(c) + r * uint32_t(c) / n;
        end = q * uint32_t(c + 1) + r * uint32_t(c + 1) / n;
    } else {
        begin = w.W * c / w.n;
        end = w.W * (c + 1) / w.n;
    }
    w.left = end - begin;
    return true;
}

// The walk's first unit, `rem` into request w.i, which is in w.s: the head, then the row tile, 32 looked at at
// a time.
template <int KT, int OVH>
__device__ __forceinline__ void paged_start(const PagedParams& p, int64_t rem, PagedWalk<KT, OVH>& w) {
    const int lane = int(lane_id()), TQ = p.unit_tokens;
    w.t0 = 0;
    if (w.s.n <= TQ) {
        w.unit(p);
        const int cost = OVH + w.count;
        w.head = min(p.Hkv - 1, w.W < (int64_t(1) << 31) ? int(uint32_t(rem) / uint32_t(cost)) : int(rem / cost));
        w.pos = min(cost, int(rem - int64_t(cost) * w.head));
        return;
    }
    int64_t per_head = 0;
    for (int64_t t = int64_t(lane) * TQ; t < w.s.n; t += int64_t(32) * TQ) {
        int first, count;
        paged_tiles<KT>(p, w.s, int(t), int(min(int64_t(w.s.n), t + TQ)), first, count);
        per_head += count + OVH;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) per_head += __shfl_xor_sync(0xffffffffu, per_head, o);
    w.head = int(min(int64_t(p.Hkv - 1), rem / per_head));
    rem -= per_head * w.head;
    for (int64_t a = 0; a < w.s.n; a += int64_t(32) * TQ) {
        const int64_t t = a + int64_t(lane) * TQ;
        int first = 0, count = -OVH;
        if (t < w.s.n) paged_tiles<KT>(p, w.s, int(t), int(min(int64_t(w.s.n), t + TQ)), first, count);
        const int64_t cost = count + OVH;
        int64_t sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, rem >= sum - cost && rem < sum);
        if (hit) {
            const int src = __ffs(hit) - 1;
            w.t0 = int(a) + src * TQ;
            w.pos = int(rem - __shfl_sync(0xffffffffu, sum - cost, src));
            break;
        }
        rem -= __shfl_sync(0xffffffffu, sum, 31);
    }
    w.unit(p);
}

template <int KT, int OVH>
__device__ __forceinline__ int64_t paged_cost(const PagedParams& p, int i) {
    if (i >= p.B) return 0;
    const PagedSeq s = paged_seq(p, i);
    return s.n > 0 ? paged_head_cost<KT, OVH>(p, s) * p.Hkv : int64_t(0);
}

// Where this CTA's share of the line begins, for batches of up to kFewRequests requests, in two steps with
// the block's barrier between them: every thread puts down a request's cost, then one warp finds the
// place. The code runs once a launch, so it is kept short: its instruction fetches are most of its time (200 decoding
// requests with a window: 13.3 us, against 13.7 us by the whole block, which larger batches take).
constexpr int kFewRequests = 256;
template <int KT, int OVH, int NT>
__device__ __forceinline__ void paged_costs(const PagedParams& p, int64_t* costs /* [kFewRequests] */) {
#pragma unroll 1
    for (int i = int(threadIdx.x); i < kFewRequests; i += NT) costs[i] = paged_cost<KT, OVH>(p, i);
    fence_proxy_async_smem();  // copies may land there next
}
template <int KT, int OVH>
__device__ __forceinline__ bool paged_share_warp(const PagedParams& p, int min_cost, const int64_t* costs, PagedWalk<KT, OVH>& w) {
    const int lane = int(lane_id()), per = (p.B + 31) / 32;  // consecutive requests of a lane
    int64_t mine = 0;
#pragma unroll 1
    for (int k = 0; k < per; ++k) mine += costs[lane * per + k];
    int64_t incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    w.W = __shfl_sync(0xffffffffu, incl, 31);
    int64_t begin;
    if (!paged_cut(w, min_cost, begin)) return false;
    int64_t rem = begin - (incl - mine);
    const int src = __ffs(__ballot_sync(0xffffffffu, rem >= 0 && rem < mine)) - 1;
    int i = __shfl_sync(0xffffffffu, lane * per, src);
    rem = __shfl_sync(0xffffffffu, rem, src);
#pragma unroll 1
    while (i + 1 < p.B && rem >= costs[i]) rem -= costs[i++];
    fence_proxy_async_smem();
    w.i = i;
    w.s = paged_seq(p, i);
    paged_start(p, rem, w);
    return true;
}

// The same for up to 32 requests, one to a lane, by one warp alone, without the barrier and the second look at the
// request (one request of 1500 keys: 8.4 us against 8.7 us).
constexpr int kLaneRequests = 32;
template <int KT, int OVH>
__device__ __forceinline__ bool paged_share_lanes(const PagedParams& p, int min_cost, PagedWalk<KT, OVH>& w) {
    const int lane = int(lane_id());
    PagedSeq s{};
    if (lane < p.B) s = paged_seq(p, lane);
    const int64_t mine = s.n > 0 ? paged_head_cost<KT, OVH>(p, s) * p.Hkv : int64_t(0);
    int64_t incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    w.W = __shfl_sync(0xffffffffu, incl, 31);
    int64_t begin;
    if (!paged_cut(w, min_cost, begin)) return false;
    const int64_t rem = begin - (incl - mine);
    w.i = __ffs(__ballot_sync(0xffffffffu, rem >= 0 && rem < mine)) - 1;
    w.s.start = __shfl_sync(0xffffffffu, s.start, w.i);
    w.s.n = __shfl_sync(0xffffffffu, s.n, w.i);
    w.s.kv = __shfl_sync(0xffffffffu, s.kv, w.i);
    w.s.base = __shfl_sync(0xffffffffu, s.base, w.i);
    paged_start(p, __shfl_sync(0xffffffffu, rem, w.i), w);
    return true;
}

// The same for any batch: all threads of the block call it (NT threads, a whole number of warps), and
// every warp leaves with the same walk.
template <int KT, int OVH, int NT>
__device__ __forceinline__ bool paged_share_block(const PagedParams& p, int min_cost, int64_t* sh /* [NT / 32 + 2] */,
                                                  PagedWalk<KT, OVH>& w) {
    constexpr int NW = NT / 32;
    const int tid = int(threadIdx.x);
    int64_t mine = 0;
    for (int i = tid; i < p.B; i += NT) mine += paged_cost<KT, OVH>(p, i);
    block_prefix<NT>(mine, sh, w.W);
    int64_t begin;
    if (!paged_cut(w, min_cost, begin)) return false;
    // the request that holds `begin`: a running prefix, NT requests at a time
    if (tid == 0) sh[NW] = -1;
    int64_t run = 0;
    for (int a = 0; a < p.B; a += NT) {
        const int64_t cost = paged_cost<KT, OVH>(p, a + tid);
        int64_t total;
        const int64_t incl = run + block_prefix<NT>(cost, sh, total);
        if (begin >= incl - cost && begin < incl) {
            sh[NW] = a + tid;
            sh[NW + 1] = begin - (incl - cost);
        }
        run += total;
        if (begin < run) break;  // the same in all threads
    }
    __syncthreads();
    if (sh[NW] < 0) {  // lengths that changed under the kernel
        w.left = 0;
        return false;
    }
    w.i = int(sh[NW]);
    w.s = paged_seq(p, w.i);
    paged_start(p, sh[NW + 1], w);
    return true;
}

// Joins the pieces of cut units of both kernels of a call: a unit's rows are cut into blocks of NT groups of
// four elements, one to a thread; the blocks of the units that the CTAs of `a` opened come first, then
// those of `b`. Bound by latency: N pieces are read at a time, all their loads in flight together.
template <int D, int NT, int N>
__global__ void __launch_bounds__(NT) paged_join_kernel(const PagedParams p, const PagedParts a_parts, const PagedParts b_parts) {
    const int a_blocks = a_parts.ctas > 0 ? (a_parts.ctas - 1) * (a_parts.rows * D / (4 * NT)) : 0;
    const bool second = int(blockIdx.x) >= a_blocks;
    const PagedParts& w = second ? b_parts : a_parts;
    const int block = int(blockIdx.x) - (second ? a_blocks : 0), per = w.rows * D / (4 * NT);
    const int c = block / per;
    const int x = (block - c * per) * NT + int(threadIdx.x), r = x / (D / 4), col = (x % (D / 4)) * 4;
    grid_wait();
    grid_release();
    const PagedMeta u = w.meta[c];
    if (u.pieces == 0 || r >= u.rows) return;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int a = 0; a < u.pieces; a += N) {
        float2 ml[N];
        float4 y[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a + k < u.pieces) {
                const int64_t at = int64_t(a + k == 0 ? 2 * c + 1 : 2 * (c + a + k)) * w.rows + r;
                ml[k] = w.ml[at];
                y[k] = *reinterpret_cast<const float4*>(w.o + at * D + col);
            }
        }
        float mx = m;
#pragma unroll
        for (int k = 0; k < N; ++k) mx = fmaxf(mx, ml[k].x);
        const float neg = mx == -INFINITY ? 0.f : -mx;
        const float e0 = ex2(m + neg);  // 2^-inf = 0: nothing so far, or a piece that saw no key
        m = mx;
        l *= e0;
        o.x *= e0;
        o.y *= e0;
        o.z *= e0;
        o.w *= e0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float e = ex2(ml[k].x + neg);
            l += e * ml[k].y;
            o.x += e * y[k].x;
            o.y += e * y[k].y;
            o.z += e * y[k].z;
            o.w += e * y[k].w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // 0: no key; NaN scores stay NaN
    const int row = u.row0 + r / p.G, h = u.head * p.G + r % p.G;
    *reinterpret_cast<uint2*>(p.o + (int64_t(row) * p.H + h) * D + col) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (col == 0) p.lse[int64_t(h) * p.T + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Tensor map of a pool's keys or values, (64 elements, token, head, page, 64-element chunk), for copies
// of `rows` tokens of one page and head by `chunks` chunks (chunk after chunk), 128-byte swizzle.
bool encode_pages(CUtensorMap* map, const ulysses_kv_cache_t& c, const void* base, int rows, int chunks);

// The same of an 8-bit pool's codes, (d elements, token, head, page), swizzled by the row's length.
bool encode_code_pages(CUtensorMap* map, const ulysses_kv_cache_t& c, const void* base, int rows);

// Byte offset of 16-byte unit u of key r in a tile of D-byte rows: the 128-byte swizzle for d = 128, the 64-byte one for
// d = 64. Page copies are whole multiples of the swizzle's period, so the tile is one block whatever the page size.
template <int D>
__device__ __forceinline__ uint32_t code_offset(int r, int u) {
    return D == 128 ? uint32_t(r) * 128u + (uint32_t(u ^ (r & 7)) << 4) : uint32_t(r) * 64u + (uint32_t(u ^ ((r >> 1) & 3)) << 4);
}

// Requests of few rows (paged_decode.cu), and the others (paged_chunk.cu): where their pieces lie in a
// workspace on a device of `sms` SMs (`bytes` of it, whatever the device), and their launches.
int paged_decode_rows();
PagedParts paged_decode_parts(void* workspace, int d_h, int sms, size_t* bytes);
PagedParts paged_chunk_parts(void* workspace, int d_h, int sms, size_t* bytes);
int launch_paged_decode(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream);
int launch_paged_decode8(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream);
int launch_paged_chunk(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream);
int launch_paged_chunk8(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream);

// Pieces of `most` CTAs at the front of a workspace, for a launch of `ctas` of them.
inline PagedParts paged_parts(void* workspace, int most, int ctas, int rows, int d_h, size_t* bytes) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PagedParts w{};
    w.o = reinterpret_cast<float*>(ws);
    size_t at = size_t(2) * most * rows * d_h * 4;
    w.ml = reinterpret_cast<float2*>(ws + at);
    at += size_t(2) * most * rows * 8;
    w.meta = reinterpret_cast<PagedMeta*>(ws + at);
    at += size_t(most) * sizeof(PagedMeta);
    w.rows = rows;
    w.ctas = ctas < most ? ctas : most;
    *bytes = (at + 255) / 256 * 256;
    return w;
}

}  // namespace ulysses
