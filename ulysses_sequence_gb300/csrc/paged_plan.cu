// The index work and the cache writes of one serving step over a paged key/value cache
// (include/ulysses.h, "Serving from a paged key/value cache"): block tables and slot maps built
// from request lengths, and the new tokens' keys and values moved to their slots.
#include <algorithm>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

namespace {

// ---------------------------------------------------------------------------------------
// page_plan. Two prefix sums over the requests: row starts cu (saturating at T) and new pages
// before each request A. Every CTA computes both for itself in shared memory (B <= 8192
// requests: three int32 arrays of at most 96 KB), which costs less than a second launch or a
// wait between CTAs; then tokens and new pages are spread evenly over all threads of the grid,
// each finding its request by binary search, so one long prompt among short ones does not
// leave the grid idle. Nothing a CTA reads is written by another: tokens on new pages take the
// page from the free list, not from the table.
// ---------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

struct PlanParams {
    int B, T, page_shift, max_pages, num_pages, free_capacity;
    int64_t table_stride;
    const int32_t *cached, *fresh, *free_pages, *n_free;
    int32_t *table, *cu_q, *kv_lens, *slots, *info;
};

// Inclusive prefix of v over the block with + saturating at `cap` (v, cap <= 2^31 - 1, so a sum
// of two fits 32 unsigned bits). `total` receives the block's sum.
__device__ __forceinline__ uint32_t block_scan_sat(uint32_t v, uint32_t cap, uint32_t* warp_sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = min(v + y, cap);
    }
    if (lane == 31) warp_sums[w] = v;
    __syncthreads();
    if (w == 0) {
        uint32_t s = lane < kPlanThreads / 32 ? warp_sums[lane] : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s = min(s + y, cap);
        }
        if (lane < kPlanThreads / 32) warp_sums[lane] = s;
    }
    __syncthreads();
    if (w > 0) v = min(v + warp_sums[w - 1], cap);
    total = warp_sums[kPlanThreads / 32 - 1];
    __syncthreads();
    return v;
}

// x[0 .. n) -> its exclusive prefix, x[n] = the sum; each thread owns a run of entries.
__device__ __forceinline__ void scan_array(int32_t* x, int n, uint32_t cap, uint32_t* warp_sums) {
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int a = min(n, int(threadIdx.x) * per), e = min(n, a + per);
    uint32_t sum = 0;
    for (int i = a; i < e; ++i) sum = min(sum + uint32_t(x[i]), cap);
    uint32_t total;
    const uint32_t incl = block_scan_sat(sum, cap, warp_sums, total);
    // the exclusive prefix: the inclusive one of the thread before (a saturated sum cannot be
    // taken apart by subtraction)
    uint32_t run = __shfl_up_sync(0xffffffffu, incl, 1);
    __shared__ uint32_t ends[kPlanThreads / 32];
    if ((threadIdx.x & 31) == 31) ends[threadIdx.x >> 5] = incl;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) run = threadIdx.x == 0 ? 0u : ends[(threadIdx.x >> 5) - 1];
    for (int i = a; i < e; ++i) {
        const uint32_t v = uint32_t(x[i]);
        x[i] = int32_t(run);
        run = min(run + v, cap);
    }
    if (threadIdx.x == 0) x[n] = int32_t(total);
    __syncthreads();
}

// The last i with start[i] <= x: the request that holds row (or new page) x; requests of length
// zero share a start with their successor and are passed over. start[0] = 0 <= x < start[n].
__device__ __forceinline__ int owner(const int32_t* start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
    extern __shared__ int32_t plan_smem[];
    int32_t* cu = plan_smem;             // [B + 1] row starts
    int32_t* pg = cu + p.B + 1;          // [B + 1] new pages before each request
    int32_t* held = pg + p.B + 1;        // [B] cached tokens, clamped
    __shared__ uint32_t warp_sums[kPlanThreads / 32];
    grid_wait();
    grid_release();
    const int page = 1 << p.page_shift;
    const int cap = p.max_pages << p.page_shift;
    // pages of n tokens: n may be 2^31 - 1, so the sum is unsigned
    auto pages_of = [&](int n) { return int((uint32_t(n) + uint32_t(page - 1)) >> p.page_shift); };
    const int n_free = min(max(*p.n_free, 0), p.free_capacity);

    for (int i = threadIdx.x; i < p.B; i += kPlanThreads) {
        held[i] = min(max(p.cached[i], 0), cap);
        cu[i] = min(max(p.fresh[i], 0), p.T);
    }
    __syncthreads();
    scan_array(cu, p.B, uint32_t(p.T), warp_sums);
    for (int i = threadIdx.x; i < p.B; i += kPlanThreads) {
        const int c = held[i], kv = c + cu[i + 1] - cu[i];
        pg[i] = min(pages_of(kv), p.max_pages) - pages_of(c);
    }
    __syncthreads();
    scan_array(pg, p.B, 0x7fffffffu, warp_sums);
    const int rows = cu[p.B], pages = pg[p.B];

    // new page number x of the step
    auto taken = [&](int x) {
        if (x >= n_free) return -1;
        const int id = p.free_pages[n_free - 1 - x];
        return unsigned(id) < unsigned(p.num_pages) ? id : -1;
    };
    const int64_t first = int64_t(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int64_t step = int64_t(gridDim.x) * kPlanThreads;
    for (int64_t t = first; t < p.T; t += step) {
        int slot = -1;
        if (t < rows) {
            const int i = owner(cu, p.B, int(t));
            const int c = held[i], pos = c + int(t) - cu[i], at = pos >> p.page_shift;
            const int has = pages_of(c);
            if (at < p.max_pages) {
                const int id = at < has ? p.table[i * p.table_stride + at] : taken(pg[i] + at - has);
                if (unsigned(id) < unsigned(p.num_pages)) slot = (id << p.page_shift) + (pos & (page - 1));
            }
        }
        p.slots[t] = slot;
    }
    for (int64_t x = first; x < pages; x += step) {
        const int i = owner(pg, p.B, int(x));
        const int has = pages_of(held[i]);
        p.table[i * p.table_stride + has + (int(x) - pg[i])] = taken(int(x));
    }
    if (blockIdx.x != 0) return;

    for (int i = threadIdx.x; i <= p.B; i += kPlanThreads) {
        p.cu_q[i] = cu[i];
        if (i < p.B) p.kv_lens[i] = held[i] + cu[i + 1] - cu[i];
    }
    // what was asked for and is not there: pages past the table's width, tokens past row T
    int beyond = 0;
    unsigned long long asked = 0;
    for (int i = threadIdx.x; i < p.B; i += kPlanThreads) {
        const int kv = held[i] + cu[i + 1] - cu[i];
        beyond += max(0, pages_of(kv) - p.max_pages);
        asked += static_cast<unsigned long long>(max(p.fresh[i], 0));
    }
    __shared__ int sh_beyond;
    __shared__ unsigned long long sh_asked;
    if (threadIdx.x == 0) {
        sh_beyond = 0;
        sh_asked = 0;
    }
    __syncthreads();
    beyond = __reduce_add_sync(0xffffffffu, beyond);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) asked += __shfl_down_sync(0xffffffffu, asked, o);
    if ((threadIdx.x & 31) == 0) {  // whole numbers: the order of the adds does not matter
        atomicAdd(&sh_beyond, beyond);
        atomicAdd(&sh_asked, asked);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned long long dropped = sh_asked - static_cast<unsigned long long>(rows);
        p.info[0] = rows;
        p.info[1] = min(pages, n_free);
        p.info[2] = sh_beyond + max(0, pages - n_free);
        p.info[3] = dropped > 0x7fffffffull ? 0x7fffffff : int(dropped);
    }
}

// ---------------------------------------------------------------------------------------
// kv_append: rows moved by slot with nothing to compute, bound by its reads and writes (one each of
// 4 H_kv d_h bytes a token). A CTA moves 16-byte pieces of consecutive tokens, U per thread, all of a
// thread's loads in flight before its first store; grid row 0 moves keys, row 1 values. Many pieces per
// thread pay when there are many (starting a CTA costs more than its few copies: 32768 tokens of 8 heads
// of 128 take 41.6 us with 16 pieces, 6.45 TB/s, and 76 us with two), few when there are few (128 tokens:
// 1.5 us with two, 2.8 us with 16); the two meet near 768 tokens.
// ---------------------------------------------------------------------------------------
constexpr int kAppendThreads = 128, kAppendFew = 2, kAppendMany = 16;
constexpr int64_t kAppendManyPieces = 48 * kAppendThreads * kAppendMany;  // from here on, by key rows' pieces

// n / d for n < 2^31 by a multiplication, after Granlund and Montgomery ("Division by invariant integers using
// multiplication", 1994): with 2^(s-1) < d <= 2^s and m = floor(2^32 (2^s - d) / d) + 1, the quotient is
// floor((floor(n m / 2^32) + n) / 2^s).
struct FastDiv {
    uint32_t d, m, s;
    explicit FastDiv(uint32_t div = 1) : d(div), m(0), s(0) {
        while ((uint64_t(1) << s) < d) ++s;
        m = uint32_t((((uint64_t(1) << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

struct AppendParams {
    const uint4* src[2];
    uint4* dst[2];
    int64_t src_stride[2];          // 16-byte pieces between rows
    int64_t page_stride, token_stride, head_stride;  // 16-byte pieces
    const int32_t* slots;
    int64_t pieces;                 // T * row pieces
    FastDiv row, head;              // pieces of a token, of a head
    int page_shift;
    int n_slots;                    // num_pages * page_size
};

template <int U>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    const int64_t base = int64_t(blockIdx.x) * (kAppendThreads * U);
    const int64_t t0 = p.pieces < (int64_t(1) << 31) ? int64_t(p.row(uint32_t(base))) : base / p.row.d;
    const uint32_t r0 = uint32_t(base - t0 * p.row.d) + threadIdx.x;
    const bool key = blockIdx.y == 0;
    const uint4* src = key ? p.src[0] : p.src[1];
    uint4* dst = key ? p.dst[0] : p.dst[1];
    const int64_t src_stride = key ? p.src_stride[0] : p.src_stride[1];
    uint4 v[U];
    uint32_t c[U];
    int slot[U];
    grid_wait();
    grid_release();
    // rows and slots together: a skipped token's row is read all the same
#pragma unroll
    for (int u = 0; u < U; ++u) {
        slot[u] = -1;
        const uint32_t r = r0 + u * kAppendThreads, dt = p.row(r);
        c[u] = r - dt * p.row.d;
        if (base + threadIdx.x + u * kAppendThreads < p.pieces) {
            slot[u] = p.slots[t0 + dt];
            v[u] = src[(t0 + dt) * src_stride + c[u]];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (unsigned(slot[u]) < unsigned(p.n_slots)) {
            const uint32_t h = p.head(c[u]), e = c[u] - h * p.head.d;
            const int page = slot[u] >> p.page_shift, token = slot[u] & ((1 << p.page_shift) - 1);
            dst[page * p.page_stride + token * p.token_stride + h * p.head_stride + e] = v[u];
        }
    }
}

}  // namespace

int launch_page_plan(int B, int T, int page_shift, int max_pages, int64_t table_stride, int num_pages,
                     const int32_t* cached, const int32_t* fresh, const int32_t* free_pages, int free_capacity,
                     const int32_t* n_free, int32_t* table, int32_t* cu_q, int32_t* kv_lens, int32_t* slots,
                     int32_t* info, cudaStream_t stream) {
    PlanParams p{B, T, page_shift, max_pages, num_pages, free_capacity, table_stride, cached, fresh, free_pages, n_free,
                 table, cu_q, kv_lens, slots, info};
    const int smem = (3 * B + 2) * int(sizeof(int32_t));
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(page_plan_kernel), (3 * kPlanMaxB + 2) * int(sizeof(int32_t))))
        return ULYSSES_ERR_CUDA;
    const int64_t want = (int64_t(T) + kPlanThreads - 1) / kPlanThreads;
    const int grid = int(std::max<int64_t>(1, std::min<int64_t>(want, device_sm_count())));
    return launch_chained(page_plan_kernel, dim3(unsigned(grid)), kPlanThreads, size_t(smem), stream, p) ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

int launch_kv_append(const ulysses_kv_cache_t& c, int T, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, const int32_t* slots, cudaStream_t stream) {
    AppendParams p{};
    p.src[0] = static_cast<const uint4*>(k);
    p.src[1] = static_cast<const uint4*>(v);
    p.dst[0] = static_cast<uint4*>(c.k);
    p.dst[1] = static_cast<uint4*>(c.v);
    p.src_stride[0] = k_stride / 8;
    p.src_stride[1] = v_stride / 8;
    p.page_stride = c.page_stride / 8;
    p.token_stride = c.token_stride / 8;
    p.head_stride = c.head_stride / 8;
    p.slots = slots;
    p.head = FastDiv(uint32_t(c.d_h / 8));
    p.row = FastDiv(uint32_t(c.H_kv) * p.head.d);
    p.pieces = int64_t(T) * p.row.d;
    p.page_shift = __builtin_ctz(unsigned(c.page_size));
    p.n_slots = c.num_pages * c.page_size;
    const bool many = p.pieces >= kAppendManyPieces;
    const int64_t per = kAppendThreads * (many ? kAppendMany : kAppendFew), blocks = (p.pieces + per - 1) / per;
    if (blocks > 0x7fffffffll) return ULYSSES_ERR_UNSUPPORTED;
    return launch_chained(many ? kv_append_kernel<kAppendMany> : kv_append_kernel<kAppendFew>, dim3(unsigned(blocks), 2),
                          kAppendThreads, 0, stream, p) ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace ulysses
