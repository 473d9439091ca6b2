// New tokens' keys and values rounded to 8 bits into their slots (include/ulysses.h, "ulysses_kv_append8").
//
// A run is the consecutive rows of one block of tokens. For each run and head: the largest magnitude a, the scale 2^n
// with the smallest n for which a <= 448 * 2^n (448 = 1.75 * 2^8 is e4m3's largest: n is read off a's exponent and
// mantissa), then code = x * 2^-n rounded to the nearest. A power of two costs e4m3 nothing in precision, and every
// code * scale is exact in bf16, so that attention over the cache is attention over a bf16 cache of those values.
//
// Bound by reading rows (2 bytes an element) and writing codes (1). A group of d / 8 lanes takes rows of one head of keys
// or values, 16 bytes of a row to a lane, and holds them in registers between the maximum and the rounding. Runs of
// blocks of more than 16 tokens are shared by kParts groups, 64 rows in all, whose maxima meet in shared memory; longer
// ones, and those of a group alone that pass its rows, are read a second time, out of the L2. 32761 tokens of 8 heads of
// 128 in blocks of 64 take 37 us, 5.4 TB/s; by single groups of 16 rows 52 us, by four groups 40 us; 64 single tokens
// 2.4 us, with 16 rows to a group instead of four 3.1 us. A block of threads looks for the first rows of runs in a window
// of `window` rows: one where there are few rows, for the latency, more where most rows only continue a run.
#include <algorithm>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

namespace {

constexpr int kThreads = 256, kParts = 8;
constexpr int kMinByte = 10, kMaxByte = 246;  // 2^-117 and 2^119

struct Append8Params {
    const __nv_bfloat16* src[2];
    uint8_t* dst[2];
    uint8_t* scale[2];
    int64_t src_stride[2];                           // elements between rows
    int64_t page_stride, token_stride, head_stride;  // bytes
    const int32_t* slots;
    int T, heads, n_slots, window;
    int page_shift, block_shift;
};

// e4m3 of a pair, to the nearest even, past 448 to 448; the second in the upper byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__uint_as_float(r[i] << 16) * inv, __uint_as_float(r[i] & 0xffff0000u) * inv);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Four codes times a power of two (at most 1), rounded again. The products are exact in fp32.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float by) {
    uint32_t h0, h1;
    e4m3_to_f16(c, h0, h1);
    const float2 a = __half22float2(reinterpret_cast<const __half2&>(h0)), b = __half22float2(reinterpret_cast<const __half2&>(h1));
    return e4m3x2(a.x * by, a.y * by) | e4m3x2(b.x * by, b.y * by) << 16;
}

template <int D, int PARTS, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_append8_kernel(const Append8Params p) {
    constexpr int LPG = D / 8, GROUPS = kThreads / LPG;
    __shared__ uint32_t tops[GROUPS];
    const int lane = int(threadIdx.x) & 31, col = (int(threadIdx.x) % LPG) * 8;
    const int group = int(threadIdx.x) / LPG, part = group % PARTS;
    const int pair = int(blockIdx.y) * (GROUPS / PARTS) + group / PARTS;
    const bool active = pair < 2 * p.heads;  // the others follow, for the whole warp's instructions
    const bool value = active && pair >= p.heads;
    const int head = active ? pair - (value ? p.heads : 0) : 0;
    // selected by value: an index into the parameters would copy them to local memory
    const int64_t src_stride = value ? p.src_stride[1] : p.src_stride[0];
    const __nv_bfloat16* src = (value ? p.src[1] : p.src[0]) + head * D + col;
    uint8_t* dst = (value ? p.dst[1] : p.dst[0]) + head * p.head_stride + col;
    const int block = 1 << p.block_shift, page = 1 << p.page_shift;
    grid_wait();
    grid_release();
    const int t0 = int(blockIdx.x) * p.window, t1 = min(p.T, t0 + p.window);
    for (int a = t0; a < t1; a += 32) {
        // the rows of the window that begin a run, 32 looked at at a time
        unsigned heads;
        {
            const int t = a + lane;
            const int s = t < t1 ? p.slots[t] : -1, before = t > 0 && t < t1 ? p.slots[t - 1] : -1;
            const bool in = unsigned(s) < unsigned(p.n_slots), joins = unsigned(before) < unsigned(p.n_slots) && before >> p.block_shift == s >> p.block_shift;
            heads = __ballot_sync(0xffffffffu, in && !joins);
        }
        for (; heads; heads &= heads - 1) {
            const int t = a + __ffs(heads) - 1;
            uint4 v[ROWS];
            auto load = [&](int r0, int n) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (active && r0 + i < n) v[i] = *reinterpret_cast<const uint4*>(src + (int64_t(t) + r0 + i) * src_stride);
                }
            };
            // a long run is likely where rows are shared: they are on their way before it is known how many there are
            if (PARTS > 1) load(part * ROWS, p.T - t);
            const int b = p.slots[t] >> p.block_shift;
            uint8_t* scale = (value ? p.scale[1] : p.scale[0]) + int64_t(b) * p.heads + head;
            const int old = min(int(*scale), kMaxByte);
            // the run: its rows, and whether one is the block's first token
            int n = 0;
            bool fresh = false;
            for (bool more = true; more;) {
                constexpr int AHEAD = PARTS > 1 ? 3 : 1;  // slots looked at at a time, by 32
                int s[AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const int64_t r = int64_t(t) + n + 32 * k + lane;
                    s[k] = r < p.T ? p.slots[r] : -1;
                }
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const unsigned out = __ballot_sync(0xffffffffu, unsigned(s[k]) >= unsigned(p.n_slots) || s[k] >> p.block_shift != b);
                    const int run = !more ? 0 : out ? __ffs(out) - 1 : 32;
                    fresh |= __any_sync(0xffffffffu, lane < run && (s[k] & (block - 1)) == 0);
                    n += run;
                    more = more && run == 32;
                }
            }
            if (PARTS == 1) load(0, n);
            uint32_t top = 0;
            for (int r0 = part * ROWS;;) {
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
                    if (r0 + i < n) top = max_abs2(max_abs2(max_abs2(max_abs2(top, v[i].x), v[i].y), v[i].z), v[i].w);
                r0 += PARTS * ROWS;
                if (r0 >= n) break;
                load(r0, n);
            }
#pragma unroll
            for (int o = 1; o < LPG; o <<= 1) top = max_abs2(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (PARTS > 1) {
                if (threadIdx.x % LPG == 0) tops[group] = top;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < PARTS; ++k) top = max_abs2(top, tops[group - part + k]);
            }
            const int bits = int(max(top & 0xffffu, top >> 16));  // of the largest: exponent above, 7 bits of mantissa
            const int need = min(max((bits >> 7) - 8 + ((bits & 127) > 96 ? 1 : 0), kMinByte), kMaxByte);
            const int now = fresh ? need : max(old, need);
            const int64_t first = int64_t(b) << p.block_shift;  // slot of the block's first token
            uint8_t* base = dst + (first >> p.page_shift) * p.page_stride + (first & (page - 1)) * p.token_stride;
            if (active && !fresh && now > old) {
                // factors below 2^-24 make zeros of every code, as 2^-126 does
                const float by = pow2f(max(old - now, -126));
                for (int i = part; i < block; i += PARTS) {
                    uint2* c = reinterpret_cast<uint2*>(base + i * p.token_stride);
                    const uint2 was = *c;
                    *c = make_uint2(recode4(was.x, by), recode4(was.y, by));
                }
            }
            if (PARTS > 1) __syncthreads();  // new codes go over what another part has rounded
            if (active && part == 0 && threadIdx.x % LPG == 0 && (fresh || now != old)) *scale = uint8_t(now);
            const float inv = pow2f(127 - now);
            for (int r0 = part * ROWS; r0 < n; r0 += PARTS * ROWS) {
                if (n > PARTS * ROWS) load(r0, n);
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
                    if (active && r0 + i < n)
                        *reinterpret_cast<uint2*>(base + (p.slots[t + r0 + i] & (block - 1)) * p.token_stride) = codes8(v[i], inv);
            }
        }
    }
}

}  // namespace

int launch_kv_append8(const ulysses_kv_cache8_t& c, int T, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      const int32_t* slots, cudaStream_t stream) {
    Append8Params p{};
    p.src[0] = static_cast<const __nv_bfloat16*>(k);
    p.src[1] = static_cast<const __nv_bfloat16*>(v);
    p.dst[0] = static_cast<uint8_t*>(c.k);
    p.dst[1] = static_cast<uint8_t*>(c.v);
    p.scale[0] = c.k_scale;
    p.scale[1] = c.v_scale;
    p.src_stride[0] = k_stride;
    p.src_stride[1] = v_stride;
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    p.slots = slots;
    p.T = T;
    p.heads = c.H_kv;
    p.n_slots = c.num_pages * c.page_size;
    p.page_shift = __builtin_ctz(unsigned(c.page_size));
    p.block_shift = __builtin_ctz(unsigned(c.block));
    // Few rows are mostly single tokens: short groups, for the latency. From 1025 rows on runs are taken to be long, which the
    // host does not know: 32761 tokens of one prompt, 8 heads of 128 in blocks of 64, take 36.8 us shared by kParts groups, 52 us
    // by groups of 16 rows, 56 us by those of four. Single tokens lose by it: 1500 of them take 50 us, 14.5 and 6.3 us, 6000 take
    // 196, 49 and 20 us.
    const int groups = kThreads / (c.d_h / 8);
    const bool parts = c.block > 16 && T > 1024;
    const int y = (2 * c.H_kv * (parts ? kParts : 1) + groups - 1) / groups;
    if (y > 65535) return ULYSSES_ERR_UNSUPPORTED;
    p.window = 1;
    while (p.window < std::max(16, std::min(c.block, 64)) && int64_t(T) * y > int64_t(p.window) * 16 * device_sm_count()) p.window *= 2;
    const dim3 grid(unsigned((int64_t(T) + p.window - 1) / p.window), unsigned(y));
    auto kern = c.d_h == 128 ? kv_append8_kernel<128, 1, 4> : kv_append8_kernel<64, 1, 4>;
    if (parts) kern = c.d_h == 128 ? kv_append8_kernel<128, kParts, 64 / kParts> : kv_append8_kernel<64, kParts, 64 / kParts>;
    else if (T > 1024) kern = c.d_h == 128 ? kv_append8_kernel<128, 1, 16> : kv_append8_kernel<64, 1, 16>;
    return launch_chained(kern, grid, kThreads, 0, stream, p) ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace ulysses
