// New tokens' keys and values rounded to 8 bits into their slots (include/ulysses.h, "ulysses_kv_append8").
//
// A run is the consecutive rows of one block of tokens. For each run and head: the largest magnitude a, the scale 2^n
// with the smallest n for which a <= 448 * 2^n (448 = 1.75 * 2^8 is e4m3's largest: n is read off a's exponent and
// mantissa), then code = x * 2^-n rounded to the nearest. A power of two costs e4m3 nothing in precision, and every
// code * scale is exact in bf16, so that attention over the cache is attention over a bf16 cache of those values.
//
// Bound by reading rows (2 bytes an element) and writing codes (1). A group of d / 8 lanes takes one run of one head of
// keys or values, 16 bytes of a row to a lane; up to kRows rows stay in registers between the maximum and the rounding,
// longer runs are read a second time, out of the L2. All rows of a lane lie in the same column, and a lane rounds
// its column of a block's older tokens before it writes new ones there, so nothing has to wait for another lane. A block
// of threads looks for the first rows of runs in a window of `window` rows: one where there are few rows, for the
// latency, more where most rows only continue a run.
#include <algorithm>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

namespace {

constexpr int kThreads = 256, kRows = 16;
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

template <int D>
__global__ void __launch_bounds__(kThreads) kv_append8_kernel(const Append8Params p) {
    constexpr int LPG = D / 8;
    const int lane = int(threadIdx.x) & 31, col = (int(threadIdx.x) % LPG) * 8;
    const int pair = int(blockIdx.y) * (kThreads / LPG) + int(threadIdx.x) / LPG;
    const bool active = pair < 2 * p.heads;  // the others follow, for the whole warp's instructions
    const bool value = active && pair >= p.heads;
    const int head = active ? pair - (value ? p.heads : 0) : 0;
    const int64_t src_stride = p.src_stride[value];
    const __nv_bfloat16* src = p.src[value] + head * D + col;
    uint8_t* dst = p.dst[value] + head * p.head_stride + col;
    const int block = 1 << p.block_shift, page = 1 << p.page_shift;
    grid_wait();
    grid_release();
    const int t0 = int(blockIdx.x) * p.window, t1 = min(p.T, t0 + p.window);
    for (int t = t0; t < t1; ++t) {
        // the run that row t begins, if it does: its rows and whether one is the block's first token
        const int slot = p.slots[t], before = t > 0 ? p.slots[t - 1] : -1;
        if (unsigned(slot) >= unsigned(p.n_slots)) continue;
        const int b = slot >> p.block_shift;
        if (unsigned(before) < unsigned(p.n_slots) && before >> p.block_shift == b) continue;
        uint8_t* scale = p.scale[value] + int64_t(b) * p.heads + head;
        const int old = min(int(*scale), kMaxByte);
        int n = 0;
        bool fresh = false;
        for (;;) {
            const int64_t r = int64_t(t) + n + lane;
            const int s = r < p.T ? p.slots[r] : -1;
            const unsigned out = __ballot_sync(0xffffffffu, unsigned(s) >= unsigned(p.n_slots) || s >> p.block_shift != b);
            const int run = out ? __ffs(out) - 1 : 32;
            fresh |= __any_sync(0xffffffffu, lane < run && (s & (block - 1)) == 0);
            n += run;
            if (run < 32) break;
        }
        uint4 v[kRows];
        uint32_t top = 0;
        auto load = [&](int r0) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                v[i] = make_uint4(0, 0, 0, 0);
                if (active && r0 + i < n) v[i] = *reinterpret_cast<const uint4*>(src + (int64_t(t) + r0 + i) * src_stride);
            }
        };
        for (int r0 = 0; r0 < n; r0 += kRows) {
            load(r0);
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                top = max_abs2(max_abs2(max_abs2(max_abs2(top, v[i].x), v[i].y), v[i].z), v[i].w);
        }
#pragma unroll
        for (int o = 1; o < LPG; o <<= 1) top = max_abs2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int a = int(max(top & 0xffffu, top >> 16));  // bits of the largest: exponent above, 7 bits of mantissa
        const int need = min(max((a >> 7) - 8 + ((a & 127) > 96 ? 1 : 0), kMinByte), kMaxByte);
        const int now = fresh ? need : max(old, need);
        const int64_t first = int64_t(b) << p.block_shift;  // slot of the block's first token
        uint8_t* base = dst + (first >> p.page_shift) * p.page_stride + (first & (page - 1)) * p.token_stride;
        if (active && !fresh && now > old) {
            // factors below 2^-24 make zeros of every code, as 2^-126 does
            const float by = pow2f(max(old - now, -126));
            for (int i = 0; i < block; ++i) {
                uint2* c = reinterpret_cast<uint2*>(base + i * p.token_stride);
                const uint2 was = *c;
                *c = make_uint2(recode4(was.x, by), recode4(was.y, by));
            }
        }
        if (active && threadIdx.x % LPG == 0 && (fresh || now != old)) *scale = uint8_t(now);
        const float inv = pow2f(127 - now);
        for (int r0 = 0; r0 < n; r0 += kRows) {
            if (n > kRows) load(r0);
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (active && r0 + i < n)
                    *reinterpret_cast<uint2*>(base + (p.slots[t + r0 + i] & (block - 1)) * p.token_stride) = codes8(v[i], inv);
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
    const int groups = kThreads / (c.d_h / 8), y = (2 * c.H_kv + groups - 1) / groups;
    p.window = 1;
    while (p.window < 16 && int64_t(T) * y > int64_t(p.window) * 16 * device_sm_count()) p.window *= 2;
    if (y > 65535) return ULYSSES_ERR_UNSUPPORTED;
    const dim3 grid(unsigned((int64_t(T) + p.window - 1) / p.window), unsigned(y));
    return launch_chained(c.d_h == 128 ? kv_append8_kernel<128> : kv_append8_kernel<64>, grid, kThreads, 0, stream, p)
               ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace ulysses
