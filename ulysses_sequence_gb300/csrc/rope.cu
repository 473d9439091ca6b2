// Rotary positions of queries and keys, with the RMS norm of every head in the same pass, forward and backward.
//
// With x a head of d elements, its first `rot` elements cut into pairs (x_e, x_{e + rot/2}), or (x_2e, x_{2e+1}):
//   forward   z = w * x / sqrt(mean x^2 + eps) (or z = x without weights),  y = R z,
//             R: (a, b) -> A (a cos - b sin, b cos + a sin) with the angle p f_e of the pair and an amplitude A;
//   backward  dz = R^T dy,  g = w dz,  r = 1 / sqrt(mean x^2 + eps),  dx = r (g - r x mean(g r x)),
//             dw = sum over tokens and heads of dz r x.
// Angles: f_e comes as turns a token in units of 2^-64, so that the product with the position, kept to 64 bits, is the
// angle modulo one turn to 2^-34 turns at positions below 2^31, without a division or a 64-bit float. Its upper 32 bits,
// rounded to the 24 of fp32, go through sincospi: the angle used is off by up to 2^-26 turns (2^-23 radians), far below
// the outputs' bf16.
//
// Bound by reading and writing the heads once. A warp takes a row's heads D / 16 lanes to a head: a lane holds 16
// elements as two 16-byte pieces that are the two sides of its 8 pairs (or neighbours), so that pairs never leave the
// lane and the norm is three (two) shuffles. The row's cosines and sines are computed once a row, D / 64 of them to a lane,
// and handed round by shuffles. blockIdx.y names a part of the heads of q or k, so that weights and their
// gradients stay in registers while a warp goes down its rows. 32768 tokens of 32 + 8 heads of 128 with norms take 106 us
// forward (6.4 TB/s, 0.94 of the measured copy bandwidth) and 169 us backward (6.0 TB/s). Gradients of weights are summed in fp32 in a fixed order: by
// lane, by warp, by block into the workspace, and over the blocks by a second kernel, so they do not vary.
#include <algorithm>

#include "common.cuh"
#include "ulysses_internal.h"

namespace ulysses {

namespace {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBwdCtas = 1024;  // bounds the partial sums in the workspace

template <int D>
struct RopeCfg {
    static constexpr int LPH = D / 16;      // lanes of a head
    static constexpr int HPW = 32 / LPH;    // heads of a pass
    static constexpr int PPL = D / 64;      // pairs whose angle a lane computes
};

struct RopeSide {          // q or k
    const __nv_bfloat16* x;   // forward: input; backward: the forward's input (with weights)
    const __nv_bfloat16* dy;  // backward
    __nv_bfloat16* out;
    const void* w;            // nullptr: no norm
    float* dw;
    int64_t x_stride, out_stride;  // elements between rows
    int heads, chunks, passes;  // passes of a chunk
};

struct RopeParams {
    RopeSide side[2];
    const uint64_t* turns;
    int rot;
    float amplitude, sign;  // of the sine: -1 turns back
    float eps;
    int wide;               // weights are fp32
    int rows;
    // positions: given, or of the request that owns the row, or by place in a shard
    const int32_t* positions;
    const int32_t *cu_q, *kv_lens;
    int B;
    int64_t pos0;
    int seg, shard_rows;    // row m: pos0 + m % seg + m / shard_rows * shard_step
    int64_t shard_step;
    float* partial;         // [blockIdx.y][gridDim.x][D]
};

// The position of row m; false where the row belongs to no request. Called by whole warps.
__device__ __forceinline__ bool rope_position(const RopeParams& p, int m, int64_t& pos) {
    if (p.positions) {
        pos = p.positions[m];
        return true;
    }
    if (!p.cu_q) {
        pos = p.pos0 + m % p.seg + m / p.shard_rows * p.shard_step;
        return true;
    }
    // how many requests end at or before the row: 32 ends looked at at a time
    const int lane = int(lane_id());
    int lo = 0, hi = p.B;
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5;
        const int64_t at = int64_t(lo) + int64_t(lane) * step;
        const int ends = __popc(__ballot_sync(0xffffffffu, at < hi && p.cu_q[at + 1] <= m));
        if (ends == 0) break;
        hi = int(min(int64_t(hi), int64_t(lo) + int64_t(ends) * step));
        lo += (ends - 1) * step + 1;
    }
    if (lo >= p.B || p.cu_q[lo] > m) return false;
    const int len = min(max(p.kv_lens[lo], 0), kPagedMaxLen);
    pos = int64_t(len) - (min(p.cu_q[lo + 1], p.rows) - m);
    return true;
}

// cos and sin of the lane's 8 pairs; `f` holds the turns of its own D / 64.
template <int D>
__device__ __forceinline__ void rope_angles(const RopeParams& p, const uint64_t* f, int64_t pos, float* c, float* s) {
    using C = RopeCfg<D>;
    float cs[C::PPL], sn[C::PPL];
#pragma unroll
    for (int x = 0; x < C::PPL; ++x) {
        const int32_t turn = int32_t((f[x] * uint64_t(pos) + 0x80000000ull) >> 32);  // of 2^32
        sincospif(float(turn) * 4.656612873077393e-10f, &sn[x], &cs[x]);               // 2^-31: half turns
        cs[x] *= p.amplitude;
        sn[x] *= p.amplitude * p.sign;
    }
    const int j8 = (int(lane_id()) % C::LPH) * (8 / C::PPL);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = __shfl_sync(0xffffffffu, cs[i % C::PPL], j8 + i / C::PPL);
        s[i] = __shfl_sync(0xffffffffu, sn[i % C::PPL], j8 + i / C::PPL);
    }
}

// A lane's 16 elements as pairs of neighbours, the first piece's four and the second's: two fp32 operations to an
// instruction.
__device__ __forceinline__ void unpack8(const uint4& v, float2* f) {
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2* f) {
    return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
}

template <bool INTER>
__device__ __forceinline__ void rope_turn(float2* v, const float* c, const float* s) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i)  // v[i] = (a, b)
            v[i] = fma2(v[i], make_float2(c[i], c[i]), mul2(make_float2(v[i].y, v[i].x), make_float2(-s[i], s[i])));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a of two pairs in v[i], b in v[4 + i]
            const float2 a = v[i], b = v[4 + i], cc = make_float2(c[2 * i], c[2 * i + 1]), ss = make_float2(s[2 * i], s[2 * i + 1]);
            v[i] = fma2(a, cc, mul2(b, make_float2(-ss.x, -ss.y)));
            v[4 + i] = fma2(b, cc, mul2(a, ss));
        }
    }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean x^2 + eps) of the lane's head
template <int D>
__device__ __forceinline__ float inverse_rms(const float2* x, float eps) {
    float2 ss = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) ss = fma2(x[i], x[i], ss);
    return rsqrtf(head_sum<RopeCfg<D>::LPH>(ss.x + ss.y) * (1.0f / D) + eps);
}

__device__ __forceinline__ void load_weights(const void* w, int wide, int at, float2* out) {
    if (wide) {
        const float* f = static_cast<const float*>(w) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = make_float2(f[2 * i], f[2 * i + 1]);
    } else {
        const __nv_bfloat16* f = static_cast<const __nv_bfloat16*>(w) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = make_float2(__bfloat162float(f[2 * i]), __bfloat162float(f[2 * i + 1]));
    }
}

// What a lane has to know of its place: its head within a pass and its two pieces within a head.
template <int D, bool INTER>
struct RopeLane {
    int g, ea, eb;
    bool turned;
    __device__ __forceinline__ explicit RopeLane(int rot) {
        const int lane = int(lane_id()), j = lane % RopeCfg<D>::LPH;
        g = lane / RopeCfg<D>::LPH;
        turned = 16 * j < rot;
        ea = INTER || !turned ? 16 * j : 8 * j;
        eb = INTER || !turned ? 16 * j + 8 : rot / 2 + 8 * j;
    }
};

template <int D>
__device__ __forceinline__ void load_turns(const RopeParams& p, uint64_t* f) {
#pragma unroll
    for (int x = 0; x < RopeCfg<D>::PPL; ++x) {
        const int at = int(lane_id()) * RopeCfg<D>::PPL + x;
        f[x] = at < p.rot / 2 ? p.turns[at] : 0;
    }
}

// A warp goes through its chunk's passes U at a time; U passes' loads go out together, the first before the angles are known.
template <int D, bool NORM, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_fwd_kernel(const RopeParams p) {
    using C = RopeCfg<D>;
    const bool key = int(blockIdx.y) >= p.side[0].chunks;
    const RopeSide& t = p.side[key ? 1 : 0];
    const int begin = (int(blockIdx.y) - (key ? p.side[0].chunks : 0)) * t.passes * C::HPW;
    const int end = min(t.heads, begin + t.passes * C::HPW);
    const RopeLane<D, INTER> at(p.rot);
    grid_wait();
    grid_release();
    uint64_t f[C::PPL];
    load_turns<D>(p, f);
    float2 w[8];
    if (NORM) {
        load_weights(t.w, p.wide, at.ea, w);
        load_weights(t.w, p.wide, at.eb, w + 4);
    }
    for (int64_t m = int64_t(blockIdx.x) * kRopeWarps + warp_id(); m < p.rows; m += int64_t(gridDim.x) * kRopeWarps) {
        const __nv_bfloat16* src = t.x + m * t.x_stride;
        __nv_bfloat16* dst = t.out + m * t.out_stride;
        uint4 v[U][2];
        auto load = [&](int first) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = first + u * C::HPW + at.g;
                v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
                if (h < end) {
                    v[u][0] = *reinterpret_cast<const uint4*>(src + h * D + at.ea);
                    v[u][1] = *reinterpret_cast<const uint4*>(src + h * D + at.eb);
                }
            }
        };
        load(begin);
        int64_t pos;
        if (!rope_position(p, int(m), pos)) continue;
        float c[8], s[8];
        rope_angles<D>(p, f, pos, c, s);
        for (int first = begin;;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = first + u * C::HPW + at.g;
                float2 x[8];
                unpack8(v[u][0], x);
                unpack8(v[u][1], x + 4);
                if (NORM) {
                    const float r = inverse_rms<D>(x, p.eps);
                    const float2 rr = make_float2(r, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = mul2(mul2(x[i], rr), w[i]);
                }
                if (at.turned) rope_turn<INTER>(x, c, s);
                if (h < end) {
                    *reinterpret_cast<uint4*>(dst + h * D + at.ea) = pack8(x);
                    *reinterpret_cast<uint4*>(dst + h * D + at.eb) = pack8(x + 4);
                }
            }
            first += U * C::HPW;
            if (first >= end) break;
            load(first);
        }
    }
}

// The gradient through the norm: x and dy in, dx out, the weights' gradients to the block's row of `partial`.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_norm_bwd_kernel(const RopeParams p) {
    using C = RopeCfg<D>;
    const bool key = int(blockIdx.y) >= p.side[0].chunks;
    const RopeSide& t = p.side[key ? 1 : 0];
    const int first = (int(blockIdx.y) - (key ? p.side[0].chunks : 0)) * U * C::HPW;
    const RopeLane<D, INTER> at(p.rot);
    grid_wait();
    grid_release();
    uint64_t f[C::PPL];
    load_turns<D>(p, f);
    float2 w[8], dw[8];
    load_weights(t.w, p.wide, at.ea, w);
    load_weights(t.w, p.wide, at.eb, w + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = make_float2(0.f, 0.f);
    for (int64_t m = int64_t(blockIdx.x) * kRopeWarps + warp_id(); m < p.rows; m += int64_t(gridDim.x) * kRopeWarps) {
        uint4 v[U][2], y[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = first + u * C::HPW + at.g;
            v[u][0] = v[u][1] = y[u][0] = y[u][1] = make_uint4(0, 0, 0, 0);
            if (h < t.heads) {
                const int64_t row = m * t.x_stride + h * D;
                y[u][0] = *reinterpret_cast<const uint4*>(t.dy + row + at.ea);
                y[u][1] = *reinterpret_cast<const uint4*>(t.dy + row + at.eb);
                v[u][0] = *reinterpret_cast<const uint4*>(t.x + row + at.ea);
                v[u][1] = *reinterpret_cast<const uint4*>(t.x + row + at.eb);
            }
        }
        int64_t pos;
        if (!rope_position(p, int(m), pos)) continue;
        float c[8], s[8];
        rope_angles<D>(p, f, pos, c, s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = first + u * C::HPW + at.g;
            float2 x[8], g[8];
            unpack8(v[u][0], x);
            unpack8(v[u][1], x + 4);
            unpack8(y[u][0], g);
            unpack8(y[u][1], g + 4);
            if (at.turned) rope_turn<INTER>(g, c, s);
            // a head that is not there is zeros, and with eps = 0 its 1 / sqrt(0) would make NaN of them
            const float rms = inverse_rms<D>(x, p.eps), r = h < t.heads ? rms : 0.f;
            const float2 rr = make_float2(r, r);
            float2 gx = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = mul2(x[i], rr);
                dw[i] = fma2(g[i], x[i], dw[i]);  // a head that is not there adds 0
                g[i] = mul2(g[i], w[i]);
                gx = fma2(g[i], x[i], gx);
            }
            const float mean = head_sum<C::LPH>(gx.x + gx.y) * (-1.0f / D);
            const float2 mm = make_float2(mean, mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul2(rr, fma2(mm, x[i], g[i]));
            if (h < t.heads) {
                __nv_bfloat16* dst = t.out + m * t.out_stride + h * D;
                *reinterpret_cast<uint4*>(dst + at.ea) = pack8(x);
                *reinterpret_cast<uint4*>(dst + at.eb) = pack8(x + 4);
            }
        }
    }
    // heads of a pass, then warps
    __shared__ float sum[kRopeWarps][D];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float d = i & 1 ? dw[i / 2].y : dw[i / 2].x;
#pragma unroll
        for (int o = C::LPH; o < 32; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (at.g == 0) sum[warp_id()][(i < 8 ? at.ea : at.eb) + i % 8] = d;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < kRopeWarps; ++k) total += sum[k][threadIdx.x];
        p.partial[(int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x] = total;
    }
}

// Adds the blocks' rows: block 0 those of q, block 1 those of k. Every thread takes every NG-th row of one element,
// then the threads of an element join, always in the same order.
constexpr int kRopeSumThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kRopeSumThreads) rope_dw_kernel(const float* partial, int q_rows, int k_rows, float* dw_q, float* dw_k) {
    constexpr int NG = kRopeSumThreads / D;
    __shared__ float sum[NG][D];
    const int e = int(threadIdx.x) % D, g = int(threadIdx.x) / D;
    const int first = blockIdx.x == 0 ? 0 : q_rows, rows = blockIdx.x == 0 ? q_rows : k_rows;
    grid_wait();
    grid_release();
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    int r = g;
    for (; r + 3 * NG < rows; r += 4 * NG)
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] += partial[int64_t(first + r + k * NG) * D + e];
    for (; r < rows; r += NG) a[0] += partial[int64_t(first + r) * D + e];
    sum[g][e] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (threadIdx.x < D) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) total += sum[k][e];
        (blockIdx.x == 0 ? dw_q : dw_k)[e] = total;
    }
}

int passes(int heads, int d) { return (heads + 512 / d - 1) / (512 / d); }
int chunks_of(int heads, int d, int U) { return (passes(heads, d) + U - 1) / U; }

// A warp's passes of a row in the backward kernel (32768 tokens of 32 + 8 heads of 128: 175 us; with four, which spill, 186 us).
// Two blocks to an SM: with three its 128 registers do not fit and it takes 255 us, more rows of blocks change nothing.
constexpr int kBwdPasses = 2;

template <int D, bool NORM, int U>
int launch_fwd_t(const RopeParams& p, bool inter, dim3 grid, cudaStream_t stream) {
    auto kern = inter ? rope_fwd_kernel<D, NORM, true, U> : rope_fwd_kernel<D, NORM, false, U>;
    return launch_chained(kern, grid, kRopeThreads, 0, stream, p) ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

template <int D>
int launch_fwd_d(RopeParams& p, bool inter, cudaStream_t stream) {
    const bool norm = p.side[0].w != nullptr;
    // A warp takes all heads of q or k of its row, two passes at a time, and computes the row's angles once for them; where that
    // leaves the GPU's warps without work, parts of them, down to one pass (64 rows of 32 + 8 heads of 128: 2.0 us; with all
    // heads to a warp 4.1 us; 32768 rows with norms: 106 us, with one pass to a warp 177 us).
    const int most = std::max(passes(p.side[0].heads, D), passes(p.side[1].heads, D)), warps = device_sm_count() * 24;
    int per = 1;
    while (per < most && int64_t(p.rows) * (most / (2 * per) + 1) >= warps) per *= 2;
    for (RopeSide& t : p.side) {
        t.passes = per;
        t.chunks = chunks_of(t.heads, D, per);
    }
    const int64_t blocks = (int64_t(p.rows) + kRopeWarps - 1) / kRopeWarps;
    const dim3 grid(unsigned(blocks), unsigned(p.side[0].chunks + p.side[1].chunks));
    if (per == 1) return norm ? launch_fwd_t<D, true, 1>(p, inter, grid, stream) : launch_fwd_t<D, false, 1>(p, inter, grid, stream);
    return norm ? launch_fwd_t<D, true, 2>(p, inter, grid, stream) : launch_fwd_t<D, false, 2>(p, inter, grid, stream);
}

int bwd_classes(int H, int Hkv, int d) { return chunks_of(H, d, kBwdPasses) + chunks_of(Hkv, d, kBwdPasses); }

template <int D>
int launch_norm_bwd_d(RopeParams& p, bool inter, cudaStream_t stream) {
    for (RopeSide& t : p.side) t.chunks = chunks_of(t.heads, D, kBwdPasses);
    const int classes = p.side[0].chunks + p.side[1].chunks;
    if (p.rows == 0)  // sums of nothing
        return launch_chained(rope_dw_kernel<D>, dim3(2), kRopeSumThreads, 0, stream, p.partial, 0, 0, p.side[0].dw, p.side[1].dw)
                   ? ULYSSES_OK : ULYSSES_ERR_CUDA;
    const int64_t want = (int64_t(p.rows) + kRopeWarps - 1) / kRopeWarps;
    const int most = std::max(1, std::min(kRopeBwdCtas, 2 * device_sm_count()) / classes);
    const int x = int(std::min<int64_t>(want, most));
    auto kern = inter ? rope_norm_bwd_kernel<D, true, kBwdPasses> : rope_norm_bwd_kernel<D, false, kBwdPasses>;
    if (!launch_chained(kern, dim3(unsigned(x), unsigned(classes)), kRopeThreads, 0, stream, p)) return ULYSSES_ERR_CUDA;
    return launch_chained(rope_dw_kernel<D>, dim3(2), kRopeSumThreads, 0, stream, p.partial, x * p.side[0].chunks,
                          x * p.side[1].chunks, p.side[0].dw, p.side[1].dw) ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

RopeParams params_of(const RopeArgs& a) {
    RopeParams p{};
    for (int i = 0; i < 2; ++i) {
        RopeSide& t = p.side[i];
        const RopeTensors& s = i == 0 ? a.q : a.k;
        t.x = static_cast<const __nv_bfloat16*>(s.x);
        t.dy = static_cast<const __nv_bfloat16*>(s.dy);
        t.out = static_cast<__nv_bfloat16*>(s.out);
        t.w = s.w;
        t.dw = s.dw;
        t.x_stride = s.x_stride;
        t.out_stride = s.out_stride;
        t.heads = s.heads;
    }
    p.turns = a.rope.turns;
    p.rot = a.rope.rot;
    p.amplitude = a.rope.amplitude;
    p.sign = a.back ? -1.f : 1.f;
    p.eps = a.eps;
    p.wide = a.wide;
    p.rows = a.rows;
    p.positions = a.positions;
    p.cu_q = a.cu_q;
    p.kv_lens = a.kv_lens;
    p.B = a.B;
    p.pos0 = a.pos0;
    p.seg = a.seg;
    p.shard_rows = a.shard_rows;
    p.shard_step = a.shard_step;
    p.partial = static_cast<float*>(a.workspace);
    return p;
}

}  // namespace

size_t rope_bwd_workspace_bytes(int H, int Hkv, int d) {
    // up to kRopeBwdCtas blocks, or one for each part of the heads
    return size_t(std::max(kRopeBwdCtas, bwd_classes(H, Hkv, d))) * d * sizeof(float);
}

int launch_rope(const RopeArgs& a, cudaStream_t stream) {
    RopeParams p = params_of(a);
    if (a.rows == 0 && !(a.back && a.q.w)) return ULYSSES_OK;
    if (a.back && a.q.w)
        return a.d == 128 ? launch_norm_bwd_d<128>(p, a.rope.interleaved, stream) : launch_norm_bwd_d<64>(p, a.rope.interleaved, stream);
    if (a.back)  // without weights the gradient is the rotation the other way
        for (RopeSide& t : p.side) t.x = t.dy;
    return a.d == 128 ? launch_fwd_d<128>(p, a.rope.interleaved, stream) : launch_fwd_d<64>(p, a.rope.interleaved, stream);
}

}  // namespace ulysses
