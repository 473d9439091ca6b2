// Paged attention over an 8-bit cache for few new rows per key/value head, at most 16 (see paged_decode.cu, whose walk, ring
// and joins these are; there is half as much to read here).
//
// A ring stage holds 16 KB of key codes and 16 KB of value codes: 128 keys of d = 128, 256 of d = 64. The matrix
// instruction is m16n8k16 in fp16, into which e4m3 codes convert exactly, two to an instruction, on their way from shared
// memory to its registers:
// - keys: ldmatrix hands a thread four consecutive codes of a key, which it takes as elements k, k + 1, k + 8, k + 9 of
//   the instruction; the order within a dot product is free, and the query's fragments are loaded in the same order;
// - values: a transposed ldmatrix of 16-bit units hands it two neighbouring elements of two keys; a byte
//   permutation makes of them the pairs of the even and of the odd element, so that a thread ends up with four
//   consecutive elements of O.
// Queries go to fp16 divided by a power of two a row, which puts the row's largest magnitude into [2^14, 2^15): elements down to
// 2^-28 of it stay exact. The keys' scales, powers of two by 16 keys at the finest, multiply the scores.
// The values' scales belong to the weights, and fp16 has few exponents. With s the scores in the log2 domain and v the
// log2 of the value scales, a row therefore holds two running maxima: m of s, for the sum of the weights, and n of s + v,
// for O, whose weights are 2^(s + v - n + 7), at most 2^15 and for the heaviest key at least 2^7. fp16 keeps them to 2^-11 of
// themselves, and to 2^-25 where they are small: 2^-32 of the row's largest weight times scale, whatever the scales. That
// maximum does not know the codes, which span 2^18: where the heaviest key's codes are small or zero under a scale that its
// neighbours set, a key of codes up to 448 may lose 448 * 2^-32 of that largest product, which can be more than 2^-32 of the
// row's largest contribution. O goes back to the units of m at the end of a unit.
// 64 requests of 64 to 8192 keys (32/8 heads of 128) take 104 to 109 us with the join, 5.1 to 5.3 TB/s of codes, 0.75 to 0.79 of
// the measured copy bandwidth (8191 keys each, twice the bytes: 179 to 191 us, 5.6 to 6.0 TB/s); leaving all products out changes 2%. One request of 1500 keys
// takes 9.3 us, a chain of latencies.
#include <algorithm>

#include "paged_common.cuh"

namespace ulysses {

namespace {

constexpr int kDecodeRows = 16;
constexpr int kDecodeThreads = 160;
// The smallest share of a CTA, in key tiles: one request of 1500 keys takes 9.3 us with 1, 9.6 us with 2 and 11.6 us with 4;
// batches that fill the grid do not notice.
constexpr int kDecodeMinCost = 1;
// The fixed cost of a unit, in key tiles, with 1, 2, 3, 4: 64 requests of 64 to 8192 keys 115, 108.5, 107.8, 108.2 us; 200 of up
// to 1500 keys -, 82.3, 83.8, 85.4 us.
constexpr int kDecodeUnitCost = 2;

template <int D>
struct Decode8Cfg {
    static constexpr int KT = 16384 / D;             // keys per tile
    static constexpr int KW = KT / 4;                // keys of one warp
    static constexpr int KG = KT / 16;               // groups of 16 keys: one page and one scale each
    static constexpr int STAGES = 3;
    static constexpr uint32_t KV_BYTES = KT * D;
    static constexpr uint32_t STAGE_BYTES = 2 * KV_BYTES;
    static constexpr uint32_t Q_PITCH = D * 2 + 16;  // 16 bytes of padding: rows on different banks
    static constexpr uint32_t Q_BYTES = kDecodeRows * Q_PITCH;
    static constexpr uint32_t DESC_BYTES = 192;
    static constexpr uint32_t OFF_Q = STAGES * STAGE_BYTES;
    static constexpr uint32_t OFF_DESC = OFF_Q + STAGES * Q_BYTES;
    static constexpr uint32_t OFF_ML = OFF_DESC + STAGES * DESC_BYTES;
    static constexpr uint32_t OFF_SH = OFF_ML + 4 * kDecodeRows * 8;
    static constexpr uint32_t OFF_BAR = OFF_SH + 128;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 128 + 1024;
    static_assert(4 * kDecodeRows * D * 4 <= STAGE_BYTES, "the join of the warps fits a stage");
    static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
    static_assert(2 * KG <= 32, "one lane for each scale of a tile, and for each copy");
};

enum : int { TILE_FIRST = 1, TILE_LAST = 2, TILE_MASKED = 4, TILE_END = 8 };  // END: no tile, the share is done

// One key tile as the producer describes it to the consumers.
struct Decode8Tile {
    int flags, key0, kv, base;   // first key, the request's keys, position of the unit's first row
    int rows, row0, head, slot;  // rows, first row of q, key/value head; slot of a piece or -1
    uint32_t valid;              // bit i: the page of keys [16 i, 16 i + 16) exists
    uint32_t pad[3];
    float scale[2][16];          // of keys [16 i, 16 i + 16): the keys' scale; log2 of the values'
};
static_assert(sizeof(Decode8Tile) <= Decode8Cfg<64>::DESC_BYTES, "descriptor");

// c += a b, 16 x 8 x 16, fp16 with fp32 sums
__device__ __forceinline__ void mma16816_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t&>(v);
}

// The exponent of a row's largest magnitude, from the bits of |q| (bf16 pairs) of the lane's part, over the four lanes of
// the row. At least -100, so that 2^(14 - e) is finite; 128 with an infinity.
__device__ __forceinline__ int row_exponent(uint32_t top) {
    uint32_t t = max(top & 0xffffu, top >> 16);
    t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
    t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
    return max(int(t >> 7) - 127, -100);
}

template <int D>
__global__ void __launch_bounds__(kDecodeThreads, 2)
paged_decode8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedParams p,
                     const PagedScales scales, int log_rows /* of one page copy */) {
    using C = Decode8Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [4][16]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* full = bars;                // [STAGES]
    uint64_t* empty = full + C::STAGES;   // [STAGES], the four consumer warps
    uint64_t* join = empty + C::STAGES;   // the four consumer warps, twice a unit
    int* abort_flag = reinterpret_cast<int*>(join + 1);
    auto tile_desc = [&](int st) { return reinterpret_cast<Decode8Tile*>(smem + C::OFF_DESC + st * C::DESC_BYTES); };

    const int warp = int(warp_id()), lane = int(lane_id());
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 4);
        }
        mbar_init(join, 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    grid_wait();
    grid_release();  // not before the wait: the chunk kernel starts behind this without one
    const int cta = int(blockIdx.x);
    PagedWalk<C::KT, kDecodeUnitCost> w;
    int64_t* costs = reinterpret_cast<int64_t*>(smem);  // before the first copy
    if (p.B > kFewRequests)
        paged_share_block<C::KT, kDecodeUnitCost, kDecodeThreads>(p, kDecodeMinCost, reinterpret_cast<int64_t*>(smem + C::OFF_SH), w);
    else if (p.B > kLaneRequests) paged_costs<C::KT, kDecodeUnitCost, kDecodeThreads>(p, costs);
    __syncthreads();
    const Abort ab{abort_flag, p.err, KID_PAGED};

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        if (p.B <= kLaneRequests) paged_share_lanes(p, kDecodeMinCost, w);
        else if (p.B <= kFewRequests) paged_share_warp(p, kDecodeMinCost, costs, w);
        const int copies = 2 * (C::KT >> log_rows);  // one per page and operand
        const int my_row = (lane >> 1) << log_rows;  // of this lane's copy within the tile
        const int my_group = min(lane >> 1, C::KG - 1) * 16;  // first key of this lane's scale: keys' and values' in turn
        const int group_copy = (my_group >> log_rows) * 2;    // the copy that brings them
        const uint8_t* scale_of = (lane & 1) ? scales.v : scales.k;
        int lo, hi;                                  // keys that the unit's rows may see
        auto lookup = [&](int key0) {                // only their pages are copied
            const int key = key0 + my_row;
            return lane < copies && key < hi && key + (1 << log_rows) > lo ? p.table[w.i * p.table_stride + (key >> p.page_shift)]
                                                                           : -1;
        };
        PagedMeta meta{0, 0, 0, 0};
        int issued = 0;
        bool ok = true, first_piece = true;
        auto free_stage = [&](int st) {
            if (issued >= C::STAGES)
                ok = __all_sync(0xffffffffu, mbar_wait(empty + st, ((issued / C::STAGES) - 1) & 1, ab, ROLE_LOAD, 1));
            return ok;
        };
        while (ok && w.left > 0) {
            int off, tiles;
            w.take(off, tiles);
            if (tiles > 0) {
                int slot = -1;
                const bool ends = off + tiles == w.count;
                if (first_piece && off > 0) {
                    slot = 2 * cta;
                } else if (!ends) {
                    slot = 2 * cta + 1;
                    meta = PagedMeta{w.pieces(cta), w.head, w.s.start + w.t0, (w.t1 - w.t0) * p.G};
                }
                first_piece = false;
                const int rows = (w.t1 - w.t0) * p.G;
                paged_range(p, w.s, w.t0, w.t1, lo, hi);
                int id = lookup((w.first + off) * C::KT);
                for (int x = 0; x < tiles; ++x) {
                    const int st = issued % C::STAGES;
                    const int key0 = (w.first + off + x) * C::KT;
                    const int id_next = x + 1 < tiles ? lookup(key0 + C::KT) : -1;
                    const bool good = unsigned(id) < unsigned(p.num_pages);
                    // the scale's byte, on its way while the stage becomes free
                    const int page = __shfl_sync(0xffffffffu, good ? id : -1, group_copy);
                    int byte = 127;
                    if (page >= 0) {
                        const int token = (key0 + my_group) & ((1 << p.page_shift) - 1);
                        const int64_t at = (int64_t(page) << (p.page_shift - scales.block_shift)) + (token >> scales.block_shift);
                        byte = scale_of[at * p.Hkv + w.head];
                    }
                    if (!free_stage(st)) break;
                    // one bit per copy, and one per 16 keys
                    const unsigned pages = __ballot_sync(0xffffffffu, good);
                    const int page_of = (min(lane, C::KG - 1) * 16) >> log_rows;  // of keys [16 lane, 16 lane + 16)
                    const uint32_t valid = __ballot_sync(0xffffffffu, lane < C::KG && ((pages >> (2 * page_of)) & 1u));
                    uint8_t* stage = smem + st * C::STAGE_BYTES;
                    Decode8Tile* t = tile_desc(st);
                    if (lane < 2 * C::KG)
                        t->scale[lane & 1][lane >> 1] = (lane & 1) ? float(byte - 127) : __uint_as_float(uint32_t(byte) << 23);
                    __syncwarp();
                    if (lane == 0) {
                        const int pos0 = w.s.base + w.t0, pos1 = w.s.base + w.t1 - 1;  // of the first and last row
                        const bool clear = valid == (1u << C::KG) - 1 && key0 + C::KT <= w.s.kv &&
                                           (!p.causal || (key0 + C::KT <= pos0 + 1 && (p.window == 0 || key0 > pos1 - p.window)));
                        t->flags = (x == 0 ? TILE_FIRST : 0) | (x + 1 == tiles ? TILE_LAST : 0) | (clear ? 0 : TILE_MASKED);
                        t->key0 = key0; t->kv = w.s.kv; t->base = pos0;
                        t->rows = rows; t->row0 = w.s.start + w.t0; t->head = w.head; t->slot = slot;
                        t->valid = valid;
                        mbar_arrive_expect_tx(full + st, (__popc(pages) << log_rows) * D + (x == 0 ? rows * D * 2 : 0));
                    }
                    __syncwarp();
                    if (good)
                        tma_load_5d(stage + (lane & 1) * C::KV_BYTES + my_row * D, (lane & 1) ? &tm_v : &tm_k, full + st, 0,
                                    (key0 + my_row) & ((1 << p.page_shift) - 1), w.head, id, 0);
                    if (x == 0 && lane < rows) {
                        const __nv_bfloat16* src = p.q + int64_t(w.s.start + w.t0 + lane / p.G) * p.q_stride +
                                                   int64_t(w.head * p.G + lane % p.G) * D;
                        bulk_load(smem + C::OFF_Q + st * C::Q_BYTES + lane * C::Q_PITCH, src, D * 2, full + st);
                    }
                    ++issued;
                    id = id_next;
                }
            }
            if (ok && w.left > 0) w.next_unit(p);
        }
        if (lane == 0) p.parts.meta[cta] = meta;
        if (ok && free_stage(issued % C::STAGES)) {
            if (lane == 0) {
                tile_desc(issued % C::STAGES)->flags = TILE_END;
                mbar_arrive(full + issued % C::STAGES);
            }
            ++issued;
        }
        // every copy lands before the CTA can exit, also where a consumer has given up since
        if (lane == 0) ring_drain<C::STAGES>(full, issued);
    } else {
        // ------------------------------------------------------------------ consumers
        const int cw = warp - 1;
        constexpr int NT = C::KW / 8;   // 8-key column tiles of this warp's scores
        constexpr int NG = C::KW / 16;  // its groups of 16 keys
        uint32_t qf[D / 16][4];
        float o[D / 16][2][4];          // 16 elements: the even ones, the odd ones
        float m0 = -INFINITY, m1 = -INFINITY, n0 = -INFINITY, n1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float f0 = 0.f, f1 = 0.f;       // the rows' powers of two, and the softmax scale
        int tok0 = 0, tok1 = 0;         // tokens of this thread's two rows
        int joins = 0;
        const int r0 = lane >> 2, r1 = r0 + 8, quad = lane & 3;
        for (int it = 0;; ++it) {
            const int st = it % C::STAGES;
            if (!__all_sync(0xffffffffu, mbar_wait(full + st, (it / C::STAGES) & 1, ab, ROLE_SOFTMAX, 1))) break;
            const Decode8Tile& t = *tile_desc(st);
            const int flags = t.flags;
            if (flags & TILE_END) break;
            const uint32_t sK = smem_u32(smem + st * C::STAGE_BYTES), sV = sK + C::KV_BYTES;
            if (flags & TILE_FIRST) {
                const uint8_t* sQ = smem + C::OFF_Q + st * C::Q_BYTES;
                uint2 q[D / 16][2];
                uint32_t top0 = 0, top1 = 0;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    q[k][0] = *reinterpret_cast<const uint2*>(sQ + r0 * C::Q_PITCH + k * 32 + quad * 8);
                    q[k][1] = *reinterpret_cast<const uint2*>(sQ + r1 * C::Q_PITCH + k * 32 + quad * 8);
                    top0 = max_abs2(max_abs2(top0, q[k][0].x), q[k][0].y);
                    top1 = max_abs2(max_abs2(top1, q[k][1].x), q[k][1].y);
                }
                const int e0 = row_exponent(top0), e1 = row_exponent(top1);
                const float by[2] = {pow2f(14 - e0), pow2f(14 - e1)};
                f0 = pow2f(e0 - 14) * p.scale_log2;
                f1 = pow2f(e1 - 14) * p.scale_log2;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        qf[k][r] = pack_f16(__uint_as_float(q[k][r].x << 16) * by[r], __uint_as_float(q[k][r].x & 0xffff0000u) * by[r]);
                        qf[k][2 + r] = pack_f16(__uint_as_float(q[k][r].y << 16) * by[r], __uint_as_float(q[k][r].y & 0xffff0000u) * by[r]);
                    }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][0][e] = o[i][1][e] = 0.f;
                m0 = m1 = n0 = n1 = -INFINITY;
                l0 = l1 = 0.f;
                tok0 = r0 / p.G;
                tok1 = r1 / p.G;
            }
            // scores of 16 rows and KW keys
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    // 16 keys by 32 elements
                    uint32_t b[4], lo, hi;
                    const int key = cw * C::KW + i * 8 + ((lane >> 4) << 3) + (lane & 7);
                    ldsm4(sK + code_offset<D>(key, k + ((lane >> 3) & 1)), b);
                    e4m3_to_f16(b[0], lo, hi);
                    mma16816_f16(s[i], qf[k], lo, hi);
                    e4m3_to_f16(b[2], lo, hi);
                    mma16816_f16(s[i + 1], qf[k], lo, hi);
                    e4m3_to_f16(b[1], lo, hi);
                    mma16816_f16(s[i], qf[k + 1], lo, hi);
                    e4m3_to_f16(b[3], lo, hi);
                    mma16816_f16(s[i + 1], qf[k + 1], lo, hi);
                }
            }
            float sv[NG];  // log2 of the values' scales
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // finite, also for the largest queries and scales: a zero score stays zero
                const float sk = t.scale[0][cw * NG + g], k0 = fminf(sk * f0, 3e38f), k1 = fminf(sk * f1, 3e38f);
                sv[g] = t.scale[1][cw * NG + g];
#pragma unroll
                for (int i = 2 * g; i < 2 * g + 2; ++i) {
                    s[i][0] *= k0;
                    s[i][1] *= k0;
                    s[i][2] *= k1;
                    s[i][3] *= k1;
                }
            }
            const bool masked = flags & TILE_MASKED;
            const int kv = t.kv;
            const uint32_t exists = t.valid >> (cw * NG);
            const int col = t.key0 + cw * C::KW + 2 * quad;  // key of s[0][0]
            if (masked) {
                const int p0 = t.base + tok0, p1 = t.base + tok1;
                const int h0 = p.causal ? min(kv, p0 + 1) : kv, h1 = p.causal ? min(kv, p1 + 1) : kv;
                const int b0 = p.window > 0 ? p0 - p.window + 1 : 0, b1 = p.window > 0 ? p1 - p.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const bool page = (exists >> (i >> 1)) & 1u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = col + i * 8 + e;
                        if (!page || key >= h0 || key < b0) s[i][e] = -INFINITY;
                        if (!page || key >= h1 || key < b1) s[i][2 + e] = -INFINITY;
                    }
                }
            }
            float x0 = -INFINITY, x1 = -INFINITY, y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float a0 = fmaxf(fmaxf(s[2 * g][0], s[2 * g][1]), fmaxf(s[2 * g + 1][0], s[2 * g + 1][1]));
                const float a1 = fmaxf(fmaxf(s[2 * g][2], s[2 * g][3]), fmaxf(s[2 * g + 1][2], s[2 * g + 1][3]));
                x0 = fmaxf(x0, a0);
                x1 = fmaxf(x1, a1);
                y0 = fmaxf(y0, a0 + sv[g]);
                y1 = fmaxf(y1, a1 + sv[g]);
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, x));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, x));
                y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, x));
                y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, x));
            }
            // l and O are rescaled only when their maximum has grown by 2^8 (weights then stay below 2^8, O's below 2^15)
            const bool um0 = x0 > m0 + 8.f, um1 = x1 > m1 + 8.f, un0 = y0 > n0 + 8.f, un1 = y1 > n1 + 8.f;
            if (__any_sync(0xffffffffu, um0 || um1 || un0 || un1)) {
                if (um0) {
                    l0 *= ex2(m0 - x0);
                    m0 = x0;
                }
                if (um1) {
                    l1 *= ex2(m1 - x1);
                    m1 = x1;
                }
                const float a0 = un0 ? ex2(n0 - y0) : 1.f, a1 = un1 ? ex2(n1 - y1) : 1.f;
                if (un0) n0 = y0;
                if (un1) n1 = y1;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        o[i][x][0] *= a0;
                        o[i][x][1] *= a0;
                        o[i][x][2] *= a1;
                        o[i][x][3] *= a1;
                    }
            }
            const float g0 = m0 == -INFINITY ? 0.f : -m0, g1 = m1 == -INFINITY ? 0.f : -m1;
            const float z0 = n0 == -INFINITY ? 0.f : 7.f - n0, z1 = n1 == -INFINITY ? 0.f : 7.f - n1;
            // O += P V. The matrix instruction takes the weights in fp16, off by at most 2^-11 of a weight (2^-24 of the largest
            // for the smallest); their sum is taken of the weights before
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float w0 = z0 + sv[j], w1 = z1 + sv[j];
                uint32_t a[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float* x = s[2 * j + h];
                    l0 += ex2(x[0] + g0) + ex2(x[1] + g0);
                    l1 += ex2(x[2] + g1) + ex2(x[3] + g1);
                    a[2 * h] = pack_f16(ex2(x[0] + w0), ex2(x[1] + w0));
                    a[2 * h + 1] = pack_f16(ex2(x[2] + w1), ex2(x[3] + w1));
                }
                // values behind the last key, or of pages that were not copied, may be anything, NaN too:
                // their bits are cleared
                uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                if (masked) {
                    const int end = (exists >> j) & 1u ? kv : 0, key = col + j * 16;
                    keep0 = (key < end ? 0xffffu : 0u) | (key + 1 < end ? 0xffff0000u : 0u);
                    keep1 = (key + 8 < end ? 0xffffu : 0u) | (key + 9 < end ? 0xffff0000u : 0u);
                }
                const int key = cw * C::KW + j * 16 + (lane & 15);
#pragma unroll
                for (int i = 0; i < D / 16; i += 2) {
                    uint32_t b[4];
                    ldsm4_t(sV + code_offset<D>(key, i + (lane >> 4)), b);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // bytes: element 2c, 2c + 1 of key 2t, then of key 2t + 1
                        uint32_t e0, d0, e1, d1;
                        e4m3_to_f16(__byte_perm(b[2 * u] & keep0, 0, 0x3120), e0, d0);
                        e4m3_to_f16(__byte_perm(b[2 * u + 1] & keep1, 0, 0x3120), e1, d1);
                        mma16816_f16(o[i + u][0], a, e0, e1);
                        mma16816_f16(o[i + u][1], a, d0, d1);
                    }
                }
            }
            if (flags & TILE_LAST) {
                // the four warps join: each writes its rows over the tile that all have finished reading
                l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
                l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
                l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
                l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
                // from units of 2^(n - 7) to units of 2^m, in two steps that stay in range
                const float h0 = n0 == -INFINITY ? 0.f : 0.5f * (n0 - 7.f - m0), h1 = n1 == -INFINITY ? 0.f : 0.5f * (n1 - 7.f - m1);
                const float c0 = ex2(h0), c1 = ex2(h1);
                const int rows = t.rows, slot = t.slot, head = t.head, row_first = t.row0;
                __syncwarp();
                if (lane == 0) mbar_arrive(join);
                if (!__all_sync(0xffffffffu, mbar_wait(join, joins & 1, ab, ROLE_EPI, 1))) break;
                ++joins;
                float* scratch = reinterpret_cast<float*>(smem + st * C::STAGE_BYTES);
                float* mine = scratch + cw * (kDecodeRows * D);
                if (quad == 0) {
                    ml[cw * kDecodeRows + r0] = make_float2(m0, l0);
                    ml[cw * kDecodeRows + r1] = make_float2(m1, l1);
                }
                constexpr int U = D / 16;  // 16-element units of a row, moved about by row against bank conflicts
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int at = ((i ^ (r0 & (U - 1))) << 4) + 4 * quad;  // the same for r1
                    if (r0 < rows)
                        *reinterpret_cast<float4*>(mine + r0 * D + at) =
                            make_float4(o[i][0][0] * c0 * c0, o[i][1][0] * c0 * c0, o[i][0][1] * c0 * c0, o[i][1][1] * c0 * c0);
                    if (r1 < rows)
                        *reinterpret_cast<float4*>(mine + r1 * D + at) =
                            make_float4(o[i][0][2] * c1 * c1, o[i][1][2] * c1 * c1, o[i][0][3] * c1 * c1, o[i][1][3] * c1 * c1);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(join);
                if (!__all_sync(0xffffffffu, mbar_wait(join, joins & 1, ab, ROLE_EPI, 2))) break;
                ++joins;
                for (int x = cw * 32 + lane; x < rows * (D / 4); x += 128) {
                    const int r = x / (D / 4), c4 = x % (D / 4);
                    const int at = r * D + (((c4 >> 2) ^ (r & (U - 1))) << 4) + (c4 & 3) * 4;
                    float m = -INFINITY, l = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) m = fmaxf(m, ml[k * kDecodeRows + r].x);
                    const float neg = m == -INFINITY ? 0.f : -m;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 q = ml[k * kDecodeRows + r];
                        const float e = ex2(q.x + neg);
                        const float4 y = *reinterpret_cast<const float4*>(scratch + k * (kDecodeRows * D) + at);
                        l += e * q.y;
                        acc.x += e * y.x;
                        acc.y += e * y.y;
                        acc.z += e * y.z;
                        acc.w += e * y.w;
                    }
                    if (slot >= 0) {
                        const int64_t row = int64_t(slot) * kDecodeRows + r;
                        *reinterpret_cast<float4*>(p.parts.o + row * D + c4 * 4) = acc;
                        if (c4 == 0) p.parts.ml[row] = make_float2(m, l);
                    } else {
                        const float inv = l == 0.f ? 0.f : 1.0f / l;  // 0: no key; NaN scores stay NaN
                        const int row = row_first + r / p.G, h = head * p.G + r % p.G;
                        *reinterpret_cast<uint2*>(p.o + (int64_t(row) * p.H + h) * D + c4 * 4) =
                            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                        if (c4 == 0) p.lse[int64_t(h) * p.T + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                    }
                }
                // the next copy into this stage comes after these reads and writes of it
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
        }
    }
    __syncwarp();
    __syncthreads();
}

template <int D>
int launch_decode8_d(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream) {
    using C = Decode8Cfg<D>;
    const int rows = std::min(a.cache.page_size, C::KT);
    CUtensorMap mk, mv;
    if (!encode_code_pages(&mk, a.cache, a.cache.k, rows) || !encode_code_pages(&mv, a.cache, a.cache.v, rows)) return ULYSSES_ERR_CUDA;
    auto kern = paged_decode8_kernel<D>;
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ULYSSES_ERR_CUDA;
    if (!launch_chained(kern, dim3(unsigned(p.parts.ctas)), kDecodeThreads, C::SMEM_BYTES, stream, mk, mv, p, a.scales,
                        __builtin_ctz(unsigned(rows))))
        return ULYSSES_ERR_CUDA;
    return ULYSSES_OK;
}

}  // namespace

int launch_paged_decode8(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream) {
    return a.cache.d_h == 128 ? launch_decode8_d<128>(a, p, stream) : launch_decode8_d<64>(a, p, stream);
}

}  // namespace ulysses
