// Paged attention for few new rows per key/value head (decoding, or a handful of tokens): a unit has
// at most 16 rows, tokens x grouped query heads, and is bound by reading its keys and values once.
//
// A CTA keeps a ring of key/value tiles in flight, two CTAs to an SM, 192 KB of copies outstanding
// per SM in all, which is what HBM latency asks for. Sixteen rows are one m16n8k16 fragment: the
// warp-level matrix instruction is wide enough for them, while a 128-row tcgen05 tile would spend its
// softmax on empty TMEM lanes. Warp roles (160 threads):
//   warp 0     walks the CTA's share of key tiles (paged_common.cuh), looks up their pages and
//              issues one bulk tensor copy per page and operand into the ring, with the unit's
//              query rows beside its first tile; what the tile is goes along in a descriptor;
//   warps 1-4  each own a quarter of every tile's keys with a running maximum, sum and O of their
//              own (no exchange per tile); at the end of a unit the four join in shared memory, in
//              the tile's own buffer, and the rows are stored, or left as a piece for the join.
// 64 requests of 64 to 8192 keys (32/8 heads of 128) take 170 us with the join, 6.3 TB/s of keys and values, 0.93 of
// the measured copy bandwidth; the tensor pipe is 17% busy. One request of 1500 keys takes 8.4 us, of which the
// keys are 0.9: a chain of launch, lengths, block table, keys, the warps' join and the pieces' join. 64 requests of four
// tokens over up to 8192 keys take 167 us (keys and values: 143); of two to eight, 196 us (157), those of five to eight in
// the chunk kernel beside this one.
#include <algorithm>

#include "paged_common.cuh"

namespace ulysses {

namespace {

constexpr int kDecodeRows = 16;
constexpr int kDecodeThreads = 160;
constexpr int kDecodeMaxCtas = 320;  // 2 per SM, up to 160 SMs: sizes the workspace
// The smallest share of a CTA, in key tiles: one request of 1500 keys takes 8.4 us with 2, 8.9 us with 1 and 9.2 us with 4;
// batches that fill the grid do not notice.
constexpr int kDecodeMinCost = 2;
// The fixed cost of a unit, in key tiles. 1 and 2 lie within 4% of one another: 3 requests of 9000 to 32768 keys 83.1 us with
// 1 and 83.7 us with 2, 64 of four tokens 166 us and 161 us, 200 of up to 1500 keys 105.2 us and 103.2 us.
constexpr int kDecodeUnitCost = 1;

template <int D>
struct DecodeCfg {
    static constexpr int KT = D == 128 ? 64 : 128;  // keys per tile: 16 KB of K and 16 KB of V either way
    static constexpr int KW = KT / 4;               // keys of one warp
    static constexpr int STAGES = 3;
    static constexpr uint32_t KV_BYTES = KT * D * 2;
    static constexpr uint32_t STAGE_BYTES = 2 * KV_BYTES;
    static constexpr uint32_t Q_PITCH = D * 2 + 16;  // 16 bytes of padding: ldmatrix rows on different banks
    static constexpr uint32_t Q_BYTES = kDecodeRows * Q_PITCH;
    static constexpr uint32_t OFF_Q = STAGES * STAGE_BYTES;
    static constexpr uint32_t OFF_DESC = OFF_Q + STAGES * Q_BYTES;
    static constexpr uint32_t OFF_ML = OFF_DESC + STAGES * 64;
    static constexpr uint32_t OFF_SH = OFF_ML + 4 * kDecodeRows * 8;
    static constexpr uint32_t OFF_BAR = OFF_SH + 128;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 128 + 1024;
    static_assert(4 * kDecodeRows * D * 4 <= STAGE_BYTES, "the join of the warps fits a stage");
    static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
};

enum : int { TILE_FIRST = 1, TILE_LAST = 2, TILE_MASKED = 4, TILE_END = 8 };  // END: no tile, the share is done

// One key tile as the producer describes it to the consumers.
struct DecodeTile {
    int flags, key0, kv, base;   // first key, the request's keys, position of the unit's first row
    int rows, row0, head, slot;  // rows, first row of q, key/value head; slot of a piece or -1
    uint32_t valid;              // bit i: the page of keys [16 i, 16 i + 16) exists
};
static_assert(sizeof(DecodeTile) <= 64, "descriptor");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += a b, 16 x 8 x 16, bf16 with fp32 sums
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit u of key r in a tile whose pages were copied one after another, each as
// [64-element chunk][row][128 bytes] with the 128-byte swizzle; `log_rows` rows per page copy.
template <int D>
__device__ __forceinline__ uint32_t kv_offset(int r, int u, int log_rows) {
    const int j = r >> log_rows, rr = r & ((1 << log_rows) - 1);
    return (uint32_t(j) << log_rows) * (D * 2) + (uint32_t(u >> 3) << (log_rows + 7)) + uint32_t(rr) * 128u +
           (uint32_t((u & 7) ^ (rr & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kDecodeThreads, 2)
paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedParams p,
                    int log_rows /* of one page copy */) {
    using C = DecodeCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [4][16]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* full = bars;                // [STAGES]
    uint64_t* empty = full + C::STAGES;   // [STAGES], the four consumer warps
    uint64_t* join = empty + C::STAGES;   // the four consumer warps, twice a unit
    int* abort_flag = reinterpret_cast<int*>(join + 1);
    auto tile_desc = [&](int st) { return reinterpret_cast<DecodeTile*>(smem + C::OFF_DESC + st * 64); };

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
                    if (!free_stage(st)) break;
                    const bool good = unsigned(id) < unsigned(p.num_pages);
                    // one bit per copy, and one per 16 keys
                    const unsigned pages = __ballot_sync(0xffffffffu, good);
                    const int page_of = (min(lane, C::KT / 16 - 1) * 16) >> log_rows;  // of keys [16 lane, 16 lane + 16)
                    const uint32_t valid = __ballot_sync(0xffffffffu, lane < C::KT / 16 && ((pages >> (2 * page_of)) & 1u));
                    uint8_t* stage = smem + st * C::STAGE_BYTES;
                    if (lane == 0) {
                        DecodeTile t;
                        const int pos0 = w.s.base + w.t0, pos1 = w.s.base + w.t1 - 1;  // of the first and last row
                        const bool clear = valid == (1u << (C::KT / 16)) - 1 && key0 + C::KT <= w.s.kv &&
                                           (!p.causal || (key0 + C::KT <= pos0 + 1 && (p.window == 0 || key0 > pos1 - p.window)));
                        t.flags = (x == 0 ? TILE_FIRST : 0) | (x + 1 == tiles ? TILE_LAST : 0) | (clear ? 0 : TILE_MASKED);
                        t.key0 = key0; t.kv = w.s.kv; t.base = pos0;
                        t.rows = rows; t.row0 = w.s.start + w.t0; t.head = w.head; t.slot = slot;
                        t.valid = valid;
                        *tile_desc(st) = t;
                        mbar_arrive_expect_tx(full + st, (__popc(pages) << log_rows) * (D * 2) + (x == 0 ? rows * D * 2 : 0));
                    }
                    __syncwarp();
                    if (good)
                        tma_load_5d(stage + (lane & 1) * C::KV_BYTES + my_row * (D * 2), (lane & 1) ? &tm_v : &tm_k, full + st, 0,
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
        uint32_t qf[D / 16][4];
        float o[D / 8][4];
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        int tok0 = 0, tok1 = 0;         // tokens of this thread's two rows
        int joins = 0;
        const int r0 = lane >> 2, r1 = r0 + 8;
        for (int it = 0;; ++it) {
            const int st = it % C::STAGES;
            if (!__all_sync(0xffffffffu, mbar_wait(full + st, (it / C::STAGES) & 1, ab, ROLE_SOFTMAX, 1))) break;
            const DecodeTile t = *tile_desc(st);
            if (t.flags & TILE_END) break;
            const uint32_t sK = smem_u32(smem + st * C::STAGE_BYTES), sV = sK + C::KV_BYTES;
            if (t.flags & TILE_FIRST) {
                const uint32_t sQ = smem_u32(smem + C::OFF_Q + st * C::Q_BYTES);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    ldsm4(sQ + (lane & 15) * C::Q_PITCH + k * 32 + (lane >> 4) * 16, qf[k]);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
                m0 = m1 = -INFINITY;
                l0 = l1 = 0.f;
                tok0 = r0 / p.G;
                tok1 = r1 / p.G;
            }
            // scores of 16 rows and KW keys
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    uint32_t b[4];
                    const int key = cw * C::KW + i * 8 + ((lane >> 4) << 3) + (lane & 7);
                    ldsm4(sK + kv_offset<D>(key, 2 * k + ((lane >> 3) & 1), log_rows), b);
                    mma16816(s[i], qf[k], b[0], b[1]);
                    mma16816(s[i + 1], qf[k], b[2], b[3]);
                }
            }
            const bool masked = t.flags & TILE_MASKED;
            const int col = t.key0 + cw * C::KW + 2 * (lane & 3);  // key of s[0][0]
            if (masked) {
                const int p0 = t.base + tok0, p1 = t.base + tok1;
                const int h0 = p.causal ? min(t.kv, p0 + 1) : t.kv, h1 = p.causal ? min(t.kv, p1 + 1) : t.kv;
                const int b0 = p.window > 0 ? p0 - p.window + 1 : 0, b1 = p.window > 0 ? p1 - p.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const bool page = (t.valid >> ((cw * C::KW + i * 8) >> 4)) & 1u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = col + i * 8 + e;
                        if (!page || key >= h0 || key < b0) s[i][e] = -INFINITY;
                        if (!page || key >= h1 || key < b1) s[i][2 + e] = -INFINITY;
                    }
                }
            }
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                x0 = fmaxf(x0, fmaxf(s[i][0], s[i][1]));
                x1 = fmaxf(x1, fmaxf(s[i][2], s[i][3]));
            }
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
            // O and l are rescaled only when the maximum has grown by 2^8 (weights then stay below 2^8)
            const float n0 = fmaxf(m0, x0 * p.scale_log2), n1 = fmaxf(m1, x1 * p.scale_log2);
            const bool up0 = n0 > m0 + 8.f, up1 = n1 > m1 + 8.f;
            if (__any_sync(0xffffffffu, up0 || up1)) {
                const float a0 = up0 ? ex2(m0 - n0) : 1.f, a1 = up1 ? ex2(m1 - n1) : 1.f;
                if (up0) m0 = n0;
                if (up1) m1 = n1;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= a0;
                    o[i][1] *= a0;
                    o[i][2] *= a1;
                    o[i][3] *= a1;
                }
            }
            const float g0 = m0 == -INFINITY ? 0.f : -m0, g1 = m1 == -INFINITY ? 0.f : -m1;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                s[i][0] = ex2(fmaf(s[i][0], p.scale_log2, g0));
                s[i][1] = ex2(fmaf(s[i][1], p.scale_log2, g0));
                s[i][2] = ex2(fmaf(s[i][2], p.scale_log2, g1));
                s[i][3] = ex2(fmaf(s[i][3], p.scale_log2, g1));
                l0 += s[i][0] + s[i][1];
                l1 += s[i][2] + s[i][3];
            }
            // O += P V. The matrix instruction takes the weights in bf16, the type of the values, off by at most 2^-8 of
            // a weight; their sum is taken of the weights before. Errors against 64 bits are 1.2 to 1.4 times those of fp32
            // weights with one rounding at the end (0.0023 against 0.0017 of the output's size).
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                const uint32_t a[4] = {pack_bf16(s[2 * j][0], s[2 * j][1]), pack_bf16(s[2 * j][2], s[2 * j][3]),
                                       pack_bf16(s[2 * j + 1][0], s[2 * j + 1][1]), pack_bf16(s[2 * j + 1][2], s[2 * j + 1][3])};
                // values behind the last key, or of pages that were not copied, may be anything, NaN too:
                // their bits are cleared
                uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                if (masked) {
                    const int end = (t.valid >> ((cw * C::KW + j * 16) >> 4)) & 1u ? t.kv : 0, key = col + j * 16;
                    keep0 = (key < end ? 0xffffu : 0u) | (key + 1 < end ? 0xffff0000u : 0u);
                    keep1 = (key + 8 < end ? 0xffffu : 0u) | (key + 9 < end ? 0xffff0000u : 0u);
                }
                const int key = cw * C::KW + j * 16 + (lane & 15);
#pragma unroll
                for (int i = 0; i < D / 8; i += 2) {
                    uint32_t b[4];
                    ldsm4_t(sV + kv_offset<D>(key, i + (lane >> 4), log_rows), b);
                    mma16816(o[i], a, b[0] & keep0, b[1] & keep1);
                    mma16816(o[i + 1], a, b[2] & keep0, b[3] & keep1);
                }
            }
            if (t.flags & TILE_LAST) {
                // the four warps join: each writes its rows over the tile that all have finished reading
                l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
                l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
                l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
                l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
                __syncwarp();
                if (lane == 0) mbar_arrive(join);
                if (!__all_sync(0xffffffffu, mbar_wait(join, joins & 1, ab, ROLE_EPI, 1))) break;
                ++joins;
                float* scratch = reinterpret_cast<float*>(smem + st * C::STAGE_BYTES);
                float* mine = scratch + cw * (kDecodeRows * D);
                if ((lane & 3) == 0) {
                    ml[cw * kDecodeRows + r0] = make_float2(m0, l0);
                    ml[cw * kDecodeRows + r1] = make_float2(m1, l1);
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const int at = ((i ^ (r0 & 7)) << 3) + 2 * (lane & 3);  // r1 & 7 == r0 & 7
                    if (r0 < t.rows) *reinterpret_cast<float2*>(mine + r0 * D + at) = make_float2(o[i][0], o[i][1]);
                    if (r1 < t.rows) *reinterpret_cast<float2*>(mine + r1 * D + at) = make_float2(o[i][2], o[i][3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(join);
                if (!__all_sync(0xffffffffu, mbar_wait(join, joins & 1, ab, ROLE_EPI, 2))) break;
                ++joins;
                for (int x = cw * 32 + lane; x < t.rows * (D / 4); x += 128) {
                    const int r = x / (D / 4), c4 = x % (D / 4);
                    const int at = r * D + (((c4 >> 1) ^ (r & 7)) << 3) + (c4 & 1) * 4;
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
                    if (t.slot >= 0) {
                        const int64_t row = int64_t(t.slot) * kDecodeRows + r;
                        *reinterpret_cast<float4*>(p.parts.o + row * D + c4 * 4) = acc;
                        if (c4 == 0) p.parts.ml[row] = make_float2(m, l);
                    } else {
                        const float inv = l == 0.f ? 0.f : 1.0f / l;  // 0: no key; NaN scores stay NaN
                        const int row = t.row0 + r / p.G, h = t.head * p.G + r % p.G;
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
int launch_decode_d(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream) {
    using C = DecodeCfg<D>;
    const int rows = std::min(a.cache.page_size, C::KT);
    CUtensorMap mk, mv;
    if (!encode_pages(&mk, a.cache, a.cache.k, rows, D / 64) || !encode_pages(&mv, a.cache, a.cache.v, rows, D / 64))
        return ULYSSES_ERR_CUDA;
    auto kern = paged_decode_kernel<D>;
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ULYSSES_ERR_CUDA;
    if (!launch_chained(kern, dim3(unsigned(p.parts.ctas)), kDecodeThreads, C::SMEM_BYTES, stream, mk, mv, p,
                        __builtin_ctz(unsigned(rows))))
        return ULYSSES_ERR_CUDA;
    return ULYSSES_OK;
}

}  // namespace

int paged_decode_rows() { return kDecodeRows; }

PagedParts paged_decode_parts(void* workspace, int d_h, int sms, size_t* bytes) {
    return paged_parts(workspace, kDecodeMaxCtas, 2 * sms, kDecodeRows, d_h, bytes);
}

int launch_paged_decode(const PagedAttnArgs& a, const PagedParams& p, cudaStream_t stream) {
    return a.cache.d_h == 128 ? launch_decode_d<128>(a, p, stream) : launch_decode_d<64>(a, p, stream);
}

}  // namespace ulysses
