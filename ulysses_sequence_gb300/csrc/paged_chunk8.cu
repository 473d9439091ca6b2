// Paged attention over an 8-bit cache for chunks of new rows (see paged_chunk.cu, whose units, walk, tensor-memory plan and order
// of products these are).
//
// The products run in bf16: every key and value of such a cache, code x power of two, is exact in bf16, so nothing is
// rounded that attention over a bf16 cache would not round, and queries stay as they are. Codes come into a small ring of
// shared memory by bulk copies; six converter warps turn them into scaled bf16 (e4m3 pair -> fp16 pair -> two fp32, times
// the scale -> bf16 pair) in the swizzled operand tiles. Warp roles (512 threads, a warpgroup each; registers are moved from
// the first and the last to the two between):
//   warp 0       producer: walks the share, looks up pages and scales (one lane to 16 keys), copies codes and queries, and
//                publishes each piece and each tile;
//   warp 1       MMA issuer;
//   warps 4-7    softmax of tile 0, warps 8-11 of tile 1;
//   warps 2, 3 and 12-15  converters: 32 keys or values of a tile in turn. Values behind the request's last key become zeros (0 x NaN is NaN).
// A converter reads a row's 16 codes with one lane; eight lanes that read and write at once take four pieces of each of two
// rows whose numbers differ in the bits that the swizzles of codes and of bf16 put on different banks.
// 8192 new tokens over 16384 keys (32/8 heads of 128) take 1252 us, 1.32 PFLOP/s, 0.68 of the measured bf16 rate: the widening
// beside the products bounds it (1109 us with codes stored as they are; the bf16 kernel 1050 to 1060 us). With four converter
// warps 1411 us. The same with heads of 64, half the work, takes 899 us: its softmax is the same.
#define ULYSSES_SLOW_PATH __forceinline__
#include "paged_common.cuh"

namespace ulysses {

namespace {

constexpr int kChunkThreads = 512;
constexpr int kChunkRows = 2 * kTile;
// The shares of the bf16 kernel, so that calls of chunks are cut alike and give its bits. The smallest, in key tiles: one chunk of 40 tokens
// over 1000 keys takes 17.4 us with 4 and would take 14.9 us with 2. The fixed cost of a unit, with 2, 3, 5: 24 mixed requests
// 96.5, 97.3, 100.0 us, four chunks of 512 tokens 284, 286, 289 us.
constexpr int kChunkMinCost = 4;
constexpr int kChunkUnitCost = 3;
// Registers of a thread by warpgroup: 512 threads are launched with 128 each.
constexpr uint32_t kRegsSoftmax = 176, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther == 4 * 128, "no more than the launch brought");
constexpr int kConverters = 6;       // warps

template <int D>
struct Chunk8Cfg {
    static constexpr int NSC = D == 64 ? 6 : 2;  // stages of codes, keys and values in turn
    static constexpr int NSK = D == 64 ? 4 : 2;  // of K and V in bf16
    static constexpr int NSV = D == 64 ? 4 : 2;
    static constexpr int RING = D == 64 ? 16 : 8;  // tile descriptions
    static constexpr uint32_t CODE_BYTES = kTile * D;
    static constexpr uint32_t TILE_BYTES = kTile * D * 2;
    static constexpr uint32_t CHUNK_BYTES = kTile * 128;  // 128 rows x 64 elements, swizzled
    static constexpr uint32_t OFF_K = 2 * TILE_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + NSK * TILE_BYTES;
    static constexpr uint32_t OFF_C = OFF_V + NSV * TILE_BYTES;
    static constexpr uint32_t OFF_PIECE = OFF_C + NSC * CODE_BYTES;
    static constexpr uint32_t OFF_INFO = OFF_PIECE + 128;
    static constexpr uint32_t OFF_SH = OFF_INFO + RING * 128;
    static constexpr uint32_t OFF_BAR = OFF_SH + 192;
    static constexpr int BARS = 17 + 2 * (NSC + NSK + NSV) + 2 * RING;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 640 + 1024;
    static_assert((kChunkThreads / 32 + 2) * 8 <= 192 && BARS * 8 + 8 <= 640, "room for the shares and the barriers");
    static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    // TMEM: S buffers, O0, O1. d = 64 leaves room for a third S buffer.
    static constexpr bool AHEAD = D == 64;
    static constexpr uint32_t COL_O = (AHEAD ? 3 : 2) * kTile, TMEM_COLS = 512;
    static_assert(COL_O + 2 * D <= TMEM_COLS, "tensor memory");
    // the issuer names columns from 0, constants of its instructions: true of an allocation of the whole tensor memory
    static_assert(TMEM_COLS == 512, "the allocation starts at column 0");
    // Tile n is published when the stage of its keys' codes is free: those of tile n - NSC / 2 are converted, for which the
    // scores of tile n - NSC / 2 - NSK were done, and the softmax warps have read what describes the tile before that one
    // (with AHEAD the one before it).
    static_assert(NSC % 2 == 0 && NSC / 2 + NSK + (AHEAD ? 1 : 0) < RING, "tile descriptions outlive their readers");
    // A wait by parity says that the phase is complete only where the phase before it is known to be: otherwise it passes on the
    // one before that. The parts of a tile are dealt to the converter warps in turn, so a warp skips some tile's keys or
    // values, and has not seen for itself that their codes landed. Before it waits for the codes of its own tile it
    // therefore waits until the producer has found their stage free (info_full for keys, v_turn for values): the codes
    // before them in the stage have then landed and been converted. Those two rings it may wait on because it meets every
    // tile: of tile j - 1, which comes behind tile j - RING, it has seen one or the other.
    static_assert(kConverters <= 8 && RING >= 2, "a converter warp takes at least one of a tile's eight parts");
    // The same of the operand tiles: before it waits for the product of tile j - NS, that of tile j - 2 NS is known to be done, because
    // the codes of tile j - NSC / 2 could only be converted behind the product of tile j - NSC / 2 - NS.
    static_assert(NSC / 2 <= NSK && NSC / 2 <= NSV, "operand tiles are waited for one use at a time");
};

// One key tile.
struct ChunkTile {
    uint32_t what;     // kInfoMasked and the pages that exist; kInfoEnd: no tile, the share is done
    int limit;         // keys of the request from its first key on
    int pad[2];
    float k[8], v[8];  // scales of keys [16 i, 16 i + 16)
};
static_assert(sizeof(ChunkTile) <= 128, "tile ring");

// A unit's part in one CTA, as the producer describes it to the other warps.
struct ChunkPiece {
    int tiles, key0;        // key tiles (0: the share is done), first key
    int kv, pos;            // the request's keys, position of the unit's first token
    int row0, tokens;       // first row of q, tokens of the unit
    int head, slot;         // key/value head; slot of a piece or -1
};
static_assert(2 * sizeof(ChunkPiece) <= 128, "piece ring");

constexpr uint32_t kInfoEnd = 0x200;
constexpr uint32_t kInfoMasked = 0x100;  // some row does not see all of the tile; bits 0-7: pages of 16 keys that exist

// mbar_wait for kernels whose waits are inline: the first one that runs out leaves its role and site in the abort flag, from
// where the block's end takes it to the error word.
__device__ __forceinline__ bool chunk8_wait(uint64_t* bar, uint32_t parity, volatile int* flag, uint32_t role, uint32_t site) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    do {
        if (mbar_try_wait(a, parity)) return true;
        if (*flag) return false;
    } while (globaltimer_ns() - t0 <= kWaitLimitNs);
    *flag = int((role << 16) | site);
    return false;
}

// 16 codes as bf16 times a power of two, exactly: two pieces of 8.
__device__ __forceinline__ void widen16(const uint4& c, float scale, uint4& lo, uint4& hi) {
    const uint32_t r[4] = {c.x, c.y, c.z, c.w};
    const float2 by = make_float2(scale, scale);
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        e4m3_to_f16(r[i], h[0], h[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float2 f = mul2(__half22float2(reinterpret_cast<const __half2&>(h[x])), by);
            out[2 * i + x] = pack_bf16(f.x, f.y);
        }
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]);
    hi = make_uint4(out[4], out[5], out[6], out[7]);
}

// behind_decode: launched behind the decode kernel of the same call, with which it shares inputs but no
// output: its CTAs take the SMs as that kernel's leave them, and wait for it only before they end, so that
// what follows finds both done. The inputs are complete: the decode kernel waited for them before it
// released this one.
template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
paged_chunk8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedParams p, const PagedScales scales,
                    int log_rows /* of one page copy */, int behind_decode) {
    using C = Chunk8Cfg<D>;
    constexpr int NSK = C::NSK, NSV = C::NSV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V, *sC = smem + C::OFF_C;
    ChunkPiece* pieces = reinterpret_cast<ChunkPiece*>(smem + C::OFF_PIECE);  // [2]
    auto tile_info = [&](int n) { return reinterpret_cast<ChunkTile*>(smem + C::OFF_INFO + (n % C::RING) * 128); };
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* q_empty = q_full + 1;
    uint64_t* k_full = q_empty + 1;         // [NSK]
    uint64_t* k_empty = k_full + NSK;       // [NSK]
    uint64_t* v_full = k_empty + NSK;       // [NSV]
    uint64_t* v_empty = v_full + NSV;       // [NSV]
    uint64_t* s_full = v_empty + NSV;       // [2][2], by tile; with AHEAD by parity of its key tiles too
    uint64_t* p_full = s_full + 4;          // [2][2], the same
    uint64_t* o_done = p_full + 4;          // [2], by tile: a piece's products, with AHEAD a key tile's
    uint64_t* piece_full = o_done + 2;      // [2]
    uint64_t* piece_empty = piece_full + 2; // [2], MMA issuer and eight softmax warps
    uint64_t* info_full = piece_empty + 2;  // [RING]
    uint64_t* v_turn = info_full + C::RING;  // [RING], by tile: the stage of its values' codes is free
    uint64_t* c_full = v_turn + C::RING;     // [NSC]
    uint64_t* c_empty = c_full + C::NSC;     // [NSC], the converter warps
    uint64_t* drain = c_empty + C::NSC;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

    grid_release();
    const int warp = int(warp_id()), lane = int(lane_id());
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < NSK; ++i) {
            mbar_init(k_full + i, 4);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(v_full + i, 4);
            mbar_init(v_empty + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(o_done + t, 1);
            mbar_init(piece_full + t, 1);
            mbar_init(piece_empty + t, 9);
        }
        for (int i = 0; i < C::RING; ++i) {
            mbar_init(info_full + i, 1);
            mbar_init(v_turn + i, 1);
        }
        for (int i = 0; i < C::NSC; ++i) {
            mbar_init(c_full + i, 1);
            mbar_init(c_empty + i, 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    const int TOK = p.unit_tokens / 2;  // tokens of a tile
    // place and phase of the barriers of tile t's c-th key tile
    auto tile_bar = [](uint64_t* bars, int t, int c) { return bars + (C::AHEAD ? 2 * t + (c & 1) : t); };
    auto tile_phase = [](int c) { return uint32_t(C::AHEAD ? c >> 1 : c) & 1u; };
    auto next_buffer = [](int b, int by) { return b + by < 3 ? b + by : b + by - 3; };  // AHEAD
    if (!behind_decode) grid_wait();
    const int cta = int(blockIdx.x);
    PagedWalk<kTile, kChunkUnitCost> w;
    int64_t* costs = reinterpret_cast<int64_t*>(smem);  // before the first copy
    if (p.B > kFewRequests)
        paged_share_block<kTile, kChunkUnitCost, kChunkThreads>(p, kChunkMinCost, reinterpret_cast<int64_t*>(smem + C::OFF_SH), w);
    else if (p.B > kLaneRequests) paged_costs<kTile, kChunkUnitCost, kChunkThreads>(p, costs);
    __syncwarp();  // threads leave their requests' loops one by one; what follows is for whole warps
    if (warp == 1) tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* ab = abort_flag;

    // each warpgroup gives or takes its registers at the head of its branch, where the compiler counts them
    if (warp < 4 || warp >= 12) {
        regs_dec<kRegsOther>();
        if (warp == 0) {
            // ------------------------------------------------------------------ producer
            if (lane == 0) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
            }
            if (p.B <= kLaneRequests) paged_share_lanes(p, kChunkMinCost, w);
            else if (p.B <= kFewRequests) paged_share_warp(p, kChunkMinCost, costs, w);
            // lane l of the first 16 looks up the page of keys [16 (l % 8), + 16), and the scale of the keys (l < 8) or values
            // there; the first of a copy's lanes issues it
            const int my_key = (lane & 7) * 16;
            const bool copies = lane < 8 && (my_key & ((1 << log_rows) - 1)) == 0;
            auto lookup = [&](int key0) {
                const int key = key0 + my_key;
                const int id = lane < 16 && key < w.s.kv ? p.table[w.i * p.table_stride + (key >> p.page_shift)] : -1;
                return unsigned(id) < unsigned(p.num_pages) ? id : -1;
            };
            const uint8_t* scale_of = lane < 8 ? scales.k : scales.v;
            auto scale = [&](int id, int key0) {
                if (id < 0) return 127;
                const int token = (key0 + my_key) & ((1 << p.page_shift) - 1);
                const int64_t at = (int64_t(id) << (p.page_shift - scales.block_shift)) + (token >> scales.block_shift);
                return int(scale_of[at * p.Hkv + w.head]);
            };
            PagedMeta meta{0, 0, 0, 0};
            int n = 0, nc = 0, nq = 0, piece = 0;  // tiles, stages of codes, copies of queries and pieces so far
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
                return __all_sync(0xffffffffu, chunk8_wait(bar, parity, ab, ROLE_LOAD, site));
            };
            auto room = [&](uint32_t site) { return nc < C::NSC || wait(c_empty + nc % C::NSC, ((nc / C::NSC) - 1) & 1, site); };
            auto copy = [&](const CUtensorMap* map, int id, int key0) {
                const int st = nc++ % C::NSC;
                if (lane == 0) mbar_arrive_expect_tx(c_full + st, C::CODE_BYTES);
                __syncwarp();
                // a page that does not exist is copied from behind the pool: zeros
                if (copies)
                    tma_load_5d(sC + st * C::CODE_BYTES + my_key * D, map, c_full + st, 0, (key0 + my_key) & ((1 << p.page_shift) - 1),
                                w.head, id >= 0 ? id : p.num_pages, 0);
            };
            while (ok && w.left > 0) {
                // the next piece: what this CTA does of the walk's unit
                int off, tiles;
                w.take(off, tiles);
                if (tiles == 0) {
                    if (w.left > 0) w.next_unit(p);
                    continue;
                }
                const int tokens = w.t1 - w.t0, row0 = w.s.start + w.t0, pos = w.s.base + w.t0;
                const int key_first = (w.first + off) * kTile;
                int slot = -1;
                if (piece == 0 && off > 0) {
                    slot = 2 * cta;
                } else if (off + tiles < w.count) {
                    slot = 2 * cta + 1;
                    meta = PagedMeta{w.pieces(cta), w.head, row0, tokens * p.G};
                }
                if (piece >= 2 && !(ok = wait(piece_empty + (piece & 1), ((piece >> 1) - 1) & 1, 1))) break;
                if (lane == 0) {
                    pieces[piece & 1] = ChunkPiece{tiles, key_first, w.s.kv, pos, row0, tokens, w.head, slot};
                    mbar_arrive(piece_full + (piece & 1));
                }
                int id = lookup(key_first);
                int byte = scale(id, key_first);
                for (int i = 0; i < tiles; ++i) {
                    const int key0 = key_first + i * kTile;
                    const int id_next = i + 1 < tiles ? lookup(key0 + kTile) : -1;
                    if (!(ok = room(2))) break;
                    const uint32_t valid = __ballot_sync(0xffffffffu, id >= 0) & 0xffu;
                    ChunkTile* t = tile_info(n);
                    if (lane < 16) (lane < 8 ? t->k : t->v)[lane & 7] = __uint_as_float(uint32_t(byte) << 23);
                    if (lane == 0) {
                        // clear: every row of the unit sees every key of the tile
                        const bool clear = valid == 0xff && key0 + kTile <= w.s.kv &&
                                           (!p.causal || (key0 + kTile <= pos + 1 && (p.window == 0 || key0 > pos + tokens - 1 - p.window)));
                        t->what = valid | (clear ? 0u : kInfoMasked);
                        t->limit = w.s.kv - key0;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(info_full + n % C::RING);
                    copy(&tm_k, id, key0);
                    if (i == 0) {
                        // the unit's queries, once the previous piece's last scores are computed
                        if (piece >= 1 && !(ok = wait(q_empty, (piece - 1) & 1, 3))) break;
                        const int n_t = tokens > TOK ? 2 : 1;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full, uint32_t(n_t * (D / 64)) * uint32_t(TOK * p.G) * 128u);
                            for (int t = 0; t < n_t; ++t)
                                for (int c = 0; c < D / 64; ++c)
                                    tma_load_5d(sQ + t * C::TILE_BYTES + c * C::CHUNK_BYTES, &tm_q, q_full, 0, w.head * p.G,
                                                row0 + t * TOK, c, 0);
                        }
                        __syncwarp();
                        ++nq;
                    }
                    if (!(ok = room(4))) break;
                    if (lane == 0) mbar_arrive(v_turn + n % C::RING);
                    ++n;
                    copy(&tm_v, id, key0);
                    id = id_next;
                    byte = scale(id, key0 + kTile);
                }
                if (!ok) break;
                ++piece;
                if (w.left > 0) w.next_unit(p);
            }
            if (ok && (ok = room(6)) && lane == 0) {
                tile_info(n)->what = kInfoEnd;
                mbar_arrive(info_full + n % C::RING);
                mbar_arrive(v_turn + n % C::RING);
            }
            if (ok && (piece < 2 || (ok = wait(piece_empty + (piece & 1), ((piece >> 1) - 1) & 1, 5))) && lane == 0) {
                pieces[piece & 1].tiles = 0;
                mbar_arrive(piece_full + (piece & 1));
            }
            if (lane == 0) {
                p.parts.meta[cta] = meta;
                // every copy lands before the CTA can exit, also where another role has given up since
                ring_drain<1>(q_full, nq);
                ring_drain<C::NSC>(c_full, nc);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------------ MMA issuer
            {
                const uint32_t one = elect_one();
                auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
                    return __all_sync(0xffffffffu, chunk8_wait(bar, parity, ab, ROLE_MMA, site));
                };
                constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
                constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
                const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
                bool ok = true;
                int j = 0;                          // key tiles so far
                int s0 = 0, s1 = 0, c0 = 0, c1 = 0; // S_t and PV_t so far
                int bs = 0, bp = 0;                 // AHEAD: S buffer of the next S and of the next PV
                auto issue_s = [&](int t, int sk, int& c) {  // S_t = Q_t K^T
                    const uint64_t dq = sdesc_sw128(aQ + t * C::TILE_BYTES, 16, 1024);
                    const uint64_t dk = sdesc_sw128(aK + sk * C::TILE_BYTES, 16, 1024);
                    const uint32_t col = kTile * (C::AHEAD ? bs : t);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t o = (k >> 2) * C::CHUNK_BYTES + (k & 3) * 32;
                        umma_ss_one(one, col, sdesc_add(dq, o), sdesc_add(dk, o), idS, k > 0 ? 1u : 0u);
                    }
                    umma_commit_one(one, tile_bar(s_full, t, c++));
                    bs = next_buffer(bs, 1);
                };
                auto issue_pv = [&](int t, int sv, bool first, bool last) {  // O_t (+)= P_t V
                    const uint64_t dv = sdesc_sw128(aV + sv * C::TILE_BYTES, C::CHUNK_BYTES, 1024);
                    const uint32_t col = kTile * (C::AHEAD ? bp : t);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)  // 16 keys = 8 TMEM columns of P per step
                        umma_ts_one(one, C::COL_O + D * t, col + k * 8, sdesc_add(dv, k * 2048), idO, (!first || k > 0) ? 1u : 0u);
                    if (C::AHEAD || last) umma_commit_one(one, o_done + t);
                    bp = next_buffer(bp, 1);
                };
                for (int piece = 0; ok; ++piece) {
                    if (!(ok = wait(piece_full + (piece & 1), (piece >> 1) & 1, 1))) break;
                    const int n = pieces[piece & 1].tiles;
                    const bool two = pieces[piece & 1].tokens > TOK;
                    if (n == 0) break;
                    __syncwarp();
                    if (one) mbar_arrive(piece_empty + (piece & 1));
                    if (!(ok = wait(q_full, piece & 1, 2))) break;
                    if (!(ok = wait(k_full + j % NSK, (j / NSK) & 1, 3))) break;
                    tc_fence_after();
                    issue_s(0, j % NSK, s0);
                    if (two) issue_s(1, j % NSK, s1);
                    umma_commit_one(one, k_empty + j % NSK);
                    if (n == 1) umma_commit_one(one, q_empty);
                    for (int i = 0; i < n; ++i, ++j) {
                        const bool next = i + 1 < n;
                        const int sv = j % NSV, sk = (j + 1) % NSK;
                        if (C::AHEAD && next) {
                            if (!(ok = wait(k_full + sk, ((j + 1) / NSK) & 1, 6))) break;
                            tc_fence_after();
                            issue_s(0, sk, s0);
                        }
                        if (!(ok = wait(v_full + sv, (j / NSV) & 1, 4))) break;
                        if (!(ok = wait(tile_bar(p_full, 0, c0), tile_phase(c0), 5))) break;
                        ++c0;
                        tc_fence_after();
                        issue_pv(0, sv, i == 0, !next);
                        if (!C::AHEAD && next) {
                            if (!(ok = wait(k_full + sk, ((j + 1) / NSK) & 1, 6))) break;
                            tc_fence_after();
                            issue_s(0, sk, s0);
                        }
                        if (two) {
                            if (C::AHEAD && next) issue_s(1, sk, s1);
                            if (!(ok = wait(tile_bar(p_full, 1, c1), tile_phase(c1), 7))) break;
                            ++c1;
                            tc_fence_after();
                            issue_pv(1, sv, i == 0, !next);
                            if (!C::AHEAD && next) issue_s(1, sk, s1);
                        }
                        if (next) umma_commit_one(one, k_empty + sk);
                        if (i + 2 == n) umma_commit_one(one, q_empty);  // the piece's last scores are under way
                        umma_commit_one(one, v_empty + sv);
                    }
                }
                // every product is over before the tensor memory is freed, also where a softmax warp has given up since
                umma_commit_one(one, drain);
                mbar_drain(drain, 0);
            }
        } else {
            // ------------------------------------------------------------------ converters
            const int quarter = lane >> 3;
            // this lane's row within 8, and its 16 codes within 64
            const int my_row = D == 128 ? ((lane & 4) ? quarter ^ 5 : quarter) : 2 * quarter + ((lane >> 2) & 1);
            const int my_unit = lane & 3;
            auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
                return __all_sync(0xffffffffu, chunk8_wait(bar, parity, ab, ROLE_LOAD, site));
            };
            // 32 rows of a tile of keys or values, in two halves of four units: the codes of a half first, so that no unit's loads
            // stand behind another's stores, and a loop, because the roles' code together is more than the instruction cache
            // likes (8192 new tokens over 16384 keys, at the time with four converter warps: 1366 us; without the loop
            // 1500 us; with a copy of it for tiles that reach the request's end 1650 us; loops of two units, one behind the
            // other's loads, 1495 us).
            auto convert = [&](uint8_t* tile, int stage, int part, const float* by, int limit) {
                const uint32_t codes = smem_u32(sC + stage * C::CODE_BYTES), out = smem_u32(tile);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint4 x[2][D / 64];
#pragma unroll
                    for (int g = 0; g < 2; ++g)  // 8 rows each
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            x[g][c] = ld_shared_v4u(codes + code_offset<D>(32 * part + 16 * h + 8 * g + my_row, 4 * c + my_unit));
                    const float s = by[part * 2 + h];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int row = 32 * part + 16 * h + 8 * g + my_row;
                        const uint32_t a = out + row * 128, sw = row & 7;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            uint4 lo, hi;
                            widen16(x[g][c], s, lo, hi);
                            if (row >= limit) lo = hi = make_uint4(0, 0, 0, 0);
                            st_shared_v4(a + c * C::CHUNK_BYTES + (((2 * my_unit) ^ sw) << 4), lo.x, lo.y, lo.z, lo.w);
                            st_shared_v4(a + c * C::CHUNK_BYTES + (((2 * my_unit + 1) ^ sw) << 4), hi.x, hi.y, hi.z, hi.w);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            // a tile's keys and values are eight parts, dealt to the warps in turn
            for (int x = warp < 4 ? warp - 2 : warp - 10;; x += kConverters) {
                const int j = x >> 3, value = (x >> 2) & 1, part = x & 3, nc = 2 * j + value;
                if (!wait((value ? v_turn : info_full) + j % C::RING, (j / C::RING) & 1, 11)) break;
                const ChunkTile* t = tile_info(j);
                if (t->what & kInfoEnd) break;
                const int ns = value ? NSV : NSK, st = j % ns;
                uint64_t *full = (value ? v_full : k_full) + st, *empty = (value ? v_empty : k_empty) + st;
                if (!wait(c_full + nc % C::NSC, (nc / C::NSC) & 1, 12)) break;
                if (j >= ns && !wait(empty, ((j / ns) - 1) & 1, 13)) break;
                convert((value ? sV : sK) + st * C::TILE_BYTES, nc % C::NSC, part, value ? t->v : t->k, value ? t->limit : kTile);
                if (lane == 0) {
                    mbar_arrive(full);
                    mbar_arrive(c_empty + nc % C::NSC);
                }
            }
        }
    } else {
        // ------------------------------------------------------------------ softmax (tile t)
        regs_inc<kRegsSoftmax>();
        const int t = warp < 8 ? 0 : 1;
        const int wq = warp & 3;                  // TMEM lane quadrant of this warp
        const int row = wq * 32 + lane;           // row within the tile (TMEM lane)
        const uint32_t lane_off = uint32_t(wq * 32) << 16;
        uint32_t tS = tmem + kTile * t + lane_off;
        const uint32_t tO = tmem + C::COL_O + D * t + lane_off;
        const int tok = row / p.G;                // the row's token within the tile
        bool ok = true;
        int j = 0, cs = 0, units = 0;             // key tiles so far; this tile's S and O so far
        int buffer0 = 0;                          // AHEAD: S buffer of the piece's first scores
        for (int piece = 0; ok; ++piece) {
            ok = __all_sync(0xffffffffu, chunk8_wait(piece_full + (piece & 1), (piece >> 1) & 1, ab, ROLE_SOFTMAX, 1));
            if (!ok) break;
            // read again where needed: registers are short in the loop below
            const volatile ChunkPiece& u = pieces[piece & 1];
            const int tiles = u.tiles;
            if (tiles == 0) break;
            auto done_with_piece = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(piece_empty + (piece & 1));
            };
            const bool valid = tok < u.tokens - t * TOK && tok < TOK;
            if (u.tokens <= t * TOK) {  // the unit has one tile
                done_with_piece();
                j += tiles;
                if (C::AHEAD) buffer0 = next_buffer(buffer0, tiles % 3);
                continue;
            }
            int width = 0, buffer = 0;                // AHEAD: tiles of the unit, S buffer
            if (C::AHEAD) {
                width = u.tokens > TOK ? 2 : 1;
                buffer = next_buffer(buffer0, t);
                buffer0 = next_buffer(buffer0, width * tiles % 3);
            }
            const int kv = u.kv;
            int key0 = u.key0;
            float m_used = -INFINITY, l_sum = 0.f;  // running maximum (log2 domain) and sum
            for (int i = 0; i < tiles; ++i, ++j, key0 += kTile) {
                const int c = cs++;
                if (C::AHEAD) tS = tmem + kTile * buffer + lane_off;
                ok = __all_sync(0xffffffffu, chunk8_wait(tile_bar(s_full, t, c), tile_phase(c), ab, ROLE_SOFTMAX, 2) &&
                                                 chunk8_wait(info_full + j % C::RING, (j / C::RING) & 1, ab, ROLE_SOFTMAX, 3));
                if (!ok) break;
                tc_fence_after();
                const uint32_t what = tile_info(j)->what;
                const bool masked = what & kInfoMasked;
                // all 128 scores of the row at once in registers: one trip through TMEM, four independent
                // chains for the maximum and the sum
                float v[128];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld32(tS + x * 32, v + x * 32);
                tmem_wait_ld();
                if (masked) {
                    // the row sees keys [lo, hi)
                    const int pos = u.pos + t * TOK + tok;
                    const int hi = p.causal ? max(0, min(kv, pos + 1)) : kv, lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                    const int h = hi - key0, b = lo - key0;
#pragma unroll
                    for (int x = 0; x < 128; ++x)
                        if (x >= h || x < b || !((what >> (x / 16)) & 1u)) v[x] = -INFINITY;
                }
                float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int x = 4; x < 128; ++x) mx4[x & 3] = fmaxf(mx4[x & 3], v[x]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                const float m_new = fmaxf(m_used, mx * p.scale_log2);
                const bool need = valid && m_new > m_used + 8.0f;
                const float alpha = need ? ex2(m_used - m_new) : 1.0f;  // ex2(-inf) = 0 for a first maximum
                if (need) m_used = m_new;
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                // the weights over the scores' first 64 columns, all read by now. The matrix product takes them in bf16, the
                // type of the values, off by at most 2^-8 of a weight; their sum is taken of the weights before
                // (errors against 64 bits: 1.2 to 1.4 times those of fp32 weights)
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(neg_m, neg_m);
                float2 rs4[4] = {};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 e = fma2(make_float2(v[32 * g + 2 * x], v[32 * g + 2 * x + 1]), sc2, nm2);
                        e.x = ex2(e.x);
                        e.y = ex2(e.y);
                        rs4[x & 3] = add2(rs4[x & 3], e);
                        pk[x] = pack_bf16(e.x, e.y);
                    }
                    tmem_st16_u(tS + g * 16, pk);
                }
                rs4[0] = add2(add2(rs4[0], rs4[1]), add2(rs4[2], rs4[3]));
                const float rs = rs4[0].x + rs4[0].y;
                l_sum = l_sum * alpha + rs;
                if (C::AHEAD && i > 0) {
                    // O_t holds still between the product of the key tile before and this one's
                    ok = __all_sync(0xffffffffu, chunk8_wait(o_done + t, units++ & 1, ab, ROLE_SOFTMAX, 5));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (i > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int x = 0; x < D / 32; ++x) {
                        float o[32];
                        tmem_ld32(tO + x * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int y = 0; y < 32; ++y) o[y] *= alpha;
                        tmem_st32(tO + x * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tile_bar(p_full, t, c));
                if (C::AHEAD) buffer = next_buffer(buffer, width);
            }
            if (!ok) break;
            // -------------------------------------------------------------- the piece's rows
            ok = __all_sync(0xffffffffu, chunk8_wait(o_done + t, units++ & 1, ab, ROLE_EPI, 1));
            if (!ok) break;
            tc_fence_after();
            const bool any_key = l_sum != 0.f;  // NaN scores stay NaN
            const int slot = u.slot;
            const float inv = slot >= 0 ? 1.0f : (any_key ? 1.0f / l_sum : 0.f);
            const int unit_row = t * TOK * p.G + row;
            const int q_row = u.row0 + t * TOK + tok, h = u.head * p.G + row % p.G;
            __nv_bfloat16* dst = p.o + (int64_t(q_row) * p.H + h) * D;
            const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // o may be 16-byte aligned only
            float* part = p.parts.o + (int64_t(max(slot, 0)) * kChunkRows + unit_row) * D;
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
                float o[32];
                __syncwarp();  // rows that stored and rows that did not, together again
                tmem_ld32(tO + x * 32, o);
                tmem_wait_ld();
                if (!valid) continue;
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] *= inv;
                if (slot >= 0) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) st_global_v8(part + x * 32 + y * 8, reinterpret_cast<const uint32_t*>(o + 8 * y));
                } else {
                    uint32_t pk[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) pk[y] = pack_bf16(o[2 * y], o[2 * y + 1]);
                    if (wide) {
                        st_global_v8(dst + x * 32, pk);
                        st_global_v8(dst + x * 32 + 16, pk + 8);
                    } else {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            reinterpret_cast<uint4*>(dst + x * 32)[y] = make_uint4(pk[4 * y], pk[4 * y + 1], pk[4 * y + 2], pk[4 * y + 3]);
                    }
                }
            }
            if (valid) {
                if (slot >= 0) p.parts.ml[int64_t(slot) * kChunkRows + unit_row] = make_float2(m_used, l_sum);
                else p.lse[int64_t(h) * p.T + q_row] = any_key ? (m_used + log2f(l_sum)) * 0.69314718055994531f : -INFINITY;
            }
            done_with_piece();
            tc_fence_before();
        }
        tmem_wait_st();  // of a warp that has given up with weights on their way
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_error(p.err, (KID_PAGED << 24) | uint32_t(*abort_flag));
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (behind_decode) grid_wait();
}

template <int D>
int launch_chunk8_d(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream) {
    using C = Chunk8Cfg<D>;
    CUtensorMap mq;
    {
        const int tok = p.unit_tokens / 2;
        cuuint64_t dims[5] = {64, cuuint64_t(p.H), cuuint64_t(p.T), D / 64, 1};
        cuuint64_t strides[4] = {D * 2, cuuint64_t(p.q_stride) * 2, 128, 128};
        cuuint32_t box[5] = {64, cuuint32_t(p.G), cuuint32_t(tok), 1, 1};
        cuuint32_t estr[5] = {1, 1, 1, 1, 1};
        if (!encode_tensor_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.q, dims, strides, box, estr)) return ULYSSES_ERR_CUDA;
    }
    const int rows = a.cache.page_size < kTile ? a.cache.page_size : kTile;
    CUtensorMap mk, mv;
    if (!encode_code_pages(&mk, a.cache, a.cache.k, rows) || !encode_code_pages(&mv, a.cache, a.cache.v, rows)) return ULYSSES_ERR_CUDA;
    auto kern = paged_chunk8_kernel<D>;
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ULYSSES_ERR_CUDA;
    return launch_chained(kern, dim3(unsigned(p.parts.ctas)), kChunkThreads, C::SMEM_BYTES, stream, mq, mk, mv, p, a.scales,
                          __builtin_ctz(unsigned(rows)), int(behind_decode))
               ? ULYSSES_OK : ULYSSES_ERR_CUDA;
}

}  // namespace

int launch_paged_chunk8(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream) {
    return a.cache.d_h == 128 ? launch_chunk8_d<128>(a, p, behind_decode, stream) : launch_chunk8_d<64>(a, p, behind_decode, stream);
}

}  // namespace ulysses
