// Paged attention for chunks of new rows on the 5th-generation tensor cores (tcgen05, TMEM, TMA).
//
// A unit is up to 256 rows of one request with one key/value head: the rows of a token's grouped query
// heads lie next to one another (row = token x G + head), so that every key/value tile brought into
// shared memory serves all of them. Its two 128-row tiles share the key/value tiles, which halves their
// traffic per product, and their softmax warpgroups alternate, so that the tensor core works on one
// tile while the other's softmax runs. One CTA per SM walks its share of the batch's key tiles
// (paged_common.cuh); the pipeline runs on across units: while a unit's rows are normalised and stored,
// the next one's first scores are computed. Warp roles (320 threads):
//   warp 0    producer: walks the share, looks up the pages (one lane per page copy) and keeps the Q, K
//             and V copies going; publishes each piece (a unit's part in this CTA) and each tile's
//             missing pages;
//   warp 1    MMA issuer: S_t = Q_t K^T into a 128-column buffer of TMEM and O_t += P_t V into columns of its own, P_t
//             read from the first 64 columns of S_t's buffer as packed bf16 pairs. The warp runs converged and one
//             elected thread issues;
//   warps 2-5 softmax of tile 0, warps 6-9 of tile 1: thread i owns row i (TMEM lane i). It takes the row's
//             128 scores into registers, writes the weights over them, rescales O_t when the maximum grew by
//             more than 2^8, and stores the row at the end of the unit, or leaves it as a piece.
// One thread issues all products, and its tcgen05 operations complete in order.
// d = 128: S_t has buffer t, and PV_t of a key tile is issued before S_t of the next: when that is there, the
// previous PV_t is over, so O_t may be rescaled and S_t's columns reused.
// d = 64 (AHEAD): O leaves room for a third S buffer. The scores, in the order of their issue, take the three in turn,
// and S_t of a key tile is issued before PV_t of the one before, so that it is ready when that one's weights
// are done (8192 new tokens over 16384 keys, 32/8 heads: 760 us, against 855 us with two buffers). The buffer
// it takes held weights whose product is issued before it. O_t is rescaled once PV_t of the key tile before has
// completed. A fast warp may be one key tile ahead of its tile's others, hence two barriers by parity.
// A piece's first PV_t waits for that tile's weights, which its warps write only after they have read the
// previous piece's O_t.
// Values behind a request's last key may be anything: in the tile that holds the end, warps 2-5 clear
// those rows of V in shared memory before the product reads them (0 x NaN is NaN).
//
// What bounds it (32/8 heads of 128, 8192 new tokens over 16384 keys: 1050 to 1060 us, 1.56 PFLOP/s, 0.82 of the
// measured bf16 rate; 1000 us on the card where the other figures of this paragraph were taken): a step of 256 rows
// and 128 keys takes 2970 cycles, of which the issuer spends 2100 on its 32 MMAs, the tensor core's own rate, and 630
// waiting for weights: a tile's chain softmax (1530) -> PV, S (1050) is longer than the other tile's products.
// Tried and slower: one tile with three S buffers (the key/value
// traffic doubles and the L2 bounds it: 1420 us); 64-key halves with two S buffers a tile (N = 64 products
// cost nearly what N = 128 do: 1200 us); half a row to a thread with 16 softmax warps (1195 us); PV issued by
// halves of P (no difference). d = 64, P in columns of its own so that both tiles' scores come a key tile
// ahead: 980 us, both tiles' weights are then computed at once and neither's beside the products.
#include <algorithm>

#include "paged_common.cuh"

namespace ulysses {

namespace {

constexpr int kChunkThreads = 320;
constexpr int kChunkRows = 2 * kTile;
constexpr int kChunkMaxCtas = 160;   // one per SM: sizes the workspace
// The smallest share of a CTA, in key tiles. Only calls that leave CTAs idle notice: one chunk of 40 tokens over 1000 keys
// takes 22.1 us with 4, 27.4 us with 8 and 19.5 us with 2, two of 100 over 500 24.0, 23.3 and 21.5 us. 4 is from before
// such calls were measured.
constexpr int kChunkMinCost = 4;
// The fixed cost of a unit, in key tiles, with 1, 2, 3, 4: 24 mixed requests 88.2, 76.9, 77.3, 77.8 us (heads of 64: 69.8,
// 58.1, 54.8, 55.3 us), four chunks of 512 tokens 226, 217, 210, 208 us.
constexpr int kChunkUnitCost = 3;
constexpr int kInfoRing = 8;         // tiles that the producer may describe ahead (it leads by at most 7)

template <int D>
struct ChunkCfg {
    static constexpr int NSK = D == 64 ? 6 : 3;  // K and V pipeline stages
    static constexpr int NSV = D == 64 ? 6 : 2;
    static constexpr uint32_t TILE_BYTES = kTile * D * 2;
    static constexpr uint32_t CHUNK_BYTES = kTile * 128;  // 128 rows x 64 elements, swizzled
    static constexpr uint32_t OFF_K = 2 * TILE_BYTES;
    static constexpr uint32_t OFF_V = OFF_K + NSK * TILE_BYTES;
    static constexpr uint32_t OFF_PIECE = OFF_V + NSV * TILE_BYTES;
    static constexpr uint32_t OFF_INFO = OFF_PIECE + 128;
    static constexpr uint32_t OFF_SH = OFF_INFO + kInfoRing * 4;
    static constexpr uint32_t OFF_BAR = OFF_SH + 128;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 512 + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
    // TMEM: S buffers, O0, O1. d = 64 leaves room for a third S buffer.
    static constexpr bool AHEAD = D == 64;
    static constexpr uint32_t COL_O = (AHEAD ? 3 : 2) * kTile, TMEM_COLS = 512;
    static_assert(COL_O + 2 * D <= TMEM_COLS, "tensor memory");
    // the issuer names columns from 0, constants of its instructions: true of an allocation of the whole tensor memory
    static_assert(TMEM_COLS == 512, "the allocation starts at column 0");
    static_assert(NSK + (AHEAD ? 2 : 1) <= kInfoRing, "tile descriptions outlive their readers");
};

// A unit's part in one CTA, as the producer describes it to the other warps.
struct ChunkPiece {
    int tiles, key0;        // key tiles (0: the share is done), first key
    int kv, pos;            // the request's keys, position of the unit's first token
    int row0, tokens;       // first row of q, tokens of the unit
    int head, slot;         // key/value head; slot of a piece or -1
};
static_assert(2 * sizeof(ChunkPiece) <= 128, "piece ring");

constexpr uint32_t kInfoMasked = 0x100;  // some row does not see all of the tile; bits 0-7: pages of 16 keys that exist

// behind_decode: launched behind the decode kernel of the same call, with which it shares inputs but no
// output: its CTAs take the SMs as that kernel's leave them, and wait for it only before they end, so that
// what follows finds both done. The inputs are complete: the decode kernel waited for them before it
// released this one.
template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PagedParams p, int log_rows /* of one page copy */, int behind_decode) {
    using C = ChunkCfg<D>;
    constexpr int NSK = C::NSK, NSV = C::NSV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V;
    ChunkPiece* pieces = reinterpret_cast<ChunkPiece*>(smem + C::OFF_PIECE);  // [2]
    uint32_t* info = reinterpret_cast<uint32_t*>(smem + C::OFF_INFO);         // [kInfoRing]
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
    uint64_t* info_full = piece_empty + 2;  // [kInfoRing]
    uint64_t* drain = info_full + kInfoRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

    grid_release();
    const int warp = int(warp_id()), lane = int(lane_id());
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < NSK; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 1);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(v_full + i, 1);
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
        for (int i = 0; i < kInfoRing; ++i) mbar_init(info_full + i, 1);
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
    const Abort ab{abort_flag, p.err, KID_PAGED};

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        if (p.B <= kLaneRequests) paged_share_lanes(p, kChunkMinCost, w);
        else if (p.B <= kFewRequests) paged_share_warp(p, kChunkMinCost, costs, w);
        // a copy is one page (or 128 keys of a longer one) by 64 elements, or by the whole head where one
        // copy fills the tile; lane l copies page l / per, 64-element chunk l % per
        const int per = log_rows == 7 ? 1 : D / 64;
        const int copies = (kTile >> log_rows) * per;  // of one tile, at most 16
        const int my_row = (lane / per) << log_rows;
        const int my_chunk = lane % per;
        auto lookup = [&](int key0) {
            const int key = key0 + my_row;
            return lane < copies && key < w.s.kv ? p.table[w.i * p.table_stride + (key >> p.page_shift)] : -1;
        };
        PagedMeta meta{0, 0, 0, 0};
        int nk = 0, nv = 0, nq = 0, piece = 0;  // copies and pieces so far
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, ROLE_LOAD, site));
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
            for (int i = 0; i < tiles; ++i) {
                const int key0 = key_first + i * kTile;
                const int id_next = i + 1 < tiles ? lookup(key0 + kTile) : -1;
                const int sk = nk % NSK, sv = nv % NSV;
                if (nk >= NSK && !(ok = wait(k_empty + sk, ((nk / NSK) - 1) & 1, 2))) break;
                const bool good = unsigned(id) < unsigned(p.num_pages);
                // a page that does not exist is copied from behind the pool: zeros
                const int page = good ? id : p.num_pages, row = (key0 + my_row) & ((1 << p.page_shift) - 1);
                const unsigned have = __ballot_sync(0xffffffffu, good && my_chunk == 0);
                const int of = (min(lane, 7) * 16) >> log_rows;  // the copy of keys [16 lane, 16 lane + 16)
                const uint32_t valid = __ballot_sync(0xffffffffu, lane < 8 && ((have >> (of * per)) & 1u));
                const uint32_t off = my_chunk * C::CHUNK_BYTES + my_row * 128;
                if (lane == 0) {
                    // clear: every row of the unit sees every key of the tile
                    const bool clear = valid == 0xff && key0 + kTile <= w.s.kv &&
                                       (!p.causal || (key0 + kTile <= pos + 1 && (p.window == 0 || key0 > pos + tokens - 1 - p.window)));
                    info[nk % kInfoRing] = valid | (clear ? 0u : kInfoMasked);
                    mbar_arrive(info_full + nk % kInfoRing);
                    mbar_arrive_expect_tx(k_full + sk, C::TILE_BYTES);
                }
                __syncwarp();
                if (lane < copies) tma_load_5d(sK + sk * C::TILE_BYTES + off, &tm_k, k_full + sk, 0, row, w.head, page, my_chunk);
                ++nk;
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
                if (nv >= NSV && !(ok = wait(v_empty + sv, ((nv / NSV) - 1) & 1, 4))) break;
                if (lane == 0) mbar_arrive_expect_tx(v_full + sv, C::TILE_BYTES);
                __syncwarp();
                if (lane < copies) tma_load_5d(sV + sv * C::TILE_BYTES + off, &tm_v, v_full + sv, 0, row, w.head, page, my_chunk);
                ++nv;
                id = id_next;
            }
            if (!ok) break;
            ++piece;
            if (w.left > 0) w.next_unit(p);
        }
        if (ok && (piece < 2 || (ok = wait(piece_empty + (piece & 1), ((piece >> 1) - 1) & 1, 5))) && lane == 0) {
            pieces[piece & 1].tiles = 0;
            mbar_arrive(piece_full + (piece & 1));
        }
        if (lane == 0) {
            p.parts.meta[cta] = meta;
            // every copy lands before the CTA can exit, also where another role has given up since
            ring_drain<1>(q_full, nq);
            ring_drain<NSK>(k_full, nk);
            ring_drain<NSV>(v_full, nv);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        {
            const uint32_t one = elect_one();
            auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, ROLE_MMA, site));
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
        // ------------------------------------------------------------------ softmax (tile t)
        const int t = warp < 6 ? 0 : 1;
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
            ok = __all_sync(0xffffffffu, mbar_wait(piece_full + (piece & 1), (piece >> 1) & 1, ab, ROLE_SOFTMAX, 1));
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
                ok = __all_sync(0xffffffffu, mbar_wait(tile_bar(s_full, t, c), tile_phase(c), ab, ROLE_SOFTMAX, 2) &&
                                                 mbar_wait(info_full + j % kInfoRing, (j / kInfoRing) & 1, ab, ROLE_SOFTMAX, 3));
                if (!ok) break;
                tc_fence_after();
                const uint32_t what = info[j % kInfoRing];
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
                    ok = __all_sync(0xffffffffu, mbar_wait(o_done + t, units++ & 1, ab, ROLE_SOFTMAX, 5));
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
                if (t == 0 && key0 + kTile > kv) {
                    // clear the values behind the last key; tile 1's product follows tile 0's
                    const int sv = j % NSV;
                    ok = __all_sync(0xffffffffu, mbar_wait(v_full + sv, (j / NSV) & 1, ab, ROLE_SOFTMAX, 4));
                    if (!ok) break;
                    if (key0 + row >= kv) {
                        const uint32_t a = smem_u32(sV + sv * C::TILE_BYTES) + row * 128;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
#pragma unroll
                            for (int x = 0; x < 8; ++x) st_shared_v4(a + c * C::CHUNK_BYTES + x * 16, 0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();  // rows that cleared and rows that did not, together again
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tile_bar(p_full, t, c));
                if (C::AHEAD) buffer = next_buffer(buffer, width);
            }
            if (!ok) break;
            // -------------------------------------------------------------- the piece's rows
            ok = __all_sync(0xffffffffu, mbar_wait(o_done + t, units++ & 1, ab, ROLE_EPI, 1));
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
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (behind_decode) grid_wait();
}

template <int D>
int launch_chunk_d(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream) {
    using C = ChunkCfg<D>;
    const int rows = std::min(a.cache.page_size, kTile);
    const int chunks = rows == kTile ? D / 64 : 1;
    CUtensorMap mq, mk, mv;
    {
        const int tok = p.unit_tokens / 2;
        cuuint64_t dims[5] = {64, cuuint64_t(p.H), cuuint64_t(p.T), D / 64, 1};
        cuuint64_t strides[4] = {D * 2, cuuint64_t(p.q_stride) * 2, 128, 128};
        cuuint32_t box[5] = {64, cuuint32_t(p.G), cuuint32_t(tok), 1, 1};
        cuuint32_t estr[5] = {1, 1, 1, 1, 1};
        if (!encode_tensor_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.q, dims, strides, box, estr)) return ULYSSES_ERR_CUDA;
    }
    if (!encode_pages(&mk, a.cache, a.cache.k, rows, chunks) || !encode_pages(&mv, a.cache, a.cache.v, rows, chunks))
        return ULYSSES_ERR_CUDA;
    auto kern = paged_chunk_kernel<D>;
    if (!set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES)) return ULYSSES_ERR_CUDA;
    if (!launch_chained(kern, dim3(unsigned(p.parts.ctas)), kChunkThreads, C::SMEM_BYTES, stream, mq, mk, mv, p,
                        __builtin_ctz(unsigned(rows)), int(behind_decode)))
        return ULYSSES_ERR_CUDA;
    return ULYSSES_OK;
}

}  // namespace

PagedParts paged_chunk_parts(void* workspace, int d_h, int sms, size_t* bytes) {
    return paged_parts(workspace, kChunkMaxCtas, sms, kChunkRows, d_h, bytes);
}

int launch_paged_chunk(const PagedAttnArgs& a, const PagedParams& p, bool behind_decode, cudaStream_t stream) {
    return a.cache.d_h == 128 ? launch_chunk_d<128>(a, p, behind_decode, stream) : launch_chunk_d<64>(a, p, behind_decode, stream);
}

}  // namespace ulysses
