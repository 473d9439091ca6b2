// Dispatch of the paged attention: requests whose rows (new tokens x grouped query heads) fit one 16-row
// fragment go to the decode kernel, the others to the chunk kernel. Which request is which is known on
// the device only, so a call launches both, each passing over the other's requests, unless
// - the caller's bound on new tokens says that the decode kernel's are all: it then takes every request,
//   however long (the bound chooses, it does not decide what is computed);
// - the group is too wide for the decode kernel; or
// - the batch has few units of few rows, at most three to two SMs: the chunk kernel then takes them along, which saves a
//   launch and its fill (24 requests of 8 key/value heads, five of them chunks: 78 us against 83 us; 38: 114 us against
//   111 us; 100 short ones, where its larger cost of a unit counts: 102 us against 90 us).
//   Over an 8-bit cache, at most one to two SMs: the chunk kernel has codes to widen whatever a unit's rows (24 requests of 8
//   key/value heads, some of them chunks: 97 us with both kernels, 104 us with one; 40 of 4 heads of 64: 44.7 us, 46.9 us; one
//   chunk of 40 tokens over 1000 keys: 20.2 us, 17.4 us).
#include <algorithm>

#include "paged_common.cuh"

namespace ulysses {

namespace {

bool decode_fits(int G) { return G <= paged_decode_rows(); }
bool decode_only(int G, int max_q) { return decode_fits(G) && max_q > 0 && int64_t(max_q) * G <= paged_decode_rows(); }

}  // namespace

bool encode_pages(CUtensorMap* map, const ulysses_kv_cache_t& c, const void* base, int rows, int chunks) {
    cuuint64_t dims[5] = {64, cuuint64_t(c.page_size), cuuint64_t(c.H_kv), cuuint64_t(c.num_pages), cuuint64_t(c.d_h / 64)};
    cuuint64_t strides[4] = {cuuint64_t(c.token_stride) * 2, cuuint64_t(c.head_stride) * 2, cuuint64_t(c.page_stride) * 2, 128};
    cuuint32_t box[5] = {64, cuuint32_t(rows), 1, 1, cuuint32_t(chunks)};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dims, strides, box, estr);
}

bool encode_code_pages(CUtensorMap* map, const ulysses_kv_cache_t& c, const void* base, int rows) {
    cuuint64_t dims[5] = {cuuint64_t(c.d_h), cuuint64_t(c.page_size), cuuint64_t(c.H_kv), cuuint64_t(c.num_pages), 1};
    cuuint64_t strides[4] = {cuuint64_t(c.token_stride), cuuint64_t(c.head_stride), cuuint64_t(c.page_stride), cuuint64_t(c.page_stride)};
    cuuint32_t box[5] = {cuuint32_t(c.d_h), cuuint32_t(rows), 1, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, estr,
                             c.d_h == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                             c.d_h == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
}

// Behind the decode kernel alone one block joins a whole unit, of up to a dozen pieces and more; with the
// chunk kernel, whose units are 256 rows of mostly two or three pieces, smaller blocks that read two at a
// time keep more of them in flight (a chunk call of 1.2 PFLOP/s: 237 us, against 243 us with eight).
constexpr int kJoinManyThreads = 256, kJoinManyPieces = 2;

template <int D, int NT, int N>
static int launch_join_t(const PagedParams& p, const PagedParts& decode, const PagedParts& chunk, cudaStream_t stream) {
    const int64_t blocks = int64_t(std::max(decode.ctas - 1, 0)) * (decode.rows * D / (4 * NT)) +
                           int64_t(std::max(chunk.ctas - 1, 0)) * (chunk.rows * D / (4 * NT));
    if (blocks == 0) return ULYSSES_OK;
    return launch_chained(paged_join_kernel<D, NT, N>, dim3(unsigned(blocks)), NT, 0, stream, p, decode, chunk) ? ULYSSES_OK
                                                                                                             : ULYSSES_ERR_CUDA;
}

template <int D>
static int launch_join(const PagedParams& p, const PagedParts& decode, const PagedParts& chunk, cudaStream_t stream) {
    if (chunk.ctas == 0) return launch_join_t<D, 4 * D, 8>(p, decode, chunk, stream);
    return launch_join_t<D, kJoinManyThreads, kJoinManyPieces>(p, decode, chunk, stream);
}

size_t paged_attn_workspace_bytes(int H, int H_kv, int d_h, int max_q) {
    const int G = H / H_kv;
    size_t decode = 0, chunk = 0;
    if (decode_fits(G)) paged_decode_parts(nullptr, d_h, 0, &decode);
    if (!decode_only(G, max_q)) paged_chunk_parts(nullptr, d_h, 0, &chunk);
    return decode + chunk;
}

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
    PagedParams p{};
    p.B = a.B; p.T = a.T; p.H = a.H; p.Hkv = a.cache.H_kv; p.G = a.H / a.cache.H_kv;
    p.max_pages = a.max_pages; p.num_pages = a.cache.num_pages;
    p.page_shift = __builtin_ctz(unsigned(a.cache.page_size));
    p.causal = a.causal; p.window = a.window;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.q_stride = a.q_stride; p.table_stride = a.table_stride;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.cu_q = a.cu_q; p.kv_lens = a.kv_lens; p.table = a.table;
    p.o = static_cast<__nv_bfloat16*>(a.o);
    p.lse = a.lse;
    p.err = device_error_word();
    if (!p.err) return ULYSSES_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    const int d = a.cache.d_h, sms = device_sm_count();
    const bool codes = a.scales.k != nullptr;
    const bool only = decode_only(p.G, a.max_q);
    PagedParts decode{}, chunk{};
    size_t bytes = 0;
    const bool both = decode_fits(p.G) && 2 * int64_t(p.B) * p.Hkv > (codes ? 1 : 3) * sms;
    p.min_rows = 1;
    if (only || both) {
        p.max_rows = only ? 0x7fffffff : paged_decode_rows();
        p.unit_tokens = paged_decode_rows() / p.G;
        p.parts = decode = paged_decode_parts(ws, d, sms, &bytes);
        const int rc = codes ? launch_paged_decode8(a, p, stream) : launch_paged_decode(a, p, stream);
        if (rc != ULYSSES_OK) return rc;
        p.min_rows = paged_decode_rows() + 1;
    }
    if (!only) {
        p.max_rows = 0x7fffffff;
        p.unit_tokens = 2 * (kTile / p.G);
        p.parts = chunk = paged_chunk_parts(ws + bytes, d, sms, &bytes);
        const int rc = codes ? launch_paged_chunk8(a, p, both, stream) : launch_paged_chunk(a, p, both, stream);
        if (rc != ULYSSES_OK) return rc;
    }
    return d == 128 ? launch_join<128>(p, decode, chunk, stream) : launch_join<64>(p, decode, chunk, stream);
}

}  // namespace ulysses
