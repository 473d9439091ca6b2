"""GPU parity of the 8-bit cache against its oracle. Codes and scales must be equal. Attention is held to the bounds of
test_paged_gpu.py, of the keys and values that codes and scales stand for (all of them exact in bf16): the kernels' weights
are rounded to 11 bits or to 8, their queries at most to what is 2^-28 of a row's largest."""

import numpy as np
import pytest
import torch

import oracle.cache8 as cache8
import oracle.paged as paged
import ulysses_sequence_gb300 as U
from gpu_util import need_gpu
from test_paged_gpu import KV, Step, healthy, hold, i32

pytestmark = pytest.mark.gpu

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def device(x, dtype, head_major=False):
    """A uint8 array on the GPU as dtype; [page][token][head][d] in head-major memory where asked."""
    t = torch.tensor(x, device="cuda")
    return (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if head_major else t).view(dtype)


# ------------------------------------------------------------------ append

def bf16_rows(rng, *shape, spread=4.0):
    """Rows whose heads differ in size by up to 2^spread either way."""
    x = rng.standard_normal(shape) * 2.0 ** rng.uniform(-spread, spread, (*shape[:-1], 1))
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def run_append(codes, scales, rows, slots, block, head_major=False, fused=False):
    """codes, scales, rows: pairs (keys, values). Checks the GPU against the oracle and returns what it left."""
    kc, vc = (device(c, E4M3, head_major) for c in codes)
    ks, vs = (device(s, E8M0) for s in scales)
    x = [r.cuda() for r in rows]
    if fused:
        both = torch.cat([torch.zeros_like(x[0]), x[0], x[1]], 1)
        H = x[0].shape[1]
        x = [both[:, H:2 * H], both[:, 2 * H:]]
    U.kv_append(x[0], x[1], U.PagedCache8(kc, vc, ks, vs), i32(slots))
    healthy()
    got = []
    for c, s, r, gc, gs in zip(codes, scales, rows, (kc, vc), (ks, vs)):
        wc, ws = cache8.append(c, s, r.double().numpy(), slots, block)
        assert np.array_equal(raw(gs), ws), np.argwhere(raw(gs) != ws)[:4]
        assert np.array_equal(raw(gc), wc), np.argwhere(raw(gc) != wc)[:4]
        got.append((wc, ws))
    return got


def pool(rng, pages, page, H, d, block):
    """Random codes (all patterns, NaN too) and scales around 1, of keys and of values."""
    return ([rng.integers(0, 256, (pages, page, H, d)).astype(np.uint8) for _ in range(2)],
            [rng.integers(110, 130, (pages, page // block, H)).astype(np.uint8) for _ in range(2)])


def placed(rng, lens, page, pages):
    """Slots of requests (first offset, tokens), each from that offset of a page of its own on, pages anywhere."""
    order, slots = list(rng.permutation(pages)), []
    for off, n in lens:
        for t in range(off, off + n):
            if t == off or t % page == 0:
                p = order.pop()
            slots.append(p * page + t % page)
    return np.array(slots)


@pytest.mark.parametrize("H,d,page,block,head_major,fused", [(8, 128, 64, 64, False, False), (1, 64, 16, 16, False, True),
                                                             (5, 128, 256, 32, True, False), (3, 64, 128, 128, False, True),
                                                             (20, 64, 64, 16, True, False), (2, 128, 4096, 4096, False, False)])
def test_append_matches_oracle(H, d, page, block, head_major, fused):
    """Single tokens in the middle, at the start and at the end of blocks, chunks that begin anywhere and pass block and page ends,
    rows of no slot among them."""
    rng = np.random.default_rng(H * d + block)
    lens = [(0, 1), (block - 1, 1), (3, 1), (page - 1, 2), (7, 2 * block + 5), (0, page + 1), (block // 2, 16), (1, 17), (block - 1, 33), (0, 0)]
    pages = sum((o + n - 1) // page + 1 for o, n in lens) + 2
    slots = placed(rng, lens, page, pages)
    pad = [-1, pages * page, 2 ** 31 - 1, -2 ** 31]
    slots = np.concatenate([pad[:1], slots[:3], pad[1:2], slots[3:], pad[2:]])
    codes, scales = pool(rng, pages, page, H, d, block)
    rows = [bf16_rows(rng, len(slots), H, d) for _ in range(2)]
    codes, scales = zip(*run_append(codes, scales, rows, slots, block, head_major, fused))
    # the next tokens of the same blocks: scales grow or stay
    later = [s + 1 if 0 <= s < pages * page and (s + 1) % block else -1 for s in slots]
    keep = [i for i, s in enumerate(later) if s not in slots or s < 0]
    rows = [bf16_rows(rng, len(keep), H, d) for _ in range(2)]
    run_append(codes, scales, rows, np.array(later)[keep], block, head_major, fused)


@pytest.mark.parametrize("T", [64, 700, 3000, 9001])
def test_append_windows(T):
    """Enough rows for every window that a block of threads looks through; single tokens and a prompt."""
    rng = np.random.default_rng(T)
    H, d, page, block = 8, 64, 32, 16
    pages = T + 3
    codes, scales = pool(rng, pages, page, H, d, block)
    singles = rng.permutation(pages)[:T] * page + rng.integers(0, page, T)
    rows = [bf16_rows(rng, T, H, d) for _ in range(2)]
    run_append(codes, scales, rows, singles, block)
    run_append(codes, scales, rows, placed(rng, [(5, T)], page, pages), block)


@pytest.mark.parametrize("H,d,page,block,head_major", [(8, 64, 64, 64, False), (5, 64, 256, 32, True), (3, 128, 64, 32, False), (4, 128, 256, 256, False),
                                                       (1, 64, 4096, 256, False), (7, 128, 128, 128, True)])
def test_append_of_many_rows_in_long_blocks(H, d, page, block, head_major):
    """More than 1024 rows: prompts that begin and end anywhere, with blocks of one token and whole ones, single tokens, and rows of
    no slot between and behind them, in runs that begin and end inside every window of rows."""
    rng = np.random.default_rng(H + d + block)
    lens = [(int(rng.integers(0, page)), int(rng.choice([1, 1, 1, 2, 7, 8, 9, 63, 64, 65, block - 1, block, block + 1]))) for _ in range(90)]
    lens += [(block - 1, 700), (0, 2 * block), (5, 3 * block + 1)]
    lens = [lens[i] for i in rng.permutation(len(lens))]
    pages = sum((o + n - 1) // page + 1 for o, n in lens) + 2
    parts, at = [], 0
    for (_, n), gap in zip(lens, rng.integers(0, 4, len(lens))):
        parts += [(at, n), (None, int(gap) * (gap > 1))]
        at += n
    flat = placed(rng, lens, page, pages)
    slots = np.concatenate([flat[a:a + n] if a is not None else np.full(n, -1) for a, n in parts])
    assert len(slots) > 1024 and (slots < 0).any()
    codes, scales = pool(rng, pages, page, H, d, block)
    rows = [bf16_rows(rng, len(slots), H, d) for _ in range(2)]
    run_append(codes, scales, rows, slots, block, head_major, fused=H % 2 == 1)


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_many_single_tokens_in_long_blocks(d):
    """A step of 1500 requests with a token each, anywhere in blocks of 64."""
    rng = np.random.default_rng(d)
    T, H, page, block = 1500, 4, 64, 64
    codes, scales = pool(rng, T + 5, page, H, d, block)
    rows = [bf16_rows(rng, T, H, d) for _ in range(2)]
    run_append(codes, scales, rows, rng.permutation(T + 5)[:T] * page + rng.integers(0, page, T), block)


def test_append_of_extreme_values():
    """Zeros, the smallest and the largest bf16, infinities and NaN; magnitudes at and next to 448 * 2^n."""
    d = 64
    x = torch.zeros(12, 1, d)
    x[1, 0, 3] = 2.0 ** -133
    x[2, 0, :] = torch.finfo(torch.bfloat16).max
    x[3, 0, 5], x[3, 0, 6] = float("inf"), -float("inf")
    x[4, 0, 7], x[4, 0, 8] = float("nan"), 3.0
    x[5, 0, :] = float("nan")
    x[6, 0, 0], x[7, 0, 0], x[8, 0, 0] = 448.0, 450.0, 446.0
    x[9, 0, 0], x[10, 0, 0], x[11, 0, 0] = 448.0 * 2.0 ** -117, 2.0 ** -126, -0.0
    x = x.to(torch.bfloat16)
    for offset in (0, 5):  # blocks begun by these rows, and blocks with tokens of the smallest scale
        codes = [np.full((12, 16, 1, d), 0x38, np.uint8) for _ in range(2)]
        scales = [np.full((12, 1, 1), 10 if offset else 200, np.uint8) for _ in range(2)]
        run_append(codes, scales, [x, x], np.arange(12) * 16 + offset, 16)


def test_growing_scales_round_older_tokens_again():
    """Every code, at shifts up to past its last bit: the same as rounding the value at the new scale."""
    for shift in (1, 2, 5, 9, 16, 25, 60, 200):
        codes = [np.arange(256, dtype=np.uint8).reshape(1, 16, 1, 16).repeat(4, 3) for _ in range(2)]
        scales = [np.full((1, 1, 1), 30, np.uint8) for _ in range(2)]
        x = torch.zeros(1, 1, 64)
        x[0, 0, 0] = 448.0 * 2.0 ** (30 + shift - 127)
        run_append(codes, scales, [x.to(torch.bfloat16)] * 2, np.array([3]), 16)


def test_append_offsets_past_32_bits():
    pages, page, H, d = 2200, 4096, 4, 128
    kc, vc = (torch.zeros((pages, page, H, d), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    assert kc.numel() > 2 ** 32
    ks, vs = (torch.full((pages, 256, H), 127, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))
    k, v = torch.randn(2, 3, H, d, device="cuda").to(torch.bfloat16)
    slots = [pages * page - 1, pages * page - 4096, 17]
    U.kv_append(k, v, U.PagedCache8(kc, vc, ks, vs), i32(slots))
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        c, s = c.view(torch.uint8).view(-1, H, d), s.view(torch.uint8).view(-1, H)
        for t, at in enumerate(slots):
            fresh = at % 16 == 0
            wc, ws = cache8.append(np.zeros((1, 16, H, d), np.uint8), np.full((1, 1, H), 127, np.uint8), x[t:t + 1].double().cpu().numpy(),
                                   np.array([at % 16]), 16)
            assert np.array_equal(raw(c[at]), wc[0, at % 16]) and np.array_equal(raw(s[at // 16]), ws[0, 0]), fresh
        assert int(torch.count_nonzero((c & 127).amax((1, 2)))) == 3


# ------------------------------------------------------------------ attention

class Step8(Step):
    """A step whose pools are rounded to 8 bits, block by block, after the blocks have been given sizes of their own: 2^k within
    `k_spread` for keys (they move scores), v_spread for values. self.k and self.v then hold what codes and scales stand for."""

    def __init__(self, reqs, H, Hkv, d, page, block=16, k_spread=1, v_spread=6, head_major=False, seed=0, **kw):
        super().__init__(reqs, H, Hkv, d, page, head_major=head_major, seed=seed, **kw)
        rng = np.random.default_rng(seed + 1)
        pages = self.k.shape[0]
        parts = []
        for name, spread in (("k", k_spread), ("v", v_spread)):
            x = getattr(self, name).float().cpu().numpy().astype(np.float64).reshape(pages, page // block, block, Hkv, d)
            x = x * 2.0 ** rng.integers(-spread, spread + 1, (pages, page // block, 1, Hkv, 1))
            top = np.nanmax(np.where(np.isnan(x), 0, np.abs(x)), axis=(2, 4))
            n = np.vectorize(cache8.need)(top)
            scale = np.where(top > 0, n + 127, rng.integers(10, 247, n.shape)).astype(np.uint8)
            codes = cache8.encode(x * 2.0 ** (127.0 - scale[:, :, None, :, None])).reshape(pages, page, Hkv, d)
            parts.append((codes, scale))
        self.block, self.parts = block, parts
        self.put(head_major)

    def put(self, head_major=False):
        (kc, ks), (vc, vs) = self.parts
        self.cache = U.PagedCache8(device(kc, E4M3, head_major), device(vc, E4M3, head_major), device(ks, E8M0), device(vs, E8M0))
        self.k, self.v = (torch.tensor(cache8.values(c, s, self.block)) for c, s in self.parts)


@pytest.mark.parametrize("H,Hkv,d,page,block,head_major", [(8, 2, 128, 16, 16, False), (4, 4, 64, 32, 16, True), (16, 1, 128, 64, 64, False),
                                                           (6, 2, 64, 128, 32, False), (5, 1, 128, 256, 128, True), (1, 1, 64, 16, 16, False)])
def test_decode_lengths(H, Hkv, d, page, block, head_major):
    s = Step8([(1, c) for c in KV], H, Hkv, d, page, block, seed=H + d, head_major=head_major, pad=3, q_extra=2)
    s.check(max_q=1)
    s.check(max_q=0)
    healthy()


@pytest.mark.parametrize("mask,window", [("causal", 0), ("none", 0), ("causal", 1), ("causal", 37), ("causal", 128), ("causal", 700)])
@pytest.mark.parametrize("d,G,n,page,block", [(128, 4, 1, 16, 16), (64, 4, 4, 16, 16), (128, 5, 3, 64, 32), (64, 1, 1, 128, 128),
                                              (128, 1, 16, 32, 16), (64, 5, 2, 512, 256)])
def test_masks_in_the_decode_kernel(mask, window, d, G, n, page, block):
    old = (0, 3, 15, 16, 62, 63, 64, 127, 128, 129, 255, 256, 800)   # around the ends of pages and tiles, past each window
    reqs = [(0 if i == 4 else max(1, n - i % 2), c) for i, c in enumerate(old)]
    s = Step8(reqs, 2 * G, 2, d, page, block, seed=window + n, pad=3)
    s.check(max_q=n, mask=mask, window=window)
    if window > 0:
        for i, (_, c) in enumerate(reqs):
            s.table[i, :max(0, c - window + 1) // page] = -1
        s.check(max_q=n, mask=mask, window=window)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 16, 17, 31, 33, 64, 65, 130])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (3, 3, 64), (7, 1, 128)])
def test_few_and_chunk_lengths(n, H, Hkv, d):
    s = Step8([(n, c) for c in (0, 1, 30, 127, 128, 200)], H, Hkv, d, 16, seed=n, pad=1)
    s.check(max_q=n)


@pytest.mark.parametrize("n", [1, 5, 100])
def test_long_contexts_split_over_the_grid(n):
    Step8([(n, 5000), (1, 3)], 8, 1, 128, 64, 64, seed=n).check(max_q=n)


def test_rows_that_see_nothing_and_missing_pages():
    for max_q, H, Hkv in ((1, 4, 2), (20, 4, 2), (0, 8, 1)):
        n = max_q or 40
        s = Step8([(n, 5), (n, 0), (n, 200), (n, 300), (n, 90)], H, Hkv, 128, 16, seed=n)
        s.kv = [max(0, n // 2), 0, 200 + n, 300 + n, 90 + n]
        s.table[3, 0], s.table[3, 5], s.table[3, -1] = -1, s.cache.num_pages, 10 ** 9
        s.table[4, :] = -1
        s.check(max_q=max_q)
        assert np.isneginf(s.oracle()["lse"]).any()


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_very_different_scales(n, d):
    """Value scales 2^30 apart from block to block, and blocks whose size the softmax all but hides: each row is held to its own
    terms."""
    s = Step8([(n, 700), (n, 90)], 8, 2, d, 32, 16, v_spread=30, seed=n + d)
    s.check(max_q=n)
    s = Step8([(n, 700), (n, 90)], 8, 2, d, 32, 16, v_spread=30, k_spread=3, q_scale=4.0, seed=n + d)
    s.check(max_q=n)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("shift", [-100, -30, 0, 60])
def test_scales_at_the_ends(n, shift):
    """Queries 2^-shift, keys 2^shift, values at the smallest scales or near the largest."""
    s = Step8([(n, 300)], 4, 2, 64, 16, seed=n)
    (kc, ks), (vc, vs) = s.parts
    ks = (ks.astype(int) + shift).clip(10, 246).astype(np.uint8)
    vs = np.where(np.arange(vs.size).reshape(vs.shape) % 2 == 0, 10 if shift < 0 else 235, vs).astype(np.uint8)
    s.parts = [(kc, ks), (vc, vs)]
    s.q = (s.q.double() * 2.0 ** -shift).to(torch.bfloat16)
    s.put()
    s.check(max_q=n)


@pytest.mark.parametrize("n", [1, 40])
def test_zero_keys_at_the_largest_scale(n):
    """Queries of 2^100 and more against keys of zero: every score is zero, whatever the factors in front of it."""
    s = Step8([(n, 300)], 4, 2, 64, 16, seed=n)
    (kc, ks), v = s.parts
    s.parts = [(np.zeros_like(kc), np.full_like(ks, 246)), v]
    s.q = (s.q.double() * 2.0 ** 100).to(torch.bfloat16)
    s.put()
    s.check(max_q=n)


@pytest.mark.parametrize("d,shift", [(64, 6), (64, 20), (128, 30)])
def test_heaviest_key_of_zeros_under_a_large_scale(d, shift):
    """Decoding: the key with by far the largest weight has values of zero, in a block whose scale, 2^shift, its neighbours
    have set. A key's weight times scale is held to 2^-11 of itself, and no finer than 2^-32 of the row's largest such product
    (2^-25, half of fp16's smallest step, against 2^7); its codes go to 448. A score's d fp32 additions, 2^-24 of its magnitudes
    each, count in the weight and in the sum."""
    s = Step8([(1, 300)], 2, 1, d, 16, seed=shift, k_spread=0, v_spread=0)
    t = 37
    page = int(s.table[0, t // 16])
    (kc, ks), (vc, vs) = s.parts
    q = s.q[0].double().cpu().numpy()
    kc[page, t % 16, 0] = np.where(q.sum(0) < 0, 0xfe, 0x7e)  # the largest code, towards the queries
    vc[page, t % 16, 0] = 0
    vs[page, 0, 0] += shift
    s.put()
    o, lse = s.run(1)
    ref = s.oracle()
    k, v = (x.double().numpy()[s.table[0, :-1]].reshape(-1, 1, d)[:s.kv[0], 0] for x in (s.k, s.v))
    scores = q @ k.T / np.sqrt(d)
    w = np.exp(scores - scores.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    assert (w.argmax(-1) == t).all()
    by = np.repeat(2.0 ** (vs[s.table[0, :-1], 0, 0].astype(float) - 127), 16)[:s.kv[0]]
    floor = 2.0 ** -32 * (w * by).max(-1, keepdims=True) * 448 * s.kv[0]
    fp32 = 2 * 2.0 ** -24 * (d + 8) * (np.abs(q) @ np.abs(k).T).max() / np.sqrt(d)
    off = np.abs(o[0].double().cpu().numpy() - ref["o"][0])
    assert (off <= 2.0 ** -8 * np.abs(ref["o"][0]) + (2.0 ** -11 + fp32) * (w @ np.abs(v)) + floor).all()
    assert np.isfinite(lse.cpu().numpy()).all()


def test_queries_of_very_different_elements():
    """Elements of a row down to 2^-24 of its largest, and rows of zeros."""
    s = Step8([(1, 200), (3, 90), (40, 100)], 8, 2, 128, 16, seed=5)
    x = s.q.float() * torch.exp2(torch.randint(-24, 1, s.q.shape, device="cuda").float())
    x[::5] = 0
    s.q = x.to(torch.bfloat16)
    s.check(max_q=40)


@pytest.mark.parametrize("mask,window", [("causal", 0), ("none", 0), ("causal", 1), ("causal", 37), ("causal", 128), ("causal", 2 ** 31 - 1)])
@pytest.mark.parametrize("H,Hkv,d,page,block", [(8, 2, 128, 32, 32), (2, 2, 64, 16, 16), (8, 2, 128, 256, 64)])
def test_masks_in_a_mixed_batch(mask, window, H, Hkv, d, page, block):
    reqs = [(1, 500), (0, 40), (140, 0), (1, 0), (0, 0), (70, 333), (3, 129), (1, 127), (33, 700)]
    Step8(reqs, H, Hkv, d, page, block, seed=window % 1000, pad=5).check(max_q=140, mask=mask, window=window)


@pytest.mark.parametrize("H,d,n", [(32, 128, 6), (32, 64, 6), (16, 128, 70), (16, 64, 70)])
def test_many_key_tiles_in_a_row(H, d, n):
    """Units of one and of two row tiles with twenty and more key tiles to a CTA, in batches that fill the grid."""
    rng = np.random.default_rng(H + d + n)
    reqs = [(n, int(c)) for c in rng.integers(1800, 3000, 20 if n < 10 else 3)]
    Step8(reqs, H, 8, d, 64, 32, seed=d + n).check(max_q=n)


@pytest.mark.parametrize("d", [64, 128])
def test_units_of_one_and_of_two_tiles_in_turn(d):
    rng = np.random.default_rng(d)
    reqs = [(int(rng.integers(5, 33)) if i % 3 else int(rng.integers(40, 65)), int(rng.integers(0, 900))) for i in range(260)]
    Step8(reqs, 8, 2, d, 32, seed=d).check()


@pytest.mark.parametrize("H,n", [(17, 20), (100, 3), (128, 5)])
def test_more_heads_to_a_key_than_a_decode_tile(H, n):
    Step8([(n, 140), (1, 600)], H, 1, 64, 32, seed=H, pad=1).check(max_q=n)


@pytest.mark.parametrize("B,n,max_q", [(257, 1, 1), (257, 23, 23), (700, 1, 0)])
def test_many_requests(B, n, max_q):
    rng = np.random.default_rng(B + n)
    Step8([(0 if i % 9 == 4 else n, int(c)) for i, c in enumerate(rng.integers(0, 60, B))], 2, 1, 64, 16, seed=B, pad=2).check(max_q=max_q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask,window", [("causal", 0), ("causal", 90), ("none", 0)])
def test_mixed_batch_that_takes_both_kernels(d, mask, window):
    rng = np.random.default_rng(window + d)
    reqs = [(0 if i % 13 == 6 else int(rng.integers(9, 70)) if i % 10 == 3 else 1, int(rng.integers(0, 300))) for i in range(60)]
    s = Step8(reqs, 16, 8, d, 16, seed=window, pad=4)
    s.check(max_q=70, mask=mask, window=window)
    s.check(max_q=0, mask=mask, window=window)


@pytest.mark.parametrize("n", [40, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_equal_the_bf16_cache_of_the_same_values(n, d):
    """Codes times scales are exact in bf16, and the chunk kernels multiply them in the same order: the same bits."""
    s = Step8([(n, 700), (n, 3), (n + 1, 90)], 8, 2, d, 32, 16, seed=n)
    k, v = (torch.nan_to_num(x).to(torch.bfloat16).cuda() for x in (s.k, s.v))
    a = s.run(n + 1)
    s.cache = U.PagedCache(k, v)
    b = s.run(n + 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("reqs,H,Hkv,d", [([(2048, 6144)], 32, 8, 128), ([(2048, 6144)], 32, 8, 64), ([(300, 9000), (40, 4000), (700, 2500)], 8, 4, 128)])
def test_long_chunks_equal_the_bf16_cache_many_times(reqs, H, Hkv, d):
    """Shares of many key tiles, call after call, every other one with nothing in the L2, so that copies take different times: always
    the bf16 cache's bits."""
    s = Step8(reqs, H, Hkv, d, 64, 32, seed=d)
    n = max(r[0] for r in reqs)
    args = (i32(s.cu), i32(s.kv), i32(s.table), n)
    k, v = (torch.nan_to_num(x).to(torch.bfloat16).cuda() for x in (s.k, s.v))
    want = U.paged_attn_fwd(s.q, U.PagedCache(k, v), *args)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(60):
        if i % 2:
            flush.fill_(i)
        o, lse = U.paged_attn_fwd(s.q, s.cache, *args)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), i
    healthy()


@pytest.mark.parametrize("n", [1, 50])
def test_same_bits_every_time(n):
    s = Step8([(n, c) for c in (3000, 10, 700)], 8, 2, 128, 16, seed=1)
    a, b = s.run(n), s.run(n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 40])
def test_nan_keys_and_values(n):
    """NaN among a request's keys makes rows that see it NaN in o and lse; among its values, in those elements of o."""
    s = Step8([(n, 60), (n, 300)], 4, 2, 64, 16, seed=n)
    (kc, ks), (vc, vs) = s.parts
    t = 30  # a cached token of either request, in key/value head 1
    page0, page1 = int(s.table[0, t // 16]), int(s.table[1, t // 16])
    kc[page0, t % 16, 1, 9] = 0x7f
    vc[page1, t % 16, 1, 5] = 0xff
    s.put()
    o, lse = s.run(n)
    healthy()
    assert torch.isnan(o[:n, 2:]).all() and torch.isnan(lse[2:, :n]).all()
    assert torch.isfinite(o[:n, :2]).all() and torch.isfinite(lse[:2]).all() and torch.isfinite(lse[:, n:]).all()
    bad = torch.isnan(o[n:])
    assert bad[:, 2:, 5].all() and int(bad.sum()) == 2 * n


def test_two_graphs_share_a_workspace():
    a, b = Step8([(1, 3000), (1, 40)], 8, 2, 128, 16, seed=41), Step8([(150, 700), (1, 900), (0, 5)], 8, 2, 128, 16, seed=42)
    ws = U.paged_attn_workspace(b.q, b.cache, 0)
    calls = []
    for x, max_q in ((a, 1), (b, 150)):
        args = (x.q, x.cache, i32(x.cu), i32(x.kv), i32(x.table), max_q)
        want = [t.clone() for t in U.paged_attn_fwd(*args)]
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            U.paged_attn_fwd(*args, o=o, lse=lse, workspace=ws)
        calls.append((graph, o, lse, want, args))
    for i in (0, 1, 0, 0, 1, 1, 0):
        graph, o, lse, want, _ = calls[i]
        o.fill_(0)
        graph.replay()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    healthy()


def test_another_stream_and_two_at_once():
    a, b = Step8([(1, 3000)] * 4, 8, 2, 128, 16, seed=11), Step8([(70, 900)] * 3, 8, 2, 128, 16, seed=12)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    args = [(x.q, x.cache, i32(x.cu), i32(x.kv), i32(x.table), x.new[0]) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [U.paged_attn_fwd(*x, stream=st) for x, st in zip(args, (sa, sb))]
    torch.cuda.synchronize()
    for x, (o, lse) in zip((a, b), got):
        hold(o, lse, x.oracle(), 128)


# ------------------------------------------------------------------ as they are used

def test_serving_steps_with_norms_and_rotation():
    """plan -> norm and rotation -> append -> attention, in chunks and single tokens, against the oracles' chain on the codes that
    the cache holds, the appended codes against the oracle's from the rotated rows."""
    H, Hkv, d, page, block, B = 8, 2, 128, 32, 16, 3
    rng = np.random.default_rng(7)
    num, width = 60, 16
    cache = U.PagedCache8.empty(num, page, Hkv, d, block)
    cache.k.view(torch.uint8).fill_(0x7f)
    cache.v.view(torch.uint8).fill_(0x7f)
    rope = U.Rope(d)
    w = [torch.tensor(1 + 0.1 * rng.standard_normal(d), dtype=torch.float32, device="cuda").to(torch.bfloat16) for _ in range(2)]
    table = i32(np.full((B, width), -1))
    free, n_free, cached = i32(rng.permutation(num)), i32([num]), i32([0] * B)
    codes = [raw(cache.k), raw(cache.v)]
    scales = [raw(cache.k_scale), raw(cache.v_scale)]
    for step, new in enumerate(([40, 0, 7], [1, 100, 1], [1, 1, 1], [1, 1, 0], [30, 1, 1], [1, 1, 1])):
        T = sum(new) + 2
        rows = bf16_rows(rng, T, H + 2 * Hkv, d, spread=1.0).cuda()
        q, k, v = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
        cu, kv, slots, info = U.page_plan(cached, i32(new), free, n_free, table, page, num, T)
        U.qk_rope_rows(q, k, rope, cu_q=cu, kv_lens=kv, w_q=w[0], w_k=w[1], q_out=q, k_out=k)
        U.kv_append(k, v, cache, slots)
        o, lse = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, T), 7.0, device="cuda")
        U.paged_attn_fwd(q, cache, cu, kv, table, max(new), o=o, lse=lse)
        cached, n_free = kv, n_free - info[1:2]
        for i, (x, c, s) in enumerate(((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale))):
            codes[i], scales[i] = cache8.append(codes[i], scales[i], x.double().cpu().numpy(), slots.cpu().numpy(), block)
            assert np.array_equal(raw(c), codes[i]) and np.array_equal(raw(s), scales[i]), step
        pools = [cache8.values(c, s, block) for c, s in zip(codes, scales)]
        ref = paged.paged_attention(q.double().cpu().numpy(), *pools, cu.cpu().numpy(), kv.cpu().numpy(), table.cpu().numpy(), True)
        hold(o, lse, ref, d)


def test_one_step_captured_and_replayed_while_requests_grow():
    """plan -> norm and rotation in place -> append -> attention in one graph, four steps replayed with nothing but lengths, rows
    and the free list changed, each equal to the same calls made one by one on a copy of the state."""
    H, Hkv, d, page, block, B, T = 8, 2, 64, 32, 16, 4, 6
    rng = np.random.default_rng(3)
    num, width, lens0 = 30, 8, [15, 31, 0, 40]
    rope = U.Rope(d, rot=32, interleaved=True, scaling="linear", factor=2.0)
    w = [torch.ones(d, device="cuda") for _ in range(2)]
    table = np.full((B, width), -1)
    order, at = rng.permutation(num), 0
    for i, c in enumerate(lens0):
        n = -(-c // page)
        table[i, :n] = order[at:at + n]
        at += n

    def state():
        cache = U.PagedCache8.empty(num, page, Hkv, d, block)
        for t in (cache.k, cache.v):
            t.view(torch.uint8).zero_()
        s = dict(cache=cache, table=i32(table), cached=i32(lens0), free=i32(order[at:]), n_free=i32([num - at]),
                 rows=torch.zeros(T, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda"))
        hist = torch.randn(2, sum(lens0), Hkv, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
        slots = [table[i, t // page] * page + t % page for i, c in enumerate(lens0) for t in range(c)]
        U.kv_append(hist[0], hist[1], cache, i32(slots))
        return s

    def step(s):
        q, k, v = s["rows"][:, :H], s["rows"][:, H:H + Hkv], s["rows"][:, H + Hkv:]
        cu, kv, slots, info = U.page_plan(s["cached"], s["new"], s["free"], s["n_free"], s["table"], page, num, T)
        U.qk_rope_rows(q, k, rope, cu_q=cu, kv_lens=kv, w_q=w[0], w_k=w[1], q_out=q, k_out=k)
        U.kv_append(k, v, s["cache"], slots)
        o, lse = U.paged_attn_fwd(q, s["cache"], cu, kv, s["table"], 2, workspace=s["ws"])
        return kv, info, o, lse
    a, b = state(), state()
    for s in (a, b):
        s["new"] = i32([1] * B)
        s["ws"] = U.paged_attn_workspace(s["rows"][:, :H], s["cache"], 2)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kv, info, o, lse = step(a)
    for new in ([1, 1, 1, 1], [2, 1, 0, 1], [1, 1, 2, 1], [0, 1, 1, 2]):
        x = bf16_rows(rng, T, H + 2 * Hkv, d).cuda()
        for s in (a, b):
            s["rows"].copy_(x)
            s["new"].copy_(i32(new))
        graph.replay()
        want = step(b)
        n = sum(new)
        assert torch.equal(kv, want[0]) and torch.equal(info, want[1])
        assert torch.equal(o[:n], want[2][:n]) and torch.equal(lse[:, :n], want[3][:, :n]) and torch.isfinite(o[:n]).all()
        for p, q in zip((a["cache"].k, a["cache"].v, a["cache"].k_scale, a["cache"].v_scale),
                        (b["cache"].k, b["cache"].v, b["cache"].k_scale, b["cache"].v_scale)):
            assert np.array_equal(raw(p), raw(q))
        for s in (a, b):
            s["cached"].copy_(kv)
            s["n_free"].sub_(info[1:2])
    healthy()
