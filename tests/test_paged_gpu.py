"""GPU parity of the paged-cache calls against the fp64 oracle, at the sizes and masks where they can go
wrong. Whole numbers and moved bits must be equal. Attention is held to bounds counted from its
roundings, element by element:

- o: every softmax weight is rounded to bf16 once (relative 2^-8 at most), which moves o by at most
  2^-8 sum(w |v|); o is rounded once, 2^-8 |o|; the fp32 scores, exponentials and sums stay below
  2^-13 sum(w |v|) for the sizes used here.
- lse: a score is an fp32 sum of d exact products, off by at most d 2^-24 sum |q||k|, and the scale,
  the base change and the maximum round it a few times more; n additions of the sum are off by at
  most n 2^-24.
"""

import numpy as np
import pytest
import torch

import oracle.paged as paged
import ulysses_sequence_gb300 as U
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def healthy():
    st, word = U.device_status()
    assert st == U.OK, hex(word)


# ------------------------------------------------------------------ page_plan

def run_plan(cached, new, free, n_free, table, page, num_pages, T):
    t = i32(table)
    got = U.page_plan(i32(cached), i32(new), i32(free).reshape(-1), i32([n_free]), t, page, num_pages, T)
    want = paged.page_plan(cached, new, free, n_free, table, page, num_pages, T)
    for name, g, w in zip(("cu_q", "kv_lens", "slot_map", "info", "table"), (*got, t), want):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("B,page,hi,old,slack", [(1, 16, 1, 0, 0), (1, 16, 1, 16, 0), (7, 16, 40, 100, 3), (64, 64, 1, 5000, 9),
                                                 (300, 32, 200, 900, 0), (2500, 16, 30, 300, 100), (8192, 128, 3, 1000, 1)])
def test_plan_matches_oracle(B, page, hi, old, slack):
    rng = np.random.default_rng(B + page)
    cached, new = rng.integers(0, old + 1, B), rng.integers(0, hi + 1, B)
    width = -(-(old + hi) // page) + 1
    num = int(B * width) + 5
    order = rng.permutation(num)
    table = np.full((B, width), -1)
    at = 0
    for i in range(B):
        n = -(-cached[i] // page)
        table[i, :n] = order[at:at + n]
        at += n
    run_plan(cached, new, order[at:], len(order) - at, table, page, num, int(new.sum()) + slack)


@pytest.mark.parametrize("n_free,T", [(-3, 90), (0, 90), (4, 90), (9, 90), (100, 90), (9, 0), (9, 1), (9, 41), (9, 70)])
def test_plan_short_lists_tables_and_rows(n_free, T):
    """Too few pages, too narrow a table, too few rows, bad lengths and bad page ids: the same in the oracle."""
    cached, new = [5, -4, 31, 64, 0, 200, 16], [12, 20, -1, 3, 17, 9, 16]
    table = np.full((7, 4), -1)
    table[0, 0], table[2, :2], table[3, :4], table[5, :4], table[6, 0] = 12, [99, 3], [1, 2, 4, 5], [6, 7, 8, -7], 9
    run_plan(cached, new, [0, 10, 11, 13, 1000, 14, 15, -2, 16, 17], n_free, table, 16, 20, T)


def test_plan_empty_batches():
    run_plan(np.zeros(0, int), np.zeros(0, int), [1, 2], 2, np.zeros((0, 3), int), 16, 4, 5)
    run_plan([3, 4], [0, 0], [1, 2], 2, np.array([[0, -1], [3, -1]]), 16, 4, 0)
    run_plan([0, 0], [3, 4], np.zeros(0, int), 0, np.zeros((2, 0), int), 16, 4, 9)


def test_plan_strided_table_and_large_lengths():
    """A table that is a slice of a wider one; lengths near 2^31 saturate."""
    wide = torch.full((3, 12), 7, dtype=torch.int32, device="cuda")
    table = wide[:, 2:6]
    table.copy_(i32([[1, -1, -1, -1], [-1] * 4, [2, 3, -1, -1]]))
    big = 2 ** 31 - 1
    got = U.page_plan(i32([16, big, 20]), i32([5, big, big]), i32([9, 8, 4]), i32([3]), table, 16, 10, 50)
    want = paged.page_plan([16, big, 20], [5, big, big], [9, 8, 4], 3, [[1, -1, -1, -1], [-1] * 4, [2, 3, -1, -1]], 16, 10, 50)
    for g, w in zip((*got, table), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert torch.all(wide[:, :2] == 7) and torch.all(wide[:, 6:] == 7)


@pytest.mark.parametrize("cached", [2 ** 31 - 4096, 2 ** 31 - 4106, 2 ** 31 - 9000])
def test_plan_up_to_the_last_token_of_31_bits(cached):
    """The largest table and T that are taken together: max_pages * page_size + T = 2^31 - 1."""
    page, width = 4096, 2 ** 19 - 1
    table = np.full((1, width), -1)
    table[0, : -(-cached // page)] = 5
    run_plan([cached], [4095], [9, 8, 7], 3, table, page, 10, 4095)


# ------------------------------------------------------------------ kv_append

@pytest.mark.parametrize("T,H,d,page,head_major,fused", [(1, 1, 8, 16, False, False), (5, 3, 64, 16, True, True),
                                                         (257, 8, 128, 16, False, False), (1000, 5, 128, 256, True, False),
                                                         (333, 2, 72, 32, False, True), (64, 1, 128, 4096, True, True)])
def test_append_moves_bits(T, H, d, page, head_major, fused):
    pages = T // page + 4
    g = torch.Generator(device="cuda").manual_seed(T)

    def bits(*shape):  # every 16-bit pattern, NaN payloads included
        return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16).view(torch.bfloat16)
    shape = (pages, H, page, d) if head_major else (pages, page, H, d)
    kc, vc = (bits(*shape).permute(0, 2, 1, 3) if head_major else bits(*shape) for _ in range(2))
    if fused:
        rows = bits(T, 3 * H, d)
        k, v = rows[:, H:2 * H], rows[:, 2 * H:]
    else:
        k, v = bits(T, H, d), bits(T, H, d)
    slots = np.random.default_rng(T).permutation(pages * page)[:T]
    slots[::7] = -1
    slots[1::50] = pages * page            # one past the pool
    slots[2::90] = 2 ** 31 - 1
    slots[3::70] = -2 ** 31
    as16 = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
    want = [paged.kv_append(as16(c), as16(x), slots) for c, x in ((kc, k), (vc, v))]
    U.kv_append(k, v, U.PagedCache(kc, vc), i32(slots))
    assert np.array_equal(as16(kc), want[0]) and np.array_equal(as16(vc), want[1])


def test_append_offsets_past_32_bits():
    """The last page of a pool whose values lie more than 2^32 bytes and 2^31 elements in."""
    pages, page, H, d = 1050, 4096, 4, 128
    kc, vc = (torch.zeros((pages, page, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 31
    k, v = torch.randn(2, 3, H, d, device="cuda").to(torch.bfloat16)
    slots = [pages * page - 1, pages * page - 4097, 17]
    U.kv_append(k, v, U.PagedCache(kc, vc), i32(slots))
    for t, s in enumerate(slots):
        assert torch.equal(kc.view(-1, H, d)[s], k[t]) and torch.equal(vc.view(-1, H, d)[s], v[t])
    assert int(torch.count_nonzero(kc.view(-1, H, d).abs().amax((1, 2)))) == 3


# ------------------------------------------------------------------ paged attention

class Step:
    """Requests (new tokens, cached tokens) with random pages; all that no request owns is NaN."""

    def __init__(self, reqs, H, Hkv, d, page, seed=0, head_major=False, pad=0, q_extra=0, spare=3, width_extra=1, q_scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.old = [r[0] for r in reqs], [r[1] for r in reqs]
        kv = [n + c for n, c in reqs]
        held = [-(-x // page) for x in kv]
        pages, width = sum(held) + spare, max(held + [0]) + width_extra
        order = rng.permutation(pages)
        self.table = np.full((len(reqs), width), -1)
        shape = (pages, Hkv, page, d) if head_major else (pages, page, Hkv, d)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if head_major:
            self.k, self.v = self.k.permute(0, 2, 1, 3), self.v.permute(0, 2, 1, 3)
        at = 0
        for i, n in enumerate(held):
            ids = order[at:at + n]
            self.table[i, :n] = ids
            at += n
            for pool in (self.k, self.v):
                x = torch.full((n * page, Hkv, d), float("nan"), device="cuda")
                x[:kv[i]] = torch.randn((kv[i], Hkv, d), generator=g, device="cuda")
                pool[torch.tensor(ids, device="cuda", dtype=torch.long)] = x.view(n, page, Hkv, d).to(torch.bfloat16)
        self.tokens = sum(self.new)
        T = self.tokens + pad
        self.q = (torch.randn((T, H + q_extra, d), generator=g, device="cuda") * q_scale).to(torch.bfloat16)[:, :H]
        self.cu, self.kv = [0] + list(np.cumsum(self.new)), kv
        self.cache = U.PagedCache(self.k, self.v)

    def run(self, max_q=0, mask="causal", window=0, scale=0.0, **kw):
        T, H, d = self.q.shape
        o = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, T), 7.0, device="cuda")
        U.paged_attn_fwd(self.q, self.cache, i32(self.cu), i32(self.kv), i32(self.table).reshape(len(self.new), -1), max_q,
                         U.Mask.causal() if mask == "causal" else U.Mask.none(), window, scale, o=o, lse=lse, **kw)
        return o, lse

    def oracle(self, mask="causal", window=0, scale=0.0):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        return paged.paged_attention(f(self.q), f(self.k), f(self.v), self.cu, self.kv, self.table, mask == "causal", window, scale)

    def check(self, max_q=0, **kw):
        hold(*self.run(max_q, **kw), self.oracle(**kw), self.q.shape[2])


def hold(o, lse, ref, d):
    healthy()
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    own = ref["owned"]
    assert np.all(o[~own] == 7.0) and np.all(lse[:, ~own] == 7.0), "rows that no request owns were written"
    tol = 2.0 ** -8 * np.abs(ref["o"]) + (2.0 ** -8 + 2.0 ** -13) * ref["absv"] * (1 + 2.0 ** -8)
    bad = ~(np.abs(o - ref["o"]) <= tol)
    assert not np.any(bad[own]), ("o", np.argwhere(bad & own[:, None, None])[:5], np.nanmax(np.abs(o - ref["o"])[own]))
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse)[:, own], empty[:, own])
    some = ~empty & own[None]
    lse, ref = np.where(some, lse, 0.0), {**ref, "lse": np.where(some, ref["lse"], 0.0)}
    tol = 2.0 ** -24 * ((d + 8) * ref["sqk"] + ref["keys"] + 8) + 2.0 ** -22 * np.abs(ref["lse"])
    assert np.all(np.abs(lse - ref["lse"])[some] <= tol[some]), ("lse", np.max(np.abs(lse - ref["lse"])[some]))


KV = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 300, 1000]  # around pages and tiles


@pytest.mark.parametrize("H,Hkv,d,page,head_major", [(8, 2, 128, 16, False), (4, 4, 64, 32, True), (16, 1, 128, 64, False),
                                                     (6, 2, 64, 128, False), (5, 1, 128, 256, True), (1, 1, 64, 16, False),
                                                     (24, 1, 64, 16, False), (256, 2, 64, 64, False)])
def test_decode_lengths(H, Hkv, d, page, head_major):
    s = Step([(1, c) for c in KV], H, Hkv, d, page, seed=H + d, head_major=head_major, pad=3, q_extra=2)
    s.check(max_q=1)
    s.check(max_q=0)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 16, 17, 31, 33, 64, 65, 130])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (3, 3, 64), (7, 1, 128)])
def test_few_and_chunk_lengths(n, H, Hkv, d):
    s = Step([(n, c) for c in (0, 1, 30, 127, 128, 200)], H, Hkv, d, 16, seed=n, pad=1)
    s.check(max_q=n)


@pytest.mark.parametrize("mask,window", [("causal", 0), ("none", 0), ("causal", 1), ("causal", 37), ("causal", 128),
                                         ("causal", 10 ** 6), ("causal", 2 ** 31 - 1)])
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (2, 2, 64)])
def test_masks_in_a_mixed_batch(mask, window, H, Hkv, d):
    reqs = [(1, 500), (0, 40), (140, 0), (1, 0), (0, 0), (70, 333), (3, 129), (1, 127), (33, 700)]
    s = Step(reqs, H, Hkv, d, 32, seed=window % 1000, pad=5)
    s.check(max_q=140, mask=mask, window=window)


def test_a_single_tile_long_context_splits_over_the_grid():
    for n in (1, 5, 100):
        s = Step([(n, 5000), (1, 3)], 8, 1, 128, 64, seed=n)
        s.check(max_q=n)


@pytest.mark.parametrize("H,d,n", [(32, 128, 6), (32, 64, 6), (16, 128, 70), (16, 64, 70)])
def test_many_key_tiles_in_a_row(H, d, n):
    """Units of one and of two row tiles with twenty and more key tiles to a CTA, in batches that fill the grid."""
    rng = np.random.default_rng(H + d + n)
    reqs = [(n, int(c)) for c in rng.integers(1800, 3000, 20 if n < 10 else 3)]
    s = Step(reqs, H, 8, d, 64, seed=d + n)
    s.check(max_q=n)


@pytest.mark.parametrize("d", [64, 128])
def test_units_of_one_and_of_two_tiles_in_turn(d):
    """Every CTA walks units of one row tile among units of two, each of several key tiles."""
    rng = np.random.default_rng(d)
    reqs = [(int(rng.integers(5, 33)) if i % 3 else int(rng.integers(40, 65)), int(rng.integers(0, 900))) for i in range(260)]
    Step(reqs, 8, 2, d, 32, seed=d).check()


def test_rows_that_see_nothing():
    """Lengths below the number of new tokens: early rows have negative positions. Lengths of zero: no keys."""
    for max_q, H, Hkv in ((1, 4, 2), (20, 4, 2), (0, 8, 1)):
        n = max_q or 40
        s = Step([(n, 5), (n, 0), (n, 200)], H, Hkv, 128, 16, seed=n)
        s.kv = [max(0, n // 2), 0, 200 + n]
        s.check(max_q=max_q)
        ref = s.oracle()
        assert np.isneginf(ref["lse"]).any()


@pytest.mark.parametrize("max_q", [1, 9, 100])
def test_missing_pages_hold_no_keys(max_q):
    """Entries outside the pool, first, middle and last: their keys are left out; all of them gone: no key."""
    reqs = [(max_q, 300), (max_q, 64), (max_q, 500), (max_q, 90)]
    s = Step(reqs, 8, 2, 128, 16, seed=max_q)
    s.table[0, 0], s.table[0, 5], s.table[1, -1] = -1, s.cache.num_pages, 10 ** 9
    s.table[2, 3:21] = -2 ** 31
    s.table[3, :] = -1
    s.check(max_q=max_q)


def test_a_window_with_its_old_pages_given_back():
    s = Step([(1, 700), (1, 40), (20, 900)], 4, 2, 64, 16, seed=2)
    for i in range(3):
        s.table[i, :max(0, s.old[i] - 100 + 1) // 16] = -1
    s.check(max_q=20, window=100)


def test_damaged_row_starts_and_lengths_stay_in_bounds():
    """Decreasing and outside row starts own nothing or are cut at the tensor's rows; lengths past the table
    end there, negative ones count as 0."""
    s = Step([(2, 50), (3, 70), (1, 100), (4, 20)], 4, 2, 128, 16, seed=4)
    for x in (s.k, s.v):  # the length past the table makes the rest of its last page the request's
        x[torch.isnan(x)] = 0.5
    s.cu = [3, 1, 4, 60, 10 ** 9]   # nothing; rows 1 to 4; rows 4 to 10; nothing
    s.kv = [52, -5, 10 ** 6, 24]
    got = s.run(max_q=4)
    ref = s.oracle()
    hold(*got, ref, 128)


def test_larger_scores_scale_and_strided_queries():
    s = Step([(1, 400), (60, 100)], 8, 2, 128, 64, seed=9, q_extra=3, q_scale=4.0)
    s.check(max_q=60, scale=0.25)


def test_equal_keys_and_infinite_tails():
    """What lies behind a request's last key may be infinite, in K and in V."""
    s = Step([(1, 20), (40, 90)], 4, 4, 64, 64, seed=5)
    for x, sign in ((s.k, 1.0), (s.v, -1.0)):
        x[torch.isnan(x)] = sign * float("inf")
    s.check(max_q=40)


@pytest.mark.parametrize("n,max_q", [(1, 1), (50, 50)])
def test_same_bits_every_time_and_any_hint(n, max_q):
    s = Step([(n, c) for c in (3000, 10, 700)], 8, 2, 128, 16, seed=1)
    a = s.run(max_q)
    b = s.run(max_q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    hold(*s.run(1000), s.oracle(), 128)
    hold(*s.run(1), s.oracle(), 128)   # a bound that is too low costs time, not correctness


def test_offsets_past_32_bits():
    """A request whose pages lie at the end of a pool of more than 2^31 elements."""
    pages, page, H, d = 1050, 4096, 4, 128
    pool = [torch.zeros((pages, page, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = Step([(1, 4500), (90, 2000)], 8, 4, 128, page, seed=6)
    table = np.where(small.table >= 0, small.table + pages - small.cache.num_pages, -1)
    for x, y in zip(pool, (small.k, small.v)):
        x[pages - small.cache.num_pages:] = y
    o, lse = U.paged_attn_fwd(small.q, U.PagedCache(*pool), i32(small.cu), i32(small.kv), i32(table), 90)
    o2, lse2 = U.paged_attn_fwd(small.q, small.cache, i32(small.cu), i32(small.kv), i32(small.table), 90)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    hold(o, lse, small.oracle(), 128)


@pytest.mark.parametrize("B", [257, 700])
@pytest.mark.parametrize("n,max_q", [(1, 1), (1, 0), (23, 23)])
def test_many_requests(B, n, max_q):
    """Batches beyond what one warp looks through, some requests idle."""
    rng = np.random.default_rng(B + n)
    reqs = [(0 if i % 9 == 4 else n, int(c)) for i, c in enumerate(rng.integers(0, 60, B))]
    s = Step(reqs, 2, 1, 64, 16, seed=B, pad=2)
    s.check(max_q=max_q)


def _mixed_step(seed):
    """60 requests of 8 key/value heads: too many units for one kernel, chunks among decoding and idle requests."""
    rng = np.random.default_rng(seed)
    reqs = [(0 if i % 13 == 6 else int(rng.integers(9, 70)) if i % 10 == 3 else 1, int(rng.integers(0, 300))) for i in range(60)]
    return Step(reqs, 16, 8, 64, 16, seed=seed, pad=4)


@pytest.mark.parametrize("mask,window", [("causal", 0), ("causal", 90), ("none", 0)])
def test_mixed_batch_that_takes_both_kernels(mask, window):
    s = _mixed_step(window)
    s.check(max_q=70, mask=mask, window=window)
    s.check(max_q=0, mask=mask, window=window)


def test_both_kernels_follow_what_their_stream_wrote():
    """The chunk kernel starts beside the decode kernel: both see what was written right before the call, and both are
    done with it when what follows overwrites it."""
    a, b = _mixed_step(1), _mixed_step(2)
    want = [x.run(70) for x in (a, b)]
    slots = []
    for x in (a, b):
        slots.append([x.q.clone(), x.k.clone(), x.v.clone(), i32(x.cu), i32(x.kv), i32(x.table)])
    for i in range(10):
        x, keep, (o0, l0) = ((a, slots[0], want[0]), (b, slots[1], want[1]))[i & 1]
        q, k, v = (torch.full_like(t, float("nan")) for t in keep[:3])
        big = torch.empty(100 << 20, dtype=torch.uint8, device="cuda").fill_(i)
        for dst, src in zip((q, k, v), keep[:3]):
            dst.copy_(src)
        o, lse = torch.full_like(o0, 7.0), torch.full_like(l0, 7.0)
        U.paged_attn_fwd(q, U.PagedCache(k, v), *keep[3:], 70, o=o, lse=lse)
        for t in (q, k, v):
            t.fill_(float("nan"))
        assert torch.equal(o, o0) and torch.equal(lse, l0), i
        del big
    healthy()


def test_keys_and_values_interleaved_in_one_allocation():
    """Pages that hold their keys and then their values: equal strides, neither tensor contiguous."""
    s = Step([(1, 300), (40, 77)], 8, 2, 128, 32, seed=3)
    both = torch.empty((s.cache.num_pages, 2, 32, 2, 128), dtype=torch.bfloat16, device="cuda")
    both[:, 0], both[:, 1] = s.k, s.v
    s.cache = U.PagedCache(both[:, 0], both[:, 1])
    s.check(max_q=40)
    k, v = torch.randn(2, 5, 2, 128, device="cuda").to(torch.bfloat16)
    before = both.clone()
    U.kv_append(k, v, s.cache, i32([0, 33, -1, 64, 95]))
    for t, slot in enumerate([0, 33, -1, 64, 95]):
        if slot >= 0:
            before[slot // 32, 0, slot % 32], before[slot // 32, 1, slot % 32] = k[t], v[t]
    assert torch.equal(both.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("n", [1, 40])
def test_outputs_that_are_only_16_byte_aligned(n):
    s = Step([(n, 100), (n, 3)], 8, 2, 64, 16, seed=n)
    T, H, d = s.q.shape
    o = torch.zeros(T * H * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(T, H, d)
    lse = torch.zeros(T * H + 1, device="cuda")[1:].view(H, T)
    assert o.data_ptr() % 32 == 16
    U.paged_attn_fwd(s.q, s.cache, i32(s.cu), i32(s.kv), i32(s.table), n, o=o, lse=lse)
    hold(o, lse, s.oracle(), d)


def test_empty_calls():
    """No requests, no rows, a table without columns: nothing is written, or rows without keys."""
    s = Step([(2, 30)], 4, 2, 64, 16, seed=1)
    e = torch.empty((0,), dtype=torch.int32, device="cuda")
    o, lse = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 2), 7.0, device="cuda")
    U.paged_attn_fwd(s.q, s.cache, i32([0]), e, e.view(0, 3), 1, o=o, lse=lse)
    healthy()
    assert torch.all(o == 7) and torch.all(lse == 7)
    got = U.paged_attn_fwd(s.q[:0], s.cache, i32([0, 0]), i32([5]), i32([[0, 1]]), 1)
    assert got[0].shape == (0, 4, 64) and got[1].shape == (4, 0)
    U.kv_append(s.q[:0, :2], s.q[:0, :2], s.cache, e)
    for max_q in (2, 20):
        U.paged_attn_fwd(s.q, s.cache, i32([0, 2]), i32([32]), e.view(1, 0), max_q, o=o, lse=lse)
        healthy()
        assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
        o.fill_(7.0)


def test_more_heads_to_a_key_than_a_decode_tile():
    """Groups of 17, 100 and 128 query heads: chunk units of a few tokens, of one token."""
    for H, n in ((17, 20), (100, 3), (128, 5)):
        s = Step([(n, 140), (1, 600)], H, 1, 64, 32, seed=H, pad=1)
        s.check(max_q=n)


# ------------------------------------------------------------------ streams, graphs, helpers

def test_calls_follow_copies_and_other_kernels_of_their_stream():
    """The calls' kernels may start before the kernel in front of them has ended; what they read was copied or
    written right before them, and what they wrote is overwritten right behind them."""
    a, b = Step([(1, 2000)] * 8, 8, 2, 128, 16, seed=21), Step([(1, 2000)] * 8, 8, 2, 128, 16, seed=22)
    big = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    q, k, v = a.q.clone(), a.k.clone(), a.v.clone()
    cache = U.PagedCache(k, v)
    meta = [i32(a.cu), i32(a.kv), i32(a.table)]
    other = [i32(b.cu), i32(b.kv), i32(b.table)]
    want = [U.paged_attn_fwd(x.q, x.cache, *m, 1)[0].clone() for x, m in ((a, meta), (b, other))]
    wantc = [U.paged_attn_fwd(x.q, x.cache, *m, 0)[0].clone() for x, m in ((a, meta), (b, other))]
    o, lse = torch.empty_like(want[0]), torch.empty((8, 8), device="cuda")
    ws = U.paged_attn_workspace(q, cache, 0)
    out = []
    for i in range(12):
        x, m = ((a, meta), (b, other))[i & 1]
        big.fill_(i)                                            # a kernel of some length in front
        q.copy_(x.q)
        k.copy_(x.k)
        v.copy_(x.v)
        U.paged_attn_fwd(q, cache, *m, (1, 0)[i % 3 == 0], o=o, lse=lse, workspace=ws)
        out.append(o.clone())
        o.fill_(float("nan"))
    for i, got in enumerate(out):
        assert torch.equal(got, (wantc if i % 3 == 0 else want)[i & 1]), i
    healthy()


def test_append_then_attention_without_a_pause():
    """Each step's keys are written right before they are read: 40 decoding steps of one token in a row, the last
    one against the oracle, every one against the same call made alone."""
    H, Hkv, d, page, B = 8, 2, 128, 16, 3
    s = Step([(1, 900), (1, 15), (1, 200)], H, Hkv, d, page, seed=31, width_extra=4, spare=12)
    free = [p for p in range(s.cache.num_pages) if p not in set(s.table.reshape(-1))]
    cached, new, table, fr, n_free = i32(s.kv), i32([1] * B), i32(s.table), i32(free), i32([len(free)])
    ws = U.paged_attn_workspace(s.q, s.cache, 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    steps = [tuple(torch.randn((B, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv)) for _ in range(40)]
    torch.cuda.synchronize()
    outs, states = [], []
    for q, k, v in steps:
        cu, kv, slots, info = U.page_plan(cached, new, fr, n_free, table, page, s.cache.num_pages, B)
        U.kv_append(k, v, s.cache, slots)
        outs.append(U.paged_attn_fwd(q, s.cache, cu, kv, table, 1, workspace=ws))
        states.append((cu, kv))
        cached = kv
        n_free = n_free - info[1:2]
    torch.cuda.synchronize()
    for i, ((q, _, _), (cu, kv), (o, lse)) in enumerate(zip(steps, states, outs)):
        again = U.paged_attn_fwd(q, s.cache, cu, kv, table, 1)   # later tokens lie behind kv: they are not seen
        torch.cuda.synchronize()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1]), i
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = paged.paged_attention(f(steps[-1][0]), f(s.cache.k), f(s.cache.v), *(x.cpu().numpy() for x in states[-1]),
                                table.cpu().numpy(), True)
    hold(*outs[-1], ref, d)


def test_two_graphs_share_a_workspace():
    """A decoding graph and a mixed graph captured over one workspace and replayed in turn."""
    a, b = Step([(1, 3000), (1, 40)], 8, 2, 128, 16, seed=41), Step([(150, 700), (1, 900), (0, 5)], 8, 2, 128, 16, seed=42)
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
        calls.append((graph, o, lse, want, args))   # a graph reads its arguments where they were
    for i in (0, 1, 0, 0, 1, 1, 0):
        graph, o, lse, want, _ = calls[i]
        o.fill_(0)
        graph.replay()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    healthy()


def test_another_stream_and_two_at_once():
    """Two calls on two streams with their own workspaces, and one call whose outputs belong to a side stream."""
    a, b = Step([(1, 3000)] * 4, 8, 2, 128, 16, seed=11), Step([(70, 900)] * 3, 8, 2, 128, 16, seed=12)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    args = [(x.q, x.cache, i32(x.cu), i32(x.kv), i32(x.table), x.new[0]) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [U.paged_attn_fwd(*x, stream=st) for x, st in zip(args, (sa, sb))]
    torch.cuda.synchronize()
    for x, (o, lse) in zip((a, b), got):
        hold(o, lse, x.oracle(), 128)


def test_one_step_captured_and_replayed_while_requests_grow():
    """plan -> append -> attention in one graph: three decoding steps replayed with nothing but the lengths,
    the new rows and the free list changed on the device, each checked against the oracle."""
    H, Hkv, d, page, B = 8, 2, 128, 16, 5
    rng = np.random.default_rng(8)
    lens0 = [15, 16, 0, 40, 31]
    num, width, T = 40, 8, 6                       # one padding row
    cache = U.PagedCache(*(torch.full((num, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    order = rng.permutation(num)
    table = np.full((B, width), -1)
    at = 0
    for i, c in enumerate(lens0):
        n = -(-c // page)
        table[i, :n] = order[at:at + n]
        at += n
    cached, new, table_t, free, n_free = i32(lens0), i32([1] * B), i32(table), i32(order[at:]), i32([num - at])
    # the cached tokens come in through the same calls
    hist = torch.randn((2, sum(lens0), Hkv, d), device="cuda").to(torch.bfloat16)
    slots = [table[i, t // page] * page + t % page for i, c in enumerate(lens0) for t in range(c)]
    U.kv_append(hist[0], hist[1], cache, i32(slots))
    q, k, v = (torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    ws = U.paged_attn_workspace(q, cache, 1)

    def step():
        cu, kv, slot, info = U.page_plan(cached, new, free, n_free, table_t, page, num, T)
        U.kv_append(k, v, cache, slot)
        o, lse = U.paged_attn_fwd(q, cache, cu, kv, table_t, 1, workspace=ws)
        return cu, kv, slot, info, o, lse
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = (table_t.clone(), cache.k.clone(), cache.v.clone())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((table_t, cache.k, cache.v), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cu, kv, slot, info, o, lse = step()
    for i in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        before = cached.cpu().numpy()
        plan = paged.page_plan(before, [1] * B, free.cpu().numpy(), int(n_free), table_t.cpu().numpy(), page, num, T)
        pool = [paged.kv_append(x.double().cpu().numpy(), y.double().cpu().numpy(), plan[2]) for x, y in ((cache.k, k), (cache.v, v))]
        graph.replay()
        for g, w in zip((cu, kv, slot, info, table_t), plan):
            assert np.array_equal(g.cpu().numpy(), w)
        ref = paged.paged_attention(q.double().cpu().numpy(), *pool, plan[0], plan[1], plan[4], True)
        own = ref["owned"]
        assert own.sum() == B
        healthy()
        oo = o.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref["o"]) + (2.0 ** -8 + 2.0 ** -13) * ref["absv"] * (1 + 2.0 ** -8)
        assert np.all(np.abs(oo - ref["o"])[own] <= tol[own])
        cached.copy_(kv)
        n_free.sub_(info[1:2])
    assert cached.tolist() == [c + 3 for c in lens0]


def test_a_block_from_hidden_states_to_outputs():
    """The operators as a serving step uses them, between the framework's projections: hidden states -> QKV
    projection -> plan, append, paged attention -> output projection, in two chunks of a 400-token prompt, equal to
    the training form of the same block on the whole prompt."""
    H, Hkv, d, hidden, page, L = 8, 2, 64, 256, 16, 400
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = rnd(1, 1, L, hidden).to(torch.bfloat16)
    w = (rnd((H + 2 * Hkv) * d, hidden) / 16).to(torch.bfloat16)
    wo = (rnd(hidden, H * d) / 22).to(torch.bfloat16)
    q, k, v = U.qkv_proj(x, w, 1, H, Hkv, d)
    o_ref, lse_ref = U.attn_fwd(q, k, v, 1, U.Mask.causal())
    y_ref = U.out_proj(o_ref, wo, 1)
    cache = U.PagedCache.empty(30, page, Hkv, d)
    table = torch.full((1, 30), -1, dtype=torch.int32, device="cuda")
    cached, free, n_free = i32([0]), i32(np.random.default_rng(1).permutation(30)), i32([30])
    ys = []
    for a, e in ((0, 152), (152, 400)):
        qi, ki, vi = U.qkv_proj(x[:, :, a:e].contiguous(), w, 1, H, Hkv, d)
        cu, kv, slots, info = U.page_plan(cached, i32([e - a]), free, n_free, table, page, 30, e - a)
        U.kv_append(ki[0, 0], vi[0, 0], cache, slots)
        o, lse = U.paged_attn_fwd(qi[0, 0], cache, cu, kv, table, e - a)
        ys.append(U.out_proj(o[None, None], wo, 1))
        cached, n_free = kv, n_free - info[1:2]
        s = (lse - lse_ref[0, 0, :, a:e]).abs().max()
        assert s < 1e-4, s
    healthy()
    assert int(n_free) == 5 and int(cached) == L
    y = torch.cat(ys, 2).double()
    # both forms round weights and o to bf16: the difference of two such results, through the projection
    tol = 2.0 ** -8 * 4 * (o_ref.double().abs().max() + v.double().abs().max()) * wo.double().abs().sum(1).max()
    assert (y - y_ref.double()).abs().max() <= tol
    assert (y - y_ref.double()).norm() / y_ref.double().norm() < 2.0 ** -6


def test_helpers_refuse_what_the_kernels_cannot_read():
    s = Step([(2, 30)], 4, 2, 64, 16, seed=1)
    cu, kv, tab = i32(s.cu), i32(s.kv), i32(s.table)
    ok = dict(q=s.q, cache=s.cache, cu_q=cu, kv_lens=kv, block_table=tab, max_q=2)
    U.paged_attn_fwd(**ok)
    for bad in (dict(q=s.q.float()), dict(q=s.q.transpose(0, 1)), dict(cu_q=cu.long()), dict(cu_q=cu[:1]), dict(kv_lens=kv.cpu()),
                dict(block_table=tab.t().expand(3, 3)), dict(o=torch.empty(2, 4, 64, device="cuda")),
                dict(lse=torch.empty(2, 4, device="cuda")), dict(block_table=tab.float())):
        with pytest.raises(ValueError):
            U.paged_attn_fwd(**{**ok, **bad})
    with pytest.raises(U.UlyssesError):
        U.paged_attn_fwd(**ok, window=-1)
    with pytest.raises(U.UlyssesError):
        U.paged_attn_fwd(**ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        U.kv_append(s.q, s.q, s.cache, kv)
    with pytest.raises(ValueError):
        U.PagedCache(s.k, s.v.float())
    with pytest.raises(ValueError):
        U.PagedCache(s.k, s.v[1:])
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        U.kv_append(k, k.cpu(), s.cache, i32([0, 1]))


def test_helpers_refuse_sizes_past_32_bits():
    """The library's sizes are 32-bit: a larger one is refused, not taken by its low bits."""
    s = Step([(2, 30)], 4, 2, 64, 16, seed=1)
    ok = dict(q=s.q, cache=s.cache, cu_q=i32(s.cu), kv_lens=i32(s.kv), block_table=i32(s.table))
    for bad in (dict(window=2 ** 32 + 1), dict(max_q=2 ** 32 + 1), dict(window=-2 ** 32 + 1)):
        with pytest.raises(ValueError):
            U.paged_attn_fwd(**{**ok, **bad})
    U.paged_attn_fwd(**ok, window=2 ** 31 - 1, max_q=2 ** 31 - 1)
    with pytest.raises(ValueError):
        U.paged_attn_workspace(s.q, s.cache, 2 ** 32)
    one = i32([1])
    for sizes in ((16, 10, -1), (16, 2 ** 32 + 10, 1), (2 ** 32 + 16, 10, 1), (16, 10, 2 ** 32)):
        with pytest.raises(ValueError):
            U.page_plan(one, one, one, one, i32([[0, -1]]), *sizes)
    healthy()
