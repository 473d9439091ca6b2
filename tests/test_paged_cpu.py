"""CPU checks of the paged-cache calls: every refusal of the C ABI and of the torch helpers that
needs no GPU, and pins of the oracle against hand-worked cases and against the plain attention
oracle."""

import numpy as np
import pytest
import torch

import oracle
import oracle.paged as paged
import ulysses_sequence_gb300 as U

A, BIG = 1 << 20, 1 << 40  # addresses that are never dereferenced: each call is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ulysses_sequence_gb300 import build
    build.build()
    return U.load()


def cache(k=A, v=2 * A, pages=10, page=16, H_kv=2, d=64, strides=None):
    s = strides or (page * H_kv * d, H_kv * d, d)
    return U.KVCacheStruct(k, v, pages, page, H_kv, d, *s)


# ------------------------------------------------------------------ page_plan

def plan(B=2, T=8, page=16, width=4, stride=4, pages=10, cached=A, new=2 * A, free=3 * A, cap=10, n_free=4 * A, table=5 * A,
         cu=6 * A, kv=7 * A, slots=8 * A, info=9 * A):
    return U.ulysses_page_plan(B, T, page, width, stride, pages, cached, new, free, cap, n_free, table, cu, kv, slots, info, 0)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(T=-1), dict(page=8), dict(page=24), dict(page=8192), dict(page=0), dict(width=-1),
                                dict(stride=3), dict(pages=0), dict(cap=-1), dict(pages=1 << 28), dict(width=1 << 27),
                                dict(cached=0), dict(new=0), dict(n_free=0), dict(free=0), dict(table=0), dict(cu=0), dict(kv=0),
                                dict(slots=0), dict(info=0), dict(kv=A), dict(cu=4 * A), dict(table=3 * A), dict(info=6 * A),
                                dict(slots=5 * A)])
def test_plan_refuses_bad_arguments(kw):
    assert plan(**kw) == U.ERR_INVALID_ARG


def test_plan_refuses_what_it_cannot_do():
    assert plan(B=8193) == U.ERR_UNSUPPORTED
    assert plan(slots=8 * A + 2) == U.ERR_MISALIGNED
    assert plan(cached=A + 1) == U.ERR_MISALIGNED


def test_oracle_plan_by_hand():
    # page 16, three requests: 20 cached + 13 new fill two pages and start a third; nothing new; 0 + 33 new
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 3]
    table[1, :1] = [5]
    cu, kv, slots, info, out = paged.page_plan([20, 9, 0], [13, 0, 33], [1, 9, 0, 4, 6], 5, table, 16, 10, 48)
    assert cu.tolist() == [0, 13, 13, 46] and kv.tolist() == [33, 9, 33]
    assert out.tolist() == [[7, 3, 6, -1], [5, -1, -1, -1], [4, 0, 9, -1]]
    assert slots[:13].tolist() == [3 * 16 + 4 + t for t in range(12)] + [6 * 16]
    assert slots[13:46].tolist() == [4 * 16 + t for t in range(16)] + [t for t in range(16)] + [9 * 16]
    assert slots[46:].tolist() == [-1, -1] and info.tolist() == [46, 4, 0, 0]
    # a list of two pages, a row limit of 40: the last request loses a page and six tokens
    cu, kv, slots, info, out = paged.page_plan([20, 9, 0], [13, 0, 33], [1, 9, 0, 4, 6], 2, table, 16, 10, 40)
    assert cu.tolist() == [0, 13, 13, 40] and kv.tolist() == [33, 9, 27] and info.tolist() == [40, 2, 1, 6]
    assert out.tolist() == [[7, 3, 9, -1], [5, -1, -1, -1], [1, -1, -1, -1]]
    assert slots[29:].tolist() == [-1] * 11


# ------------------------------------------------------------------ kv_append

def append(c=None, T=4, k=3 * A, ks=128, v=4 * A, vs=128, slots=5 * A):
    return U.ulysses_kv_append(cache() if c is None else c, T, k, ks, v, vs, slots, 0)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(k=0), dict(v=0), dict(slots=0), dict(ks=120), dict(vs=0), dict(k=A), dict(v=2 * A),
                                dict(c=cache(pages=0)), dict(c=cache(page=12)), dict(c=cache(k=0)), dict(c=cache(v=A)),
                                dict(c=cache(H_kv=0)), dict(c=cache(d=0)), dict(c=cache(strides=(2048, 32, 64))),
                                dict(c=cache(strides=(-2048, 128, 64))), dict(c=cache(strides=(0, 128, 64))),
                                dict(c=cache(pages=1 << 27)), dict(c=cache(strides=(BIG, 128, 64)))])
def test_append_refuses_bad_arguments(kw):
    assert append(**kw) == U.ERR_INVALID_ARG


def test_append_refuses_what_it_cannot_do():
    assert append(c=cache(d=60)) == U.ERR_UNSUPPORTED
    assert append(k=3 * A + 8) == U.ERR_MISALIGNED
    assert append(vs=132) == U.ERR_MISALIGNED
    assert append(c=cache(k=A + 8)) == U.ERR_MISALIGNED
    assert append(c=cache(strides=(2052, 128, 64))) == U.ERR_MISALIGNED
    assert U.ulysses_kv_append(None, 4, 3 * A, 128, 4 * A, 128, 5 * A, 0) == U.ERR_INVALID_ARG
    assert append(T=0, k=0, v=0, slots=0) == U.OK


# ------------------------------------------------------------------ paged attention

def attn(c=None, B=2, T=4, H=4, max_q=1, kind=U.MASK_CAUSAL, window=0, q=3 * A, qs=256, cu=4 * A, kv=5 * A, table=6 * A, ts=4,
         width=4, o=7 * A, lse=8 * A, ws=9 * A, nbytes=1 << 30):
    return U.ulysses_paged_attn_fwd(cache() if c is None else c, B, T, H, max_q, kind, window, 0.0, q, qs, cu, kv, table, ts,
                                    width, o, lse, ws, nbytes, 0)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(T=-1), dict(H=0), dict(H=3), dict(max_q=-1), dict(kind=9), dict(window=-1),
                                dict(kind=U.MASK_NONE, window=5), dict(q=0), dict(cu=0), dict(kv=0), dict(table=0), dict(o=0),
                                dict(lse=0), dict(ws=0), dict(qs=248), dict(ts=3), dict(width=-1), dict(o=3 * A), dict(o=A),
                                dict(lse=7 * A), dict(ws=7 * A), dict(nbytes=0), dict(c=cache(pages=0)), dict(c=cache(page=20))])
def test_attn_refuses_bad_arguments(kw):
    assert attn(**kw) == U.ERR_INVALID_ARG


def test_attn_refuses_what_it_cannot_do():
    assert attn(kind=U.MASK_BLOCK_SPARSE) == U.ERR_UNSUPPORTED
    assert attn(c=cache(d=96)) == U.ERR_UNSUPPORTED
    assert attn(H=2 * 129) == U.ERR_UNSUPPORTED                       # more than 128 query heads to a key/value head
    assert attn(width=1 << 27, ts=1 << 27) == U.ERR_UNSUPPORTED       # more than 2^30 keys
    assert attn(q=3 * A + 8) == U.ERR_MISALIGNED
    assert attn(qs=260) == U.ERR_MISALIGNED
    assert attn(ws=9 * A + 128) == U.ERR_MISALIGNED
    assert attn(o=7 * A + 8) == U.ERR_MISALIGNED
    assert attn(B=0, q=0, cu=0, kv=0, table=0, o=0, lse=0, ws=0, nbytes=0) == U.OK
    assert attn(T=0, q=0, cu=0, kv=0, table=0, o=0, lse=0, ws=0, nbytes=0) == U.OK


def test_attn_workspace_size_depends_on_heads_alone():
    n = U.ulysses_paged_attn_workspace_size(32, 8, 128, 0)
    assert n > 0 and U.ulysses_paged_attn_workspace_size(32, 8, 128, 1) <= n
    for bad in ((0, 8, 128, 1), (32, 5, 128, 1), (32, 8, 96, 1), (32, 8, 128, -1), (258, 2, 64, 1)):
        assert U.ulysses_paged_attn_workspace_size(*bad) == 0


def test_torch_helpers_refuse_cpu_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        U.PagedCache(torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16))
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        U.page_plan(i, i, i, i, torch.zeros(1, 4, dtype=torch.int32), 16, 4, 1)
    with pytest.raises(ValueError, match="int32"):
        U.page_plan(i.long(), i, i, i, torch.zeros(1, 4, dtype=torch.int32), 16, 4, 1)
    with pytest.raises(ValueError, match="block_table"):
        U.page_plan(i, i, i, i, torch.zeros(1, 4), 16, 4, 1)


@pytest.mark.parametrize("causal", [True, False])
def test_oracle_attention_matches_the_plain_oracle(causal):
    """One request whose pages hold a whole sequence, all of it new: the paged oracle and the attention
    oracle agree; a later chunk alone gives the later rows."""
    L, H, Hkv, d, page = 48, 4, 2, 8, 16
    rng = np.random.default_rng(3)
    x = {n: torch.tensor(rng.standard_normal((1, 1, L, h, d))).to(torch.bfloat16) for n, h in (("q", H), ("k", Hkv), ("v", Hkv))}
    bits = {n: t.view(torch.int16).numpy().view(np.uint16) for n, t in x.items()}
    ref = oracle.attention_full(bits["q"], bits["k"], bits["v"], 1, oracle.Mask("causal" if causal else "none"))
    f = {n: t.double().numpy()[0, 0] for n, t in x.items()}
    order = [2, 0, 3]
    pool = {n: np.full((4, page, Hkv, d), np.nan) for n in "kv"}
    for i, p in enumerate(order):
        for n in "kv":
            pool[n][p] = f[n][i * page:(i + 1) * page]
    for start in (0, 17):
        got = paged.paged_attention(f["q"][start:], pool["k"], pool["v"], [0, L - start], [L], np.array([order]), causal)
        assert np.abs(got["o"] - ref["o"][0, 0, start:]).max() < 1e-12
        assert np.abs(got["lse"] - ref["lse"].reshape(H, L)[:, start:]).max() < 1e-12


def test_oracle_attention_window_and_missing_pages_by_hand():
    """Equal scores: a row's output is the mean of the values it may see."""
    page, d = 16, 8
    k, v = np.zeros((3, page, 1, d)), np.arange(3 * page)[:, None] * np.ones(d)
    v = v.reshape(3, page, 1, d)
    q = np.ones((2, 1, d))
    got = paged.paged_attention(q, k, v, [0, 2], [40], np.array([[0, 1, 2]]), True, window=4)
    assert np.allclose(got["o"][:, 0, 0], [np.mean([35, 36, 37, 38]), np.mean([36, 37, 38, 39])])
    got = paged.paged_attention(q, k, v, [0, 2], [40], np.array([[0, -1, 2]]), True)
    assert np.allclose(got["lse"][0], np.log([16 + 7, 16 + 8]))
    got = paged.paged_attention(q, k, v, [0, 2], [1], np.array([[0, 1, 2]]), True)      # the first row's position is -1
    assert got["lse"][0, 0] == -np.inf and np.all(got["o"][0] == 0) and got["lse"][0, 1] == 0.0
