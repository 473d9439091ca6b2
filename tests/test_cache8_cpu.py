"""CPU checks of the 8-bit cache calls: every refusal of the C ABI and of the torch helpers that needs no GPU, and pins of
the oracle (e4m3 by hand and against torch, the append by hand)."""

import re

import numpy as np
import pytest
import torch

import oracle.cache8 as cache8
import test_kernel_sources_cpu as sources
import ulysses_sequence_gb300 as U

A, BIG = 1 << 20, 1 << 40  # addresses that are never dereferenced: each call is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ulysses_sequence_gb300 import build
    build.build()
    return U.load()


def cache(k=A, v=2 * A, ks=20 * A, vs=21 * A, pages=10, page=32, H_kv=2, d=64, strides=None, block=16):
    s = strides or (page * H_kv * d, H_kv * d, d)
    return U.KVCache8Struct(k, v, ks, vs, pages, page, H_kv, d, *s, block)


def append(c=None, T=4, k=3 * A, k_stride=128, v=4 * A, v_stride=128, slots=5 * A):
    return U.ulysses_kv_append8(cache() if c is None else c, T, k, k_stride, v, v_stride, slots, 0)


BAD_CACHE = [dict(pages=0), dict(page=24), dict(page=8), dict(k=0), dict(v=A), dict(ks=0), dict(vs=0), dict(vs=20 * A), dict(ks=A), dict(vs=2 * A),
             dict(H_kv=0), dict(d=0), dict(block=8), dict(block=24), dict(block=64), dict(block=0), dict(strides=(4096, 32, 64)),
             dict(strides=(-4096, 128, 64)), dict(strides=(0, 128, 64)), dict(strides=(BIG, 128, 64)), dict(pages=1 << 27)]


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_calls_refuse_bad_caches(kw):
    assert append(c=cache(**kw)) == U.ERR_INVALID_ARG
    assert attn(c=cache(**kw)) == U.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(T=-1), dict(k=0), dict(v=0), dict(slots=0), dict(k_stride=120), dict(v_stride=0), dict(k=A), dict(v=20 * A),
                                dict(slots=21 * A)])
def test_append_refuses_bad_arguments(kw):
    assert append(**kw) == U.ERR_INVALID_ARG


def test_append_refuses_what_it_cannot_do():
    assert append(c=cache(d=96)) == U.ERR_UNSUPPORTED
    assert append(c=cache(d=72)) == U.ERR_UNSUPPORTED
    assert append(k=3 * A + 8) == U.ERR_MISALIGNED
    assert append(v_stride=132) == U.ERR_MISALIGNED
    assert append(slots=5 * A + 2) == U.ERR_MISALIGNED
    assert append(c=cache(k=A + 8)) == U.ERR_MISALIGNED
    assert append(c=cache(strides=(4096 + 8, 128, 64))) == U.ERR_MISALIGNED
    assert U.ulysses_kv_append8(None, 4, 3 * A, 128, 4 * A, 128, 5 * A, 0) == U.ERR_INVALID_ARG
    assert append(T=0, k=0, v=0, slots=0) == U.OK


def attn(c=None, B=2, T=4, H=4, max_q=1, kind=U.MASK_CAUSAL, window=0, q=3 * A, qs=256, cu=4 * A, kv=5 * A, table=6 * A, ts=4,
         width=4, o=7 * A, lse=8 * A, ws=9 * A, nbytes=1 << 30):
    return U.ulysses_paged_attn8_fwd(cache() if c is None else c, B, T, H, max_q, kind, window, 0.0, q, qs, cu, kv, table, ts,
                                     width, o, lse, ws, nbytes, 0)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(T=-1), dict(H=0), dict(H=3), dict(max_q=-1), dict(kind=9), dict(window=-1),
                                dict(kind=U.MASK_NONE, window=5), dict(q=0), dict(cu=0), dict(kv=0), dict(table=0), dict(o=0),
                                dict(lse=0), dict(ws=0), dict(qs=248), dict(ts=3), dict(width=-1), dict(o=3 * A), dict(o=A),
                                dict(o=20 * A), dict(lse=21 * A), dict(lse=7 * A), dict(ws=7 * A), dict(nbytes=0)])
def test_attn_refuses_bad_arguments(kw):
    assert attn(**kw) == U.ERR_INVALID_ARG


def test_attn_refuses_what_it_cannot_do():
    assert U.ulysses_paged_attn8_fwd(None, 2, 4, 4, 1, 1, 0, 0.0, *([3 * A] * 1), 256, 4 * A, 5 * A, 6 * A, 4, 4, 7 * A, 8 * A, 9 * A, 1 << 30, 0) \
        == U.ERR_INVALID_ARG
    assert attn(kind=U.MASK_BLOCK_SPARSE) == U.ERR_UNSUPPORTED
    assert attn(c=cache(d=96)) == U.ERR_UNSUPPORTED
    assert attn(H=2 * 129) == U.ERR_UNSUPPORTED
    assert attn(width=1 << 26, ts=1 << 26) == U.ERR_UNSUPPORTED
    assert attn(q=3 * A + 8) == U.ERR_MISALIGNED
    assert attn(ws=9 * A + 128) == U.ERR_MISALIGNED
    assert attn(B=0, q=0, cu=0, kv=0, table=0, o=0, lse=0, ws=0, nbytes=0) == U.OK
    assert attn(T=0, q=0, cu=0, kv=0, table=0, o=0, lse=0, ws=0, nbytes=0) == U.OK


def test_helpers_refuse_by_name():
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    k = torch.zeros(3, 32, 2, 64, dtype=torch.uint8).view(f8)
    s = torch.zeros(3, 2, 2, dtype=torch.uint8).view(e8)
    with pytest.raises(ValueError, match="CUDA"):
        U.PagedCache8(k, k.clone(), s, s.clone())
    for bad in ((k, k[:2], s, s), (k.view(torch.uint8), k.view(torch.uint8), s, s), (k[0], k[0], s, s)):
        with pytest.raises(ValueError, match="k and v must"):
            U.PagedCache8(*bad)
    for bad in (s[:2], s.view(torch.uint8), s.transpose(1, 2), s[0], torch.zeros(3, 5, 2, dtype=torch.uint8).view(e8),
                torch.zeros(3, 0, 2, dtype=torch.uint8).view(e8)):
        with pytest.raises(ValueError, match="k_scale|v_scale"):
            U.PagedCache8(k, k, bad, bad)
    for block in (0, 5, 64):
        with pytest.raises(ValueError, match="block"):
            U.PagedCache8.empty(2, 32, 1, 64, block=block, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        U.PagedCache8.empty(2, 32, 1, 64, device="cpu")


# ------------------------------------------------------------------ the oracle

def test_oracle_e4m3_is_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.tensor(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.TABLE, want, equal_nan=True)
    x = np.concatenate([np.random.default_rng(1).standard_normal(4000) * 2.0 ** np.random.default_rng(2).integers(-14, 9, 4000),
                        (cache8.TABLE[:126] + cache8.TABLE[1:127]) / 2, cache8.TABLE[:127], [0.0, -0.0, 448.0, 460.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = np.concatenate([x, -x]).clip(-448, 448).astype(np.float32)
    assert np.array_equal(cache8.encode(x), torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert cache8.encode([np.inf, -np.inf, np.nan, 1e9]).tolist() == [0x7e, 0xfe, 0x7f, 0x7e]


def test_oracle_scales_by_hand():
    assert [cache8.need(x) for x in (448.0, 448.1, 224.0, 224.1, 1.75, 1.76, 0.0, 1e-40, 3e38)] == [0, 1, -1, 0, -8, -7, -117, -117, 119]


def test_oracle_append_by_hand():
    codes, scale = np.zeros((1, 32, 1, 1), np.uint8), np.full((1, 2, 1), 127, np.uint8)
    codes[0, :, 0, 0] = 0x38  # 1.0
    # block 0 begins anew with 448 and 1; block 1 goes on with 896: its scale doubles and 1.0 becomes a code of 0.5
    x = np.array([448.0, 1.0, 896.0]).reshape(3, 1, 1)
    c, s = cache8.append(codes, scale, x, [0, 1, 20], 16)
    assert s.reshape(-1).tolist() == [127, 128]
    assert cache8.TABLE[c[0, [0, 1, 2, 16, 20, 21], 0, 0]].tolist() == [448.0, 1.0, 1.0, 0.5, 448.0, 0.5]
    assert np.array_equal(cache8.values(c, s, 16)[0, [0, 2, 16, 20], 0, 0], [448.0, 1.0, 1.0, 896.0])
    # a smaller token changes no scale; rows outside the pool change nothing
    c2, s2 = cache8.append(c, s, x * 0 + 3.0, [5, -1, 32], 16)
    assert np.array_equal(s2, s) and cache8.TABLE[c2[0, 5, 0, 0]] == 3.0 and int((c2 != c).sum()) == 1


# ------------------------------------------------------------------ the kernels' sources

@pytest.mark.parametrize("name,waits", [("paged_decode8.cu", 1), ("paged_chunk8.cu", 3)])
def test_kernels_wait_for_what_is_on_its_way(name, waits):
    sources.test_kernels_wait_for_what_is_on_its_way_whatever_a_role_has_seen(name, waits)


def test_chunk_warps_meet_before_instructions_for_whole_warps():
    """Rows that leave the loop that stores them, and threads that loop over their own requests, meet before the next
    tcgen05.ld and the allocation."""
    text = sources.source("paged_chunk8.cu")
    turn = text.index("if (!valid) continue;")
    head = [m.end() for m in re.finditer(r"\bfor \([^{]*\{", text[:turn])][-1]
    for at in (head, text.index("paged_costs<")):
        before = text[at:at + re.search(sources.ALIGNED, text[at:]).start()]
        assert sources.MEETS.search(before), before
