"""CPU checks of the rotary calls: every refusal of the C ABI and of the torch helpers that needs no GPU, the frequencies'
scalings, and pins of the oracle (by hand, and its gradients against differences)."""

import math
import types

import numpy as np
import pytest
import torch

import oracle.rope as rope
import ulysses_sequence_gb300 as U

A = 1 << 20  # addresses that are never dereferenced: each call is refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ulysses_sequence_gb300 import build
    build.build()
    return U.load()


def turn(turns=A, rot=64, inter=0, amplitude=1.0):
    return U.RopeStruct(turns, rot, inter, amplitude)


SHAPE = (2, 64, 8, 64, 4, 4)


def fwd(shape=SHAPE, layout=0, r=None, pos0=0, q=2 * A, k=3 * A, wq=0, wk=0, wide=0, eps=1e-6, qo=4 * A, ko=5 * A):
    return U.ulysses_qk_rope_fwd(U.Shape(*shape), layout, turn() if r is None else r, pos0, q, k, wq, wk, wide, eps, qo, ko, 0)


BAD = [dict(shape=(-1, 64, 8, 64, 4, 4)), dict(shape=(2, -4, 8, 64, 4, 4)), dict(shape=(2, 64, 0, 64, 4, 4)), dict(shape=(2, 64, 8, 64, 0, 4)),
       dict(shape=(2, 63, 8, 64, 4, 4)), dict(shape=(2, 64, 8, 64, 4, 3)), dict(shape=(2, 64, 8, 64, 4, -1)), dict(layout=2),
       dict(shape=(2, 64, 6, 64, 4, 6), layout=1), dict(r=turn(rot=-16)), dict(r=turn(rot=80)), dict(r=turn(turns=0)),
       dict(r=turn(amplitude=math.inf)), dict(r=turn(amplitude=math.nan)), dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(qo=5 * A),
       dict(qo=3 * A), dict(ko=2 * A), dict(qo=A), dict(wq=6 * A), dict(wk=6 * A), dict(wq=6 * A, wk=7 * A, eps=-1.0),
       dict(wq=6 * A, wk=7 * A, eps=math.nan), dict(wq=6 * A, wk=7 * A, eps=math.inf), dict(wq=4 * A, wk=7 * A)]


@pytest.mark.parametrize("kw", BAD)
def test_fwd_refuses_bad_arguments(kw):
    assert fwd(**kw) == U.ERR_INVALID_ARG


def test_one_tensor_as_queries_and_keys_is_not_written_in_place():
    """Where q is k, a result over q would be read as keys."""
    assert fwd(k=2 * A, qo=2 * A) == U.ERR_INVALID_ARG
    assert fwd(k=2 * A, ko=2 * A) == U.ERR_INVALID_ARG
    assert bwd(dko=2 * A, dq=2 * A) == U.ERR_INVALID_ARG
    assert bwd(**dict(NORM, k=6 * A, dk=6 * A)) == U.ERR_INVALID_ARG
    assert bwd(**dict(NORM, dko=6 * A, dq=6 * A)) == U.ERR_INVALID_ARG
    assert rows(k=2 * A, qo=2 * A) == U.ERR_INVALID_ARG


def test_fwd_refuses_no_rope():
    assert U.ulysses_qk_rope_fwd(U.Shape(*SHAPE), 0, None, 0, 2 * A, 3 * A, 0, 0, 0, 0.0, 4 * A, 5 * A, 0) == U.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(shape=(2, 64, 8, 96, 4, 4)), dict(r=turn(rot=24)), dict(shape=(65536, 65536, 8, 64, 4, 4)),
                                dict(shape=(32768, 32768, 8, 64, 4, 4), layout=1)])
def test_fwd_unsupported(kw):
    assert fwd(**kw) == U.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=2 * A + 8), dict(k=3 * A + 2), dict(qo=4 * A + 8), dict(ko=5 * A + 8), dict(r=turn(turns=A + 4)),
                                dict(wq=6 * A + 1, wk=7 * A), dict(wq=6 * A, wk=7 * A + 2, wide=1)])
def test_fwd_misaligned(kw):
    assert fwd(**kw) == U.ERR_MISALIGNED


def test_empty_shapes_launch_nothing():
    assert fwd(shape=(0, 64, 8, 64, 4, 4)) == U.OK and fwd(shape=(2, 0, 8, 64, 4, 4), q=0, k=0, qo=0, ko=0) == U.OK
    assert bwd(shape=(0, 64, 8, 64, 4, 4)) == U.OK
    assert rows(T=0) == U.OK and rows(pos=0, B=0) == U.OK


def bwd(shape=SHAPE, layout=0, r=None, dqo=2 * A, dko=3 * A, q=0, k=0, wq=0, wk=0, wide=0, eps=1e-6, dq=4 * A, dk=5 * A, dwq=0, dwk=0, ws=0,
        ws_bytes=1 << 24):
    return U.ulysses_qk_rope_bwd(U.Shape(*shape), layout, turn() if r is None else r, 0, dqo, dko, q, k, wq, wk, wide, eps, dq, dk, dwq, dwk,
                                 ws, ws_bytes, 0)


NORM = dict(q=6 * A, k=7 * A, wq=8 * A, wk=9 * A, dwq=10 * A, dwk=11 * A, ws=12 * A)


@pytest.mark.parametrize("kw", [dict(dqo=0), dict(dko=0), dict(dq=0), dict(dk=0), dict(dq=3 * A), dict(dk=4 * A), dict(layout=-1),
                                dict(NORM, q=0), dict(NORM, k=0), dict(NORM, wq=0), dict(NORM, wk=0), dict(NORM, dwq=0), dict(NORM, dwk=0),
                                dict(NORM, ws=0), dict(NORM, ws_bytes=100), dict(NORM, dwq=11 * A), dict(NORM, dwq=8 * A),
                                dict(NORM, ws=6 * A), dict(NORM, dq=7 * A), dict(NORM, eps=-1.0),
                                dict(NORM, shape=(0, 64, 8, 64, 4, 4), dwq=11 * A)])
def test_bwd_refuses_bad_arguments(kw):
    assert bwd(**kw) == U.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dqo=2 * A + 8), dict(dk=5 * A + 2), dict(NORM, q=6 * A + 8), dict(NORM, dwq=10 * A + 2),
                                dict(NORM, ws=12 * A + 8), dict(NORM, shape=(0, 64, 8, 64, 4, 4), dwk=11 * A + 2)])
def test_bwd_misaligned(kw):
    assert bwd(**kw) == U.ERR_MISALIGNED


def test_bwd_workspace_size():
    n = U.ulysses_qk_rope_bwd_workspace_size(U.Shape(*SHAPE))
    assert 0 < n <= 1 << 20 and U.ulysses_qk_rope_bwd_workspace_size(U.Shape(1, 1 << 20, 8, 64, 4, 4)) == n
    assert U.ulysses_qk_rope_bwd_workspace_size(U.Shape(2, 63, 8, 64, 4, 4)) == 0
    assert U.ulysses_qk_rope_bwd_workspace_size(U.Shape(2, 64, 8, 96, 4, 4)) == 0


def rows(T=5, H=8, H_kv=3, d=64, r=None, q=2 * A, qs=512, k=3 * A, ks=192, pos=13 * A, B=0, cu=0, kv=0, wq=0, wk=0, wide=0, eps=1e-6, qo=4 * A,
         qos=512, ko=5 * A, kos=192):
    return U.ulysses_qk_rope_rows(T, H, H_kv, d, turn() if r is None else r, q, qs, k, ks, pos, B, cu, kv, wq, wk, wide, eps, qo, qos, ko, kos, 0)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=0), dict(H_kv=0), dict(d=0), dict(B=-1), dict(q=0), dict(k=0), dict(qo=0), dict(ko=0),
                                dict(qs=504), dict(ks=184), dict(qos=0), dict(kos=-192), dict(pos=0, B=2), dict(pos=0, B=2, cu=14 * A),
                                dict(pos=4 * A), dict(pos=0, B=2, cu=4 * A, kv=15 * A), dict(qo=2 * A, qos=520), dict(qo=3 * A), dict(r=turn(rot=128)),
                                dict(wq=6 * A)])
def test_rows_refuse_bad_arguments(kw):
    assert rows(**kw) == U.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(qs=516), dict(kos=196), dict(q=2 * A + 2), dict(pos=13 * A + 2), dict(pos=0, B=2, cu=14 * A + 1, kv=15 * A)])
def test_rows_misaligned(kw):
    assert rows(**kw) == U.ERR_MISALIGNED


@pytest.mark.parametrize("kw", [dict(d=96, r=turn(rot=0)), dict(H=1 << 19, qs=1 << 26, qos=1 << 26), dict(H=(1 << 17) + 1, qs=1 << 24, qos=1 << 24), dict(qs=(1 << 31) + 8), dict(kos=1 << 33)])
def test_rows_unsupported(kw):
    assert rows(**kw) == U.ERR_UNSUPPORTED


# ------------------------------------------------------------------ the torch helpers, without a GPU

def test_rope_refuses():
    for kw in (dict(rot=24), dict(rot=-16), dict(rot=80), dict(frequencies=[1.0]), dict(frequencies=[math.nan] * 32), dict(scaling="other"),
               dict(factor=0.5), dict(base=0.0), dict(scaling="yarn", low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            U.Rope(64, device="cpu", **kw)
    with pytest.raises(ValueError, match="CUDA"):
        U.Rope(64, device="cpu")


def handle(d=64):
    return types.SimpleNamespace(d=d, rot=d, device=0, ref=None)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_helpers_refuse_by_name():
    r = handle()
    q, k = bf(2, 1, 4, 4, 64), bf(2, 1, 4, 2, 64)
    for fn in (U.qk_rope_fwd, U.qk_rope_bwd):
        with pytest.raises(ValueError, match="q must be contiguous"):
            fn(q, k, 2, r)
        with pytest.raises(ValueError, match="layout"):
            fn(q, k, 2, r, layout=3)
        for a, b in ((q[0], k), (q, k[:, :, :2]), (q[..., :32], k[..., :32])):
            with pytest.raises(ValueError, match="must be"):
                fn(a, b, 2, r)
        with pytest.raises(ValueError, match="must be"):
            fn(q, k, 4, r)
    with pytest.raises(ValueError, match="heads"):
        U.qk_rope_rows(bf(3, 4, 4, 64), bf(3, 4, 64), r, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="q must be bf16"):
        U.qk_rope_rows(bf(3, 4, 64), bf(3, 4, 64), r, positions=torch.zeros(3, dtype=torch.int32))


# ------------------------------------------------------------------ frequencies

def test_frequencies():
    f, a = U.rope_frequencies(64, base=10000.0)
    assert a == 1.0 and len(f) == 32 and f[0] == 1.0 and f[16] == pytest.approx(0.01, rel=1e-14)
    assert U.rope_frequencies(64, scaling="linear", factor=4.0)[0] == [x / 4 for x in f]
    ntk, a = U.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert a == 1.0 and ntk[0] == 1.0 and ntk[-1] == pytest.approx(f[-1] / 4, rel=1e-12)
    yarn, a = U.rope_frequencies(64, scaling="yarn", factor=4.0, trained=2048)
    assert a == pytest.approx(0.1 * math.log(4) + 1)
    for x, y in zip(f, yarn):
        r = 2048 * x / (2 * math.pi)
        assert y == x if r >= 32 else y == pytest.approx(x / 4, rel=1e-14) if r <= 1 else x / 4 < y < x
    assert U.rope_frequencies(0) == ([], 1.0)


# ------------------------------------------------------------------ the oracle

def test_oracle_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = np.array([[math.pi / 2, math.pi]])
    assert np.allclose(rope.turn(x, quarter, False, 1.0), [[[-3.0, -2.0, 1.0, -4.0, 5.0]]])
    assert np.allclose(rope.turn(x, quarter, True, 2.0), [[[-4.0, 2.0, -6.0, -8.0, 5.0]]])
    y = rope.forward(np.array([[[3.0, 4.0]]]), np.zeros((1, 1)), False, w=np.array([1.0, 2.0]), eps=12.5)
    assert np.allclose(y, [[[0.6, 1.6]]])
    assert rope.shard_positions(2, 2, 3, False, 5).tolist() == [5, 6, 7, 5, 6, 7, 8, 9, 10, 8, 9, 10]
    assert rope.shard_positions(2, 1, 2, True).tolist() == [0, 1, 2, 3] * 2


def test_oracle_angles_of_far_positions():
    # a whole number of turns and a quarter, from a frequency that 64 bits hold exactly
    f = 0.5
    p = 2 ** 30 + 7
    exact = (p * f) % (2 * math.pi)  # fmod of a value below 2^53 is exact but for 2 pi itself: 2^30 / (2 pi) turns of 1e-16
    assert rope.angles([p], [f])[0, 0] == pytest.approx(exact, abs=1e-6)
    assert rope.angles([-1], [1.0])[0, 0] == pytest.approx(2 * math.pi - 1, abs=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradients_against_differences(interleaved):
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 2, 16)), 1 + rng.standard_normal(16)
    theta = rng.uniform(0, 6, (3, 4))

    def loss(x, w):
        return float((rope.forward(x, theta, interleaved, 1.3, w, 1e-3) * dy).sum())
    dx, dw = rope.backward(dy, theta, interleaved, 1.3, x, w, 1e-3)
    h = 1e-5  # central differences: h^2 of the third derivative, and 1e-16 / h of rounding
    for _ in range(5):
        u, v = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        assert (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h) == pytest.approx(float((dx * u).sum()), abs=1e-7)
        assert (loss(x, w + h * v) - loss(x, w - h * v)) / (2 * h) == pytest.approx(float((dw * v).sum()), abs=1e-7)
