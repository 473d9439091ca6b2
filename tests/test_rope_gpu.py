"""GPU parity of the rotary calls against the fp64 oracle, element by element, to bounds counted from their roundings:

- an output is rounded to bf16 once, off by at most 2^-8 of its value;
- before it, a cosine or sine is off by at most 2^-21 (the angle, below 4, is rounded to 24 bits and the function to 2 units),
  and the few fp32 steps of the norm and the pair's products by some 2^-23 each: at most 2^-19 of |A| (|a| + |b|) of the
  element's pair in all (`reach`), through the gradient's formula the same of its terms' magnitudes;
- a weight's gradient is an fp32 sum of terms that are off by 2^-19 of their reach each, and n additions in a row by 2^-24 of the
  magnitudes' sum each.
"""

import numpy as np
import pytest
import torch

import oracle.rope as rope
import ulysses_sequence_gb300 as U
from gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu

STEP, SLACK = 2.0 ** -8, 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def weights(seed, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]


def within(got, want, bound, name):
    got = f64(got).reshape(want.shape)
    off = np.abs(got - want) - bound
    assert np.isfinite(got).all() and off.max() <= 0, (name, float(off.max()), np.unravel_index(off.argmax(), off.shape))


def check_fwd(y, x, theta, r, w, eps, name):
    z = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    want = rope.turn(z, theta, r.interleaved, r.amplitude)
    within(y, want, STEP * np.abs(want) + SLACK * rope.reach(z, r.rot, r.interleaved, r.amplitude), name)


def check_bwd(dx, dw, dy, theta, r, x, w, eps, name, chain):
    want, want_w = rope.backward(dy, theta, r.interleaved, r.amplitude, x, w, eps)
    G = rope.reach(dy, r.rot, r.interleaved, r.amplitude)
    if w is None:
        within(dx, want, STEP * np.abs(want) + SLACK * G, name)
        return
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h, Gw = np.abs(x) * inv, G * np.abs(w)
    within(dx, want, STEP * np.abs(want) + SLACK * inv * (Gw + h * (Gw * h).mean(-1, keepdims=True)), name)
    within(dw, want_w, (SLACK + chain * 2.0 ** -24) * (G * h).sum((0, 1)), name + " weights")


def flat(t):
    return f64(t).reshape(-1, *t.shape[-2:])


# (P, B, Lp, H, H_kv, d, rot, interleaved, head layout, weights, pos0, amplitude)
SHARDS = [(1, 1, 1, 1, 1, 64, 64, False, False, None, 0, 1.0), (4, 2, 5, 8, 4, 128, 128, False, False, torch.bfloat16, 0, 1.0),
          (2, 3, 17, 6, 2, 64, 32, True, False, torch.float32, 1000003, 1.2), (8, 1, 33, 4, 1, 128, 96, True, False, None, 3, 1.0),
          (2, 2, 9, 12, 6, 128, 16, False, True, torch.float32, 0, 0.7), (4, 1, 6, 8, 2, 64, 48, False, True, torch.bfloat16, 0, 1.0),
          (1, 2, 130, 5, 5, 128, 0, False, False, torch.bfloat16, 0, 1.0), (2, 1, 700, 40, 8, 128, 128, False, False, torch.bfloat16, 0, 1.0),
          (64, 1, 3, 16, 2, 64, 64, True, False, torch.float32, -50, 1.0), (2, 1, 900, 33, 3, 64, 64, False, False, None, 2 ** 30, 1.0)]


def shard_case(P, B, Lp, H, Hkv, d, rot, inter, head, wtype, pos0, amp, seed=0):
    r = U.Rope(d, rot=rot, interleaved=inter, amplitude=amp)
    lead = (P, B, P * Lp) if head else (P, B, Lp)
    hq, hk = (H // P, U.kv_heads_per_group(Hkv, P)) if head else (H, Hkv)
    q, k, dq, dk = (randn(seed + i, *lead, h, d) for i, h in enumerate((hq, hk, hq, hk)))
    w = weights(seed + 9, d, wtype) if wtype else [None, None]
    layout = U.LAYOUT_HEAD_SHARDED if head else U.LAYOUT_TOKEN_SHARDED
    theta = rope.angles(rope.shard_positions(P, B, Lp, head, pos0), r.frequencies)
    return r, q, k, dq, dk, w, dict(layout=layout, pos0=pos0, kv_heads=Hkv), theta


@pytest.mark.parametrize("case", SHARDS)
def test_shards_forward(case):
    r, q, k, _, _, w, kw, theta = shard_case(*case)
    qo, ko = U.qk_rope_fwd(q, k, case[0], r, *w, eps=1e-5, **kw)
    for name, x, y, ww in (("q", q, qo, w[0]), ("k", k, ko, w[1])):
        check_fwd(y, flat(x), theta, r, None if ww is None else f64(ww), 1e-5, name)


@pytest.mark.parametrize("case", SHARDS)
def test_shards_backward(case):
    r, q, k, dq, dk, w, kw, theta = shard_case(*case)
    normed = w[0] is not None
    got = U.qk_rope_bwd(dq, dk, case[0], r, *((q, k) if normed else (None, None)), *w, eps=1e-5, **kw)
    assert len(got) == (4 if normed else 2)
    chain = 2 * (theta.shape[0] // 8 + 1) + 3 + 8 + 700  # of a lane, its pass, the warps, the blocks' rows
    for i, (name, x, dy, ww) in enumerate((("dq", q, dq, w[0]), ("dk", k, dk, w[1]))):
        check_bwd(got[i], got[2 + i] if normed else None, flat(dy), theta, r, flat(x), f64(ww) if normed else None, 1e-5, name, chain)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 5), (12, 3), (12, 4), (16, 8)])
@pytest.mark.parametrize("d,inter", [(64, False), (128, True), (128, False)])
def test_backward_without_epsilon(H, Hkv, d, inter):
    """eps = 0, with numbers of heads that leave places of a warp without one: those add nothing to the weights' gradients."""
    r, q, k, dq, dk, w, kw, theta = shard_case(2, 1, 21, H, Hkv, d, d, inter, False, torch.float32, 5, 1.0)
    got = U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, eps=0.0, **kw)
    for i, (name, x, dy, ww) in enumerate((("dq", q, dq, w[0]), ("dk", k, dk, w[1]))):
        check_bwd(got[i], got[2 + i], flat(dy), theta, r, flat(x), f64(ww), 0.0, name, 2 * (theta.shape[0] // 8 + 1) + 3 + 8 + 700)


def test_backward_against_differences():
    """Central differences of the fp64 forward, along the GPU's own gradient: they must give its square."""
    r, q, k, dq, dk, w, kw, theta = shard_case(2, 1, 40, 8, 4, 64, 32, False, False, torch.float32, 7, 1.1)
    g = U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, eps=1e-3, **kw)
    for x, dy, ww, dx, dw in ((q, dq, w[0], g[0], g[2]), (k, dk, w[1], g[1], g[3])):
        x, dy, ww, dx, dw = flat(x), flat(dy), f64(ww), flat(dx), f64(dw)

        def loss(x, w):
            return float((rope.forward(x, theta, r.interleaved, r.amplitude, w, 1e-3) * dy).sum())
        h = 1e-5
        # the gradient's elements are off by 2^-8 of themselves: so is the product with itself; weights by far less
        assert (loss(x + h * dx, ww) - loss(x - h * dx, ww)) / (2 * h) == pytest.approx(float((dx * dx).sum()), rel=STEP)
        assert (loss(x, ww + h * dw) - loss(x, ww - h * dw)) / (2 * h) == pytest.approx(float((dw * dw).sum()), rel=1e-4)


def test_in_place_and_repeatable():
    r, q, k, dq, dk, w, kw, _ = shard_case(2, 2, 300, 8, 2, 128, 128, False, False, torch.bfloat16, 0, 1.0)
    a = U.qk_rope_fwd(q, k, 2, r, *w, **kw)
    q2, k2 = q.clone(), k.clone()
    U.qk_rope_fwd(q2, k2, 2, r, *w, q_out=q2, k_out=k2, **kw)
    assert torch.equal(a[0], q2) and torch.equal(a[1], k2)
    b = U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, **kw)
    c = U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, **kw)
    q3, dk3 = q.clone(), dk.clone()
    d = U.qk_rope_bwd(dq, dk3, 2, r, q3, k, *w, dq=q3, dk=dk3, **kw)
    for x, y, z in zip(b, c, d):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_norm_of_extreme_heads():
    """A head of zeros, one whose square overflows bf16's neighbours, one with NaN, one with infinity: only their own outputs."""
    r = U.Rope(64)
    q = randn(1, 1, 1, 6, 4, 64)
    q[0, 0, 1, 2] = 0
    q[0, 0, 2, 1] = 1e15
    q[0, 0, 3, 0, 5] = float("nan")
    q[0, 0, 4, 3, 7] = float("inf")
    w = weights(2, 64, torch.float32)
    qo, ko = U.qk_rope_fwd(q, q, 1, r, *w, eps=1e-6)
    assert torch.all(qo[0, 0, 1, 2] == 0) and torch.isnan(qo[0, 0, 3, 0]).all()
    bad = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[4, 3] = True
    assert torch.isfinite(qo[0, 0][~bad]).all()
    theta = rope.angles(range(6), r.frequencies)
    x = flat(q)
    x[3, 0] = x[4, 3] = 1
    keep = ~bad.cpu().numpy()
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * f64(w[0])
    want = rope.turn(z, theta, False, 1.0)
    assert (np.abs(flat(qo) - want) <= STEP * np.abs(want) + SLACK * rope.reach(z, 64, False, 1.0))[keep].all()


def test_passed_elements_are_untouched_bits():
    """Behind `rot` nothing is computed without a norm: NaN and infinities there stay, and reach no turned element."""
    r = U.Rope(128, rot=32, interleaved=True, amplitude=3.0)
    bits = torch.randint(-2 ** 15, 2 ** 15, (1, 1, 50, 5, 128), dtype=torch.int16, device="cuda")
    bits[..., :32] = randn(3, 1, 1, 50, 5, 32).view(torch.int16)
    q = bits.view(torch.bfloat16)
    keep = ~torch.isnan(q[..., 32:])
    qo, _ = U.qk_rope_fwd(q, q[:, :, :, :1].contiguous(), 1, r)
    assert torch.equal(qo[..., 32:].view(torch.int16)[keep], bits[..., 32:][keep])
    assert torch.isnan(qo[..., 32:][~keep]).all() and torch.isfinite(qo[..., :32]).all()


# ------------------------------------------------------------------ packed rows

def requests(seed, B, T, far):
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, T + 1, B - 1)) if B > 1 else np.zeros(0, int)
    cu = np.concatenate([[0], cuts, [T]])
    lens = np.array([int(rng.integers(cu[i + 1] - cu[i], far)) for i in range(B)])
    return cu, lens


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,T,pad,H,Hkv,d,fused,wtype,far", [(1, 1, 0, 32, 8, 128, False, None, 9000), (3, 40, 7, 8, 3, 64, True, torch.float32, 2 ** 30),
                                                             (33, 100, 0, 6, 4, 128, True, torch.bfloat16, 70000),
                                                             (1025, 900, 20, 4, 1, 64, False, None, 500000), (2000, 4100, 3, 32, 8, 128, False, torch.bfloat16, 9000)])
@pytest.mark.parametrize("given", [False, True])
def test_rows(B, T, pad, H, Hkv, d, fused, wtype, far, given):
    """Requests with no rows among them, more than one level of the search, padded rows, slices of fused rows."""
    cu, lens = requests(B, B, T, far)
    owner = np.searchsorted(cu[1:], np.arange(T), side="right")
    at = lens[owner] - cu[owner + 1] + np.arange(T)
    r = U.Rope(d, scaling="yarn", factor=8.0)
    total = T + pad
    base = randn(T, total, H + 2 * Hkv, d)
    q, k = base[:, :H], base[:, H:H + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = weights(5, d, wtype) if wtype else [None, None]
    qo, ko = (torch.full((total, h, d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv))
    where = dict(positions=i32(np.concatenate([at, -5 - np.arange(pad)]))) if given else dict(cu_q=i32(cu), kv_lens=i32(lens))
    U.qk_rope_rows(q, k, r, w_q=w[0], w_k=w[1], eps=1e-5, q_out=qo, k_out=ko, **where)
    pick = np.unique(np.concatenate([[0, T - 1], np.random.default_rng(1).integers(0, T, 60)]))
    theta = rope.angles(at[pick], r.frequencies)
    for name, x, y, ww in (("q", q, qo, w[0]), ("k", k, ko, w[1])):
        check_fwd(y[pick], f64(x[pick]), theta, r, None if ww is None else f64(ww), 1e-5, name)
        if pad and not given:
            assert torch.all(y[T:] == 7.0)
        elif pad:
            theta_pad = rope.angles(-5 - np.arange(pad), r.frequencies)
            check_fwd(y[T:], f64(x[T:]), theta_pad, r, None if ww is None else f64(ww), 1e-5, name)


@pytest.mark.parametrize("d,wtype", [(64, None), (64, torch.bfloat16), (128, None), (128, torch.float32)])
@pytest.mark.parametrize("inter", [False, True])
def test_many_rows_of_many_heads(d, wtype, inter):
    """Rows enough for a warp to take several passes of one, two of them at a time, with heads left over; both layouts of pairs."""
    T, H, Hkv = 4103, 37, 9
    r = U.Rope(d, rot=d - 16, interleaved=inter, amplitude=1.1)
    q, k = randn(d, T, H, d), randn(d + 1, T, Hkv, d)
    w = weights(5, d, wtype) if wtype else [None, None]
    at = np.random.default_rng(d).integers(0, 10 ** 6, T)
    qo, ko = U.qk_rope_rows(q, k, r, positions=i32(at), w_q=w[0], w_k=w[1], eps=1e-5)
    theta = rope.angles(at, r.frequencies)
    for name, x, y, ww in (("q", q, qo, w[0]), ("k", k, ko, w[1])):
        check_fwd(y, f64(x), theta, r, None if ww is None else f64(ww), 1e-5, name)


def test_rows_in_place_in_fused_rows():
    r = U.Rope(128)
    rows = randn(3, 70, 14, 128)
    cu, lens = i32([0, 30, 70]), i32([500, 40])
    want = U.qk_rope_rows(rows[:, :8], rows[:, 8:11], r, cu_q=cu, kv_lens=lens)
    v = rows[:, 11:].clone()
    q, k = rows[:, :8], rows[:, 8:11]
    got = U.qk_rope_rows(q, k, r, cu_q=cu, kv_lens=lens, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rows[:, 11:], v)


def test_rows_agree_with_shards():
    """The same tokens as rows with positions and as a shard: the same bits."""
    r = U.Rope(64, interleaved=True)
    w = weights(4, 64, torch.bfloat16)
    q, k = randn(6, 1, 1, 333, 8, 64), randn(7, 1, 1, 333, 2, 64)
    a = U.qk_rope_fwd(q, k, 1, r, *w, pos0=12345)
    b = U.qk_rope_rows(q[0, 0], k[0, 0], r, positions=i32(12345 + np.arange(333)), w_q=w[0], w_k=w[1])
    assert torch.equal(a[0][0, 0], b[0]) and torch.equal(a[1][0, 0], b[1])


def test_empty_calls():
    r = U.Rope(64)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert U.qk_rope_rows(q, q, r, positions=i32([]))[0].shape == (0, 4, 64)
    x = randn(1, 5, 4, 64)
    out = torch.full_like(x, 3.0)
    U.qk_rope_rows(x, x, r, cu_q=i32([0]), kv_lens=i32([]), q_out=out, k_out=out.clone())
    assert torch.all(out == 3.0)
    e = torch.zeros(2, 1, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w = weights(1, 64, torch.float32)
    got = U.qk_rope_bwd(e, e, 2, r, e, e, *w, dw_q=torch.ones(64, device="cuda"))
    assert got[0].shape == e.shape and torch.all(got[2] == 0) and torch.all(got[3] == 0)


def test_streams_and_graphs():
    """A call on a stream of its own, and a captured forward and backward replayed on new inputs."""
    r, q, k, dq, dk, w, kw, _ = shard_case(2, 1, 500, 8, 2, 128, 128, False, False, torch.bfloat16, 0, 1.0)
    want_f, want_b = U.qk_rope_fwd(q, k, 2, r, *w, **kw), U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got_f, got_b = U.qk_rope_fwd(q, k, 2, r, *w, stream=side, **kw), U.qk_rope_bwd(dq, dk, 2, r, q, k, *w, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want_f + want_b, got_f + got_b):
        assert torch.equal(a, b)
    ins = [torch.zeros_like(t) for t in (q, k, dq, dk)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf = U.qk_rope_fwd(ins[0], ins[1], 2, r, *w, **kw)
        gb = U.qk_rope_bwd(ins[2], ins[3], 2, r, ins[0], ins[1], *w, **kw)
    for t, x in zip(ins, (q, k, dq, dk)):
        t.copy_(x)
    for _ in range(2):
        graph.replay()
    for a, b in zip(want_f + want_b, gf + gb):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ as they are used: the layer around the attention

def test_attention_sees_relative_positions_only():
    """Scores of turned queries and keys depend on the distance alone: moving all positions moves no output by more than
    the rounding of q and k (2^-8 of a score's terms, twice) and the attention's own."""
    P, L, H, d = 2, 256, 4, 64
    r = U.Rope(d)
    q, k, v = (randn(i, P, 1, L // P, H, d) for i in range(3))
    outs = []
    for pos0 in (0, 777):
        qr, kr = U.qk_rope_fwd(q, k, P, r, pos0=pos0)
        outs.append(f64(U.attn_fwd(qr, kr, v, P, U.Mask.causal())[0]))
    assert np.abs(outs[0] - outs[1]).max() <= 2 * 2e-2
    assert np.linalg.norm(outs[0] - outs[1]) <= 2 * 5e-3 * np.linalg.norm(outs[0])


def test_layer_forward_and_backward():
    """qkv_proj, norm and rotation, attention and back, against the same chain in fp64 torch with its gradients."""
    P, B, L, H, Hkv, d, hidden = 2, 1, 256, 4, 2, 64, 128
    r = U.Rope(d)
    w = weights(8, d, torch.float32)
    x, wqkv = randn(1, P, B, L // P, hidden), (randn(2, (H + 2 * Hkv) * d, hidden).float() / hidden ** 0.5).to(torch.bfloat16)
    q, k, v = U.qkv_proj(x, wqkv, P, H, Hkv, d)
    qr, kr = U.qk_rope_fwd(q, k, P, r, *w)
    mask = U.Mask.causal()
    o, lse = U.attn_fwd(qr, kr, v, P, mask)
    do = randn(3, *o.shape)
    dqr, dkr, dv = U.attn_bwd(qr, kr, v, o, lse, do, P, mask)
    dq, dk, dwq, dwk = U.qk_rope_bwd(dqr, dkr, P, r, q, k, *w)

    t64 = [t.double().transpose(0, 1).reshape(B, L, -1, d).requires_grad_() for t in (q, k, v)]
    w64 = [t.double().requires_grad_() for t in w]
    theta = torch.tensor(rope.angles(range(L), r.frequencies), device="cuda")[:, None]
    c, s = theta.cos(), theta.sin()

    def turned(t, ww):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * ww
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    qq, kk = turned(t64[0], w64[0]), turned(t64[1], w64[1]).repeat_interleave(H // Hkv, 2)
    scores = torch.einsum("blhd,bmhd->bhlm", qq, kk) / d ** 0.5
    scores = scores.masked_fill(torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    out = torch.einsum("bhlm,bmhd->blhd", scores.softmax(-1), t64[2].repeat_interleave(H // Hkv, 2))
    do64 = do.double().transpose(0, 1).reshape(B, L, H, d)
    grads = torch.autograd.grad(out, [*t64, *w64], do64)

    def rel(got, want):
        got = got.double()
        got = got.transpose(0, 1).reshape(want.shape) if got.dim() == 5 else got
        return float((got - want).norm() / want.norm())
    assert rel(o, out.detach()) <= 5e-3
    # the attention's gradients (5e-3, the acceptance of the attention tests) pass a norm and a rotation, which keep
    # relative errors, and one more rounding of inputs and outputs
    for name, got, want in zip(("dq", "dk", "dv", "dw_q", "dw_k"), (dq, dk, dv, dwq, dwk), grads):
        assert rel(got, want) <= 1.5e-2, name


def test_two_backward_calls_at_once():
    """On two streams with workspaces of their own, the allocations and the sums apart."""
    cases = [shard_case(2, 1, 4000, 16, 4, 128, 128, False, False, torch.bfloat16, 0, 1.0, seed=s) for s in (1, 2)]
    want = [U.qk_rope_bwd(c[3], c[4], 2, c[0], c[1], c[2], *c[5], **c[6]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [U.qk_rope_bwd(c[3], c[4], 2, c[0], c[1], c[2], *c[5], stream=s, **c[6]) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
