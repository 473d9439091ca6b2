"""More of the paged-cache calls on the GPU, held to the oracle and the bounds of test_paged_gpu.py: the wide copy of
kv_append, masks in the decode kernel, both kernels with heads of 128, scores that are NaN, a step that a graph
captures first, and a served block with requests that pause and finish."""

import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.paged as paged
import ulysses_sequence_gb300 as U
from gpu_util import need_gpu
from test_paged_gpu import Step, healthy, hold, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# ------------------------------------------------------------------ kv_append

# 98304 16-byte pieces of keys and more take the wide copy: one token fewer, exactly as many, one more; ragged ends
@pytest.mark.parametrize("T,H,d,page,head_major,fused", [(767, 8, 128, 16, False, False), (768, 8, 128, 64, False, True),
                                                         (769, 8, 128, 16, True, False), (2477, 5, 128, 32, True, True),
                                                         (11003, 1, 72, 16, False, True), (98304, 1, 8, 4096, False, False)])
def test_wide_append_moves_bits(T, H, d, page, head_major, fused):
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
    healthy()
    assert np.array_equal(as16(kc), want[0]) and np.array_equal(as16(vc), want[1])


# ------------------------------------------------------------------ masks in the decode kernel

# max_q x G of at most 16 rows: every request goes to the decode kernel, several tokens to a unit among them
@pytest.mark.parametrize("mask,window", [("causal", 0), ("none", 0), ("causal", 1), ("causal", 37), ("causal", 128), ("causal", 700)])
@pytest.mark.parametrize("d,G,n,page", [(128, 4, 1, 16), (64, 4, 4, 16), (128, 5, 3, 64), (64, 1, 1, 128), (128, 1, 16, 32), (64, 5, 2, 256)])
def test_masks_in_the_decode_kernel(mask, window, d, G, n, page):
    old = (0, 3, 15, 16, 62, 63, 64, 127, 128, 129, 300, 800)   # around the ends of 64- and 128-key tiles, past each window
    reqs = [(0 if i == 4 else max(1, n - i % 2), c) for i, c in enumerate(old)]
    s = Step(reqs, 2 * G, 2, d, page, seed=window + n, pad=3)
    s.check(max_q=n, mask=mask, window=window)
    if window > 0:
        # pages that lie behind every row's window are given back
        for i, (_, c) in enumerate(reqs):
            s.table[i, :max(0, c - window + 1) // page] = -1
        s.check(max_q=n, mask=mask, window=window)


@pytest.mark.parametrize("mask,window", [("causal", 0), ("causal", 90), ("none", 0)])
def test_both_kernels_with_heads_of_128(mask, window):
    """60 requests of 8 key/value heads: too many units for one kernel, chunks among decoding and idle requests."""
    rng = np.random.default_rng(window)
    reqs = [(0 if i % 13 == 6 else int(rng.integers(9, 50)) if i % 10 == 3 else 1, int(rng.integers(0, 300))) for i in range(60)]
    s = Step(reqs, 16, 8, 128, 16, seed=window, pad=4)
    s.check(max_q=70, mask=mask, window=window)


# ------------------------------------------------------------------ scores that are NaN

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,old,max_q", [(1, 40, 1), (1, 5000, 1), (40, 30, 40), (40, 5000, 40), (3, 700, 0)])
def test_a_nan_score_is_not_an_empty_row(n, old, max_q, d):
    """lse = -inf says that a row saw no key. A row with a NaN among its scores, from its query or from a key, gets NaN in
    o and lse, whole or joined from pieces; rows that do not see that key, and empty ones, keep their values."""
    s = Step([(n, old), (n, 20)], 8, 2, d, 16, seed=n + old, pad=1)
    s.kv[1] = n - 1                                   # its first row has position -1: no key
    last = old + n - 1
    s.q[0, 1, 5] = float("nan")                       # one head of one row
    page, at = s.table[0, last // 16], last % 16
    s.k[page, at, 1, 3] = float("nan")                # a key that only the last row sees, second key/value head
    o, lse = s.run(max_q)
    ref = s.oracle()
    nan = np.isnan(ref["lse"])
    assert nan.sum() == 1 + 4 and np.isneginf(ref["lse"][:, n]).all()
    assert np.array_equal(np.isnan(lse.cpu().numpy()), nan)
    rows = torch.tensor(nan.T, device="cuda")
    assert torch.isnan(o[rows]).all()
    o[rows], lse[torch.tensor(nan, device="cuda")] = 0.0, 0.0
    ref = {**ref, **{x: np.where(nan, 0.0, ref[x]) for x in ("lse", "sqk")}, **{x: np.where(nan.T[..., None], 0.0, ref[x]) for x in ("o", "absv")}}
    hold(o, lse, ref, d)


# ------------------------------------------------------------------ graphs and whole steps

_CAPTURED_FIRST = """
import sys
sys.path[:0] = ["tests"]
import torch
import ulysses_sequence_gb300 as U
from test_paged_gpu import i32
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
B, T, H, Hkv, d = 40, 79, 16, 8, 128
q, k, v = rnd(T, H, d), rnd(T, Hkv, d), rnd(T, Hkv, d)
cache = U.PagedCache(torch.zeros(200, 16, Hkv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(200, 16, Hkv, d, dtype=torch.bfloat16, device="cuda"))
cached, new, free, n_free = i32([0] * B), i32([40] + [1] * 39), i32(range(200)), i32([200])
table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
def step():
    cu, kv, slots, info = U.page_plan(cached, new, free, n_free, table, 16, 200, T)
    U.kv_append(k, v, cache, slots)
    return (info, *U.paged_attn_fwd(q, cache, cu, kv, table, 0))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
for a, b in zip(got, step()):
    assert torch.equal(a, b)
assert got[0].tolist() == [79, 42, 0, 0], got[0]
assert U.device_status()[0] == U.OK
print("captured first: ok")
"""


def test_the_first_step_of_a_process_is_captured():
    """No call before the capture: the helpers and the library set up what they need inside it."""
    r = subprocess.run([sys.executable, "-c", _CAPTURED_FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("d", [64, 128])
def test_a_block_serves_requests_that_pause_and_finish(d):
    """The operators as a server runs them, between the framework's projections: three prompts in one step, then decoding
    steps of one token each in which one request pauses, and one ends and gives its pages back to the list, from which a
    request that comes later takes them. Every output row equals the training form of the same block on the
    request's whole sequence."""
    H, Hkv, hidden, page, pages, width = 8, 2, 256, 16, 24, 16
    g = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = (rnd((H + 2 * Hkv) * d, hidden) / 16).to(torch.bfloat16)
    wo = (rnd(hidden, H * d) / 22).to(torch.bfloat16)
    # prompt, and the decoding steps in which the request runs; the fourth comes in with its prompt at step 9
    prompts, runs = [37, 150, 5, 60], [range(16), range(7), [0, 1, 2, 8, 9, 10, 15], range(10, 16)]
    x = [rnd(1, 1, p + len(r), hidden).to(torch.bfloat16) for p, r in zip(prompts, runs)]
    refs = []
    for xi in x:
        # the training form takes whole groups of eight tokens: zeros behind the last one, which no row before them sees
        q, k, v = U.qkv_proj(torch.nn.functional.pad(xi, (0, 0, 0, -xi.shape[2] % 8)), w, 1, H, Hkv, d)
        o, lse = U.attn_fwd(q, k, v, 1, U.Mask.causal())
        refs.append((U.out_proj(o, wo, 1)[0, 0], lse[0, 0], o.double().abs().max() + v.double().abs().max()))
    B = len(x)
    cache = U.PagedCache.empty(pages, page, Hkv, d)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = i32(np.random.default_rng(d).permutation(pages))
    cached, n_free, done = i32([0] * B), i32([pages]), [0] * B

    def step(new, T):
        """One step of new[i] tokens each in T rows; checks every request's rows."""
        nonlocal cached, n_free
        rows = torch.zeros((1, 1, T, hidden), dtype=torch.bfloat16, device="cuda")
        at = 0
        for i, n in enumerate(new):
            rows[0, 0, at:at + n] = x[i][0, 0, done[i]:done[i] + n]
            at += n
        q, k, v = U.qkv_proj(rows, w, 1, H, Hkv, d)
        cu, kv, slots, info = U.page_plan(cached, i32(new), free, n_free, table, page, pages, T)
        U.kv_append(k[0, 0], v[0, 0], cache, slots)
        o = torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda")
        o, lse = U.paged_attn_fwd(q[0, 0], cache, cu, kv, table, max(new), o=o)
        y = U.out_proj(o[None, None], wo, 1)[0, 0]
        healthy()
        assert info.tolist()[0] == at and info.tolist()[2:] == [0, 0]
        at = 0
        for i, n in enumerate(new):
            y_ref, lse_ref, size = refs[i]
            a, e = done[i], done[i] + n
            if n:
                # both forms round weights and o to bf16: the difference of two such results, through the projection
                tol = 2.0 ** -8 * 4 * size * wo.double().abs().sum(1).max()
                assert (y[at:at + n].double() - y_ref[a:e].double()).abs().max() <= tol, i
                assert (lse[:, at:at + n] - lse_ref[:, a:e]).abs().max() < 1e-4, i
            at, done[i] = at + n, e
        cached, n_free = kv, n_free - info[1:2]

    step(prompts[:3] + [0], sum(prompts[:3]) + 3)
    for t in range(16):
        if t == 7:   # the second request has ended: its pages go back to the end of the list
            held = -(-int(cached[1]) // page)
            free[int(n_free):int(n_free) + held] = table[1, :held].clone()
            table[1] = -1
            cached, n_free = cached * i32([1, 0, 1, 1]), n_free + held
        if t == 9:
            step([1, 0, 1, prompts[3]], 64)
        else:
            step([int(t in r) for r in runs], B)
    assert done == [p + len(r) for p, r in zip(prompts, runs)]
    live = [int(p) for i in (0, 2, 3) for p in table[i, :-(-done[i] // page)].tolist()]
    spare = free[:int(n_free)].tolist()
    assert sorted(live + spare) == list(range(pages))
