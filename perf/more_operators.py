"""What is measured of the rotary and 8-bit cache operators, on one GPU, with PyTorch holding the memory.

Operators that stand between the projections and the attention of this package, in training and in serving:

- ``rope``: rotary positions of queries and keys, forward and backward, over token shards, head
  groups or packed serving rows;
- ``norm_rope``: the RMS norm of every query and key head with the rotation behind it, in one pass,
  forward and backward (with the gradients of the norms' weights);
- ``append8``: new tokens' keys and values rounded to 8 bits (e4m3) into the pages that the slot map names, with one
  power-of-two scale for each block of tokens and head;
- ``attn8``: paged attention over such a cache.

``run`` is either the operators' plain form in elementary torch operations (``own`` false) or
the calls that a user makes of the package (``own`` true). ``exact`` says in 64 bits what the
outputs are.

An 8-bit cache is returned as its codes, which are values of their own (float8), beside its scales: a key or value is code times
scale. The scale of a block and head is 2^k with the smallest whole k for which the largest new magnitude is at most
448 * 2^k, kept to [-117, 119]. A block whose first token is among the new ones starts anew; otherwise its scale
never shrinks, and where it grows the block's older tokens are rounded again.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a decoding step: one new token of each of 64 requests, whole heads rotated, positions from the lengths
        {"name": "rope_decode", "op": "rope", "form": "rows", "T": 64, "pad": 0, "B": 64, "H": 32, "H_kv": 8, "d": 128, "rot": 128,
         "inter": False, "far": 8192, "scaling": "none", "given": False, "fused": False, "wide": False, "lens": 1},
        # the backward pass over odd shards of a model with 64-wide heads, half of each rotated, neighbours paired
        {"name": "rope_bwd_odd", "op": "rope", "form": "bwd", "P": 4, "B": 3, "Lp": 1003, "H": 8, "H_kv": 4, "d": 64, "rot": 32,
         "inter": True, "head": False, "pos0": 17, "scaling": "linear", "wide": False},
        # a padded decoding step of a model with normed heads
        {"name": "norm_decode", "op": "norm_rope", "form": "rows", "T": 64, "pad": 13, "B": 51, "H": 32, "H_kv": 8, "d": 128, "rot": 128,
         "inter": False, "far": 32768, "scaling": "none", "given": False, "fused": True, "wide": True, "lens": 2},
        # chunks of prompts far into long contexts, cut out of rows of a fused QKV product, frequencies stretched
        {"name": "norm_prefill", "op": "norm_rope", "form": "rows", "T": 8192, "pad": 0, "B": 5, "H": 32, "H_kv": 8, "d": 128, "rot": 128,
         "inter": False, "far": 1000000, "scaling": "yarn", "given": False, "fused": True, "wide": False, "lens": 3},
        # the GPT-7B-like layer (32768 tokens, 8 shards) with 8 key/value heads: forward, and the largest, backward
        {"name": "norm_train_fwd", "op": "norm_rope", "form": "fwd", "P": 8, "B": 1, "Lp": 4096, "H": 32, "H_kv": 8, "d": 128, "rot": 128,
         "inter": False, "head": False, "pos0": 0, "scaling": "none", "wide": False},
        {"name": "norm_train_bwd", "op": "norm_rope", "form": "bwd", "P": 8, "B": 1, "Lp": 4096, "H": 32, "H_kv": 8, "d": 128, "rot": 128,
         "inter": False, "head": False, "pos0": 0, "scaling": "none", "wide": False},
        # a decoding step's keys and values, the last rows padding: most join a block that has tokens
        {"name": "append8_decode", "op": "append8", "T": 64, "pad": 13, "H_kv": 8, "d": 128, "page": 64, "block": 64, "pages": 160,
         "head_major": False, "fused": False, "single": True},
        # a long prompt, begun in the middle of a block
        {"name": "append8_prefill", "op": "append8", "T": 32761, "pad": 0, "H_kv": 8, "d": 128, "page": 64, "block": 64, "pages": 640,
         "head_major": False, "fused": True, "single": False},
        # one request decoding: latency
        {"name": "attn8_one", "op": "attn8", "B": 1, "H": 32, "H_kv": 8, "d": 128, "page": 16, "block": 16, "mask": "causal",
         "window": 0, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 1499, "old_hi": 1499, "idle": False, "pad": 0,
         "head_major": False, "lens": 4},
        # a full decoding batch: 64 requests of 64 to 8192 tokens, grouped heads
        {"name": "attn8_batch", "op": "attn8", "B": 64, "H": 32, "H_kv": 8, "d": 128, "page": 64, "block": 64, "mask": "causal",
         "window": 0, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 64, "old_hi": 8191, "idle": False, "pad": 0,
         "head_major": False, "lens": 5},
        # a mixed step, 64-wide heads, a sliding window whose older pages are gone, idle requests, a head-major cache
        {"name": "attn8_mixed", "op": "attn8", "B": 40, "H": 16, "H_kv": 4, "d": 64, "page": 32, "block": 16, "mask": "causal",
         "window": 1500, "single": 0.8, "q_lo": 33, "q_hi": 301, "old_lo": 0, "old_hi": 4000, "idle": True, "pad": 5,
         "head_major": True, "lens": 6},
        # the second half of a 16384-token prompt
        {"name": "attn8_prefill", "op": "attn8", "B": 1, "H": 32, "H_kv": 8, "d": 128, "page": 64, "block": 64, "mask": "causal",
         "window": 0, "single": 0.0, "q_lo": 8192, "q_hi": 8192, "old_lo": 8192, "old_hi": 8192, "idle": False, "pad": 0,
         "head_major": False, "lens": 7},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "norm_rope", "append8", "attn8", "attn8", "attn8"])
    lens = rng.randrange(1, 1 << 20)
    d = rng.choice([64, 128, 128])
    if op in ("rope", "norm_rope"):
        H_kv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "form": rng.choice(["rows", "fwd", "bwd"]), "H": H_kv * rng.choice([1, 2, 3, 4, 5, 8]), "H_kv": H_kv, "d": d,
             "rot": rng.choice([d, d, d // 2, d // 4 * 3, 16]), "inter": rng.random() < 0.4,
             "scaling": rng.choice(["none", "none", "linear", "ntk", "yarn"]), "wide": rng.random() < 0.5}
        if c["form"] == "rows":
            T = _log_int(rng, 1, 16384)
            pad = rng.choice([0, 0, 5]) if T > 5 else 0
            c.update(T=T, pad=pad, B=_log_int(rng, 1, max(1, min(T - pad, 512))), far=_log_int(rng, 20000, 1 << 24),
                     given=rng.random() < 0.3, fused=rng.random() < 0.4, lens=lens)
        else:
            c["P"] = rng.choice([1, 2, 4, 8])
            c.update(B=rng.choice([1, 1, 2, 3]), head=rng.random() < 0.3 and H_kv % c["P"] == 0, pos0=rng.choice([0, 0, 100000]),
                     Lp=_log_int(rng, 1, 131072 // c["P"] // 3 * 40 * 128 // ((c["H"] + H_kv) * d) // 4))
        return c
    if op == "append8":
        T = _log_int(rng, 1, 32768)
        page = rng.choice([16, 32, 64, 128, 256])
        return {"op": op, "T": T, "pad": min(T - 1, rng.choice([0, 0, 3, 20])), "H_kv": rng.choice([1, 2, 4, 5, 8]), "d": d, "page": page,
                "block": rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page]), "pages": (T if T < 600 else T // page) + rng.randrange(2, 60),
                "head_major": rng.random() < 0.3, "fused": rng.random() < 0.4, "single": T < 600 and rng.random() < 0.7}
    while True:
        kind = rng.choice(["decode", "decode", "few", "chunk", "mixed"])
        H_kv = rng.choice([1, 2, 4, 8, 16])
        B = _log_int(rng, 1, 128 if kind == "decode" else 16)
        old = _log_int(rng, 16, 32000)
        new = {"decode": 1, "few": _log_int(rng, 2, 8), "chunk": _log_int(rng, 9, 4096), "mixed": _log_int(rng, 9, 512)}[kind]
        mask = "none" if rng.random() < 0.15 else "causal"
        page = rng.choice([16, 32, 64, 128, 256])
        c = {"op": op, "B": B, "H": rng.choice([1, 2, 3, 4, 5, 8, 16]) * H_kv, "H_kv": H_kv, "d": d, "page": page,
             "block": rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page]),
             "mask": mask, "window": _log_int(rng, 20, 8000) if mask == "causal" and rng.random() < 0.25 else 0,
             "single": {"decode": 1.0, "mixed": 0.75}.get(kind, 0.0), "q_lo": (new + 1) // 2, "q_hi": new,
             "old_lo": 0 if rng.random() < 0.5 else old // 2, "old_hi": old, "idle": rng.random() < 0.4,
             "pad": rng.choice([0, 0, 7]), "head_major": rng.random() < 0.3, "lens": lens}
        scores = c["B"] * c["H"] * new * (old + new)        # what the plain form holds
        w = work(c)
        if c["H"] <= 64 and scores <= 1.5e9 and w["bytes"] <= 6e8 and w["flops"] <= 1.2e12 and B * (old + new) * H_kv * c["d"] <= 5e8:
            return c


def _lengths(case):
    """(new tokens, cached tokens) of each request: part of the case, not of its seed."""
    r = random.Random(case["lens"])
    new, old = [], []
    if case["op"] in ("rope", "norm_rope"):
        B, rows = case["B"], case["T"] - case["pad"]
        cuts = sorted(r.sample(range(1, rows), B - 1)) if B > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        return new, [r.randint(0, max(0, case["far"] - n)) for n in new]
    for i in range(case["B"]):
        n = 1 if r.random() < case["single"] else r.randint(case["q_lo"], case["q_hi"])
        c = r.randint(case["old_lo"], case["old_hi"])
        if case["idle"] and i % 7 == 3:
            n = 0
        if case["idle"] and i % 11 == 5:
            c = 0
        new.append(n)
        old.append(c)
    return new, old


def work(case):
    d, H_kv = case["d"], case["H_kv"]
    if case["op"] in ("rope", "norm_rope"):
        rows = case["T"] - case["pad"] if case["form"] == "rows" else case["P"] * case["B"] * case["Lp"]
        row = (case["H"] + H_kv) * d
        norm = case["op"] == "norm_rope"
        tensors = 3 if norm and case["form"] == "bwd" else 2     # a row's reads and writes
        each = (3 * case["rot"] / d + (0 if not norm else 15 if case["form"] == "bwd" else 5))
        small = 8 * (case["B"] + 1) if case["form"] == "rows" else 0
        weights = norm * 2 * d * ((4 if case["wide"] else 2) + (4 if case["form"] == "bwd" else 0))
        return {"bytes": 2 * tensors * rows * row + small + weights, "flops": int(rows * row * each)}
    if case["op"] == "append8":
        rows = case["T"] - case["pad"]
        blocks = rows if case["single"] else -(-rows // case["block"])
        return {"bytes": 3 * 2 * rows * H_kv * d + 4 * case["T"] + 2 * blocks * H_kv, "flops": 4 * rows * H_kv * d}
    new, old = _lengths(case)
    keys = pairs = tokens = 0
    for n, c in zip(new, old):
        if n == 0:
            continue
        tokens += n
        kv = c + n
        if case["mask"] == "none":
            keys += kv
            pairs += n * kv
        else:
            w = case["window"] or kv
            keys += kv - max(0, c - w + 1)
            pairs += int(np.minimum(np.arange(c + 1, kv + 1), w).sum())
    row = case["H"] * d
    return {"bytes": 2 * 2 * tokens * row + 4 * tokens * case["H"] + 2 * keys * H_kv * d + 2 * (keys // case["block"]) * H_kv
            + 4 * (keys // case["page"] + 2 * case["B"]), "flops": 4 * pairs * row}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


BASE, STRETCH, TRAINED = 10000.0, 8.0, 4096


def _frequencies(rot, scaling):
    """Radians a token for each pair, in 64 bits, and the amplitude of the rotation."""
    base = BASE * STRETCH ** (rot / (rot - 2)) if scaling == "ntk" else BASE
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / STRETCH
    if scaling == "yarn":  # pairs that turn less than once over the trained length are stretched, those of 32 turns are not
        keep = np.clip((TRAINED * f / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0, 1)
        f = f * keep + f / STRETCH * (1 - keep)
        return f, 0.1 * math.log(STRETCH) + 1.0
    return f, 1.0


def _codes(g, shape, blocks, spread):
    """Codes and scales of a pool [page][token][head][element] whose blocks differ in size by up to 2^spread either way."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    pages, page, H_kv, d = shape
    x = x.view(pages, blocks, page // blocks, H_kv, d)
    x *= torch.exp2(torch.rand(pages, blocks, 1, H_kv, 1, generator=g, device=DEV) * (2 * spread) - spread)
    k = _need(x.to(torch.bfloat16).float().abs().amax((2, 4), keepdim=True))
    codes = (x.to(torch.bfloat16).float() * _pow2(-k)).clamp(-448, 448).to(FP8)
    return codes.view(shape), (k + 127).to(torch.uint8).view(pages, blocks, H_kv).view(E8M0)


def _need(amax):
    """The smallest whole k with amax <= 448 * 2^k, in [-117, 119]: 448 = 0.875 * 2^9."""
    f, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (f > 0.875).to(torch.int32), -117).clamp(-117, 119)


def _pow2(k):
    """2^k in 32 bits, exactly, for whole k of [-126, 127]."""
    return ((k + 127).to(torch.int32) << 23).view(torch.float32)


def _head_major(x):
    return x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if own:
        import ulysses_sequence_gb300 as U
        s["U"] = U
    d, H_kv = case["d"], case["H_kv"]
    if case["op"] in ("rope", "norm_rope"):
        H = case["H"]
        f, s["amplitude"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = torch.tensor(f, device=DEV)
        if case["op"] == "norm_rope":
            w = torch.float32 if case["wide"] else torch.bfloat16
            s["w_q"], s["w_k"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(w) for _ in range(2))
        else:
            s["w_q"] = s["w_k"] = None
        if case["form"] == "rows":
            T = case["T"]
            if case["fused"]:  # the query and key parts of rows [query heads | key heads | value heads]
                rows = _randn(g, T, H + 2 * H_kv, d)
                s["q"], s["k"] = rows[:, :H], rows[:, H:H + H_kv]
            else:
                s["q"], s["k"] = _randn(g, T, H, d), _randn(g, T, H_kv, d)
            new, old = _lengths(case)
            s.update(cu_q=_i32([0] + list(np.cumsum(new))), kv_lens=_i32([c + n for n, c in zip(new, old)]), rows=sum(new))
            if case["given"]:
                at = [c + i for n, c in zip(new, old) for i in range(n)]
                s["positions"] = _i32(at + [0] * case["pad"])
                s["rows"] = T
            s["q_out"] = torch.zeros(T, H, d, device=DEV, dtype=torch.bfloat16)
            s["k_out"] = torch.zeros(T, H_kv, d, device=DEV, dtype=torch.bfloat16)
        else:
            P, B, Lp = case["P"], case["B"], case["Lp"]
            lead = (P, B, Lp * P) if case["head"] else (P, B, Lp)
            part = P if case["head"] else 1
            names = ("q", "k") if case["form"] == "fwd" else ("q", "k", "dq_out", "dk_out") if case["op"] == "norm_rope" else ("dq_out", "dk_out")
            for n in names:
                s[n] = _randn(g, *lead, (H_kv if "k" in n else H) // part, d)
        if own:
            U = s["U"]
            s["rope"] = U.Rope(d, rot=case["rot"], base=BASE, interleaved=case["inter"],
                               scaling=None if case["scaling"] == "none" else case["scaling"], factor=STRETCH, trained=TRAINED, device=DEV)
            s["layout"] = U.LAYOUT_HEAD_SHARDED if case.get("head") else U.LAYOUT_TOKEN_SHARDED
        return s
    page, blocks = case["page"], case["page"] // case["block"]
    if case["op"] == "append8":
        T, pages = case["T"], case["pages"]
        for n, spread in (("k", 1.0), ("v", 3.0)):
            codes, s[n + "_scale"] = _codes(g, (pages, page, H_kv, d), blocks, spread)
            s["cache_" + n] = _head_major(codes.view(torch.uint8)).view(FP8) if case["head_major"] else codes
        if case["fused"]:  # the last two thirds of rows [query heads | key heads | value heads]
            rows = _randn(g, T, 3 * H_kv, d)
            s["k"], s["v"] = rows[:, H_kv:2 * H_kv], rows[:, 2 * H_kv:]
        else:
            s["k"], s["v"] = _randn(g, T, H_kv, d), _randn(g, T, H_kv, d)
        at = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        if case["single"]:  # one token of each request, anywhere in a page of its own
            s["slots"] = (at[t] * page + torch.randint(0, page, (T,), generator=g, device=DEV)).to(torch.int32)
        else:               # tokens of one request, from the middle of its first page on
            t = t + page // 2 - 3
            s["slots"] = (at[t // page] * page + t % page).to(torch.int32)
        if case["pad"]:
            s["slots"][T - case["pad"]:] = -1
        if own:
            s["cache"] = s["U"].PagedCache8(s["cache_k"], s["cache_v"], s["k_scale"], s["v_scale"])
        return s
    new, old = _lengths(case)
    B, H = case["B"], case["H"]
    kv = [c + n for n, c in zip(new, old)]
    held = [-(-x // page) for x in kv]
    pages = sum(held) + 3
    width = max(held) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    has = torch.tensor(held, device=DEV)
    at = torch.arange(width, device=DEV)[None]
    first = (has.cumsum(0) - has)[:, None]
    table = torch.where(at < has[:, None], order[(first + at).clamp(max=pages - 1)], -1).to(torch.int32)
    if case["window"]:  # pages that no new token sees any more have been given back
        gone = torch.tensor([max(0, c - case["window"] + 1) // page for c in old], device=DEV)
        table.masked_fill_(at < gone[:, None], -1)
    tokens = sum(new)
    T = max(1, tokens + case["pad"])
    for n, spread in (("k", 0.7), ("v", 3.0)):
        codes, s[n + "_scale"] = _codes(g, (pages, page, H_kv, d), blocks, spread)
        s["cache_" + n] = _head_major(codes.view(torch.uint8)).view(FP8) if case["head_major"] else codes
    s.update(table=table, kv_lens=_i32(kv), cu_q=_i32([0] + list(np.cumsum(new))), tokens=tokens, max_q=max(1, max(new)),
             max_pages=max(held), q=_randn(g, T, H, d), o=torch.zeros(T, H, d, device=DEV, dtype=torch.bfloat16),
             lse=torch.zeros(H, T, device=DEV, dtype=torch.float32))
    if own:
        U = s["U"]
        s["cache"] = U.PagedCache8(s["cache_k"], s["cache_v"], s["k_scale"], s["v_scale"])
        s["kind"] = U.Mask.causal() if case["mask"] == "causal" else U.Mask.none()
        s["workspace"] = U.paged_attn_workspace(s["q"], s["cache"], s["max_q"])
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "norm_rope": _plain_rope, "append8": _plain_append8, "attn8": _plain_attn8}[s["op"]](s)


def _own(s):
    U = s["U"]
    if s["op"] in ("rope", "norm_rope"):
        norm = dict(w_q=s["w_q"], w_k=s["w_k"], eps=EPS) if s["op"] == "norm_rope" else {}
        if s["form"] == "rows":
            where = dict(positions=s["positions"]) if s["given"] else dict(cu_q=s["cu_q"], kv_lens=s["kv_lens"])
            U.qk_rope_rows(s["q"], s["k"], s["rope"], q_out=s["q_out"], k_out=s["k_out"], **where, **norm)
            return {"q": s["q_out"], "k": s["k_out"]}
        if s["form"] == "fwd":
            q, k = U.qk_rope_fwd(s["q"], s["k"], s["P"], s["rope"], layout=s["layout"], pos0=s["pos0"], **norm)
            return {"q": q, "k": k}
        if s["op"] == "rope":
            dq, dk = U.qk_rope_bwd(s["dq_out"], s["dk_out"], s["P"], s["rope"], layout=s["layout"], pos0=s["pos0"])
            return {"dq": dq, "dk": dk}
        dq, dk, dw_q, dw_k = U.qk_rope_bwd(s["dq_out"], s["dk_out"], s["P"], s["rope"], layout=s["layout"], pos0=s["pos0"],
                                           q=s["q"], k=s["k"], **norm)
        return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    if s["op"] == "append8":
        U.kv_append(s["k"], s["v"], s["cache"], s["slots"])
        return {"k": s["cache_k"], "v": s["cache_v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    U.paged_attn_fwd(s["q"], s["cache"], s["cu_q"], s["kv_lens"], s["table"], s["max_q"], s["kind"], window=s["window"],
                     o=s["o"], lse=s["lse"], workspace=s["workspace"])
    return {"o": s["o"], "lse": s["lse"]}


def _positions(s):
    """Each row's position, in the rows' own shape."""
    if s["form"] == "rows":
        if s["given"]:
            return s["positions"].long()
        cu, lens = s["cu_q"].long(), s["kv_lens"].long()
        t = torch.arange(s["rows"], device=DEV)
        of = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        return lens[of] - cu[of + 1] + t
    P, Lp = s["P"], s["Lp"]
    if s["head"]:
        return s["pos0"] + torch.arange(P * Lp, device=DEV).view(1, 1, -1).expand(P, s["B"], -1)
    return s["pos0"] + torch.arange(P * Lp, device=DEV).view(P, 1, Lp).expand(-1, s["B"], -1)


def _turn(x, cos, sin, rot, inter):
    """x [..., heads, d] in 32 bits, the pairs of its first `rot` elements turned."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1), x[..., rot:]], -1)


def _plain_rope(s):
    rot, inter = s["rot"], s["inter"]
    angle = _positions(s)[..., None, None].double() * s["freq"]
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    out = {}
    for n in ("q", "k"):
        w = s["w_" + n]
        if s["form"] == "bwd":
            dz = _turn(s["d" + n + "_out"].float(), cos, -sin, rot, inter)
            if w is None:
                out["d" + n] = dz.to(torch.bfloat16)
                continue
            x = s[n].float()
            inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            x = x * inv
            out["dw_" + n] = (dz * x).sum((0, 1, 2, 3), dtype=torch.float64).float()
            dz = dz * w.float()
            out["d" + n] = (inv * (dz - x * (dz * x).mean(-1, keepdim=True))).to(torch.bfloat16)
            continue
        x = s[n][:s["rows"]].float() if s["form"] == "rows" else s[n].float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        y = _turn(x, cos, sin, rot, inter).to(torch.bfloat16)
        if s["form"] == "rows":
            s[n + "_out"][:s["rows"]] = y
            y = s[n + "_out"]
        out[n] = y
    return out


def _plain_append8(s):
    """Scales of the touched blocks, their older tokens rounded again where a scale grew, then the new tokens."""
    rows, page, block, pages, H_kv, d = s["T"] - s["pad"], s["page"], s["block"], s["pages"], s["H_kv"], s["d"]
    blocks = page // block
    slots = s["slots"][:rows].long()
    of = slots // block
    fresh = torch.zeros(pages * blocks, dtype=torch.bool, device=DEV).index_put_((of,), slots % block == 0, accumulate=True)
    touched = torch.zeros(pages * blocks, dtype=torch.bool, device=DEV).index_fill_(0, of, True)
    for n in ("k", "v"):
        pool, x = s["cache_" + n], s[n][:rows].float()
        need = torch.full((pages * blocks, H_kv), -1000, dtype=torch.int32, device=DEV)
        need = need.scatter_reduce(0, of[:, None].expand(-1, H_kv), _need(x.abs().amax(-1)), "amax")
        old = s[n + "_scale"].view(torch.uint8).view(-1, H_kv).int() - 127
        k = torch.where(touched[:, None], torch.where(fresh[:, None], need, torch.maximum(need, old)), old)
        shift = torch.where(touched[:, None] & ~fresh[:, None], old - k, 0).view(pages, blocks, H_kv)
        shift = shift.repeat_interleave(block, 1)[..., None]
        again = (pool.float() * _pow2(shift.clamp(min=-126))).to(FP8)
        raw = pool.view(torch.uint8)
        raw.copy_(torch.where(shift < 0, again.view(torch.uint8), raw))
        code = (x * _pow2(-k[of][..., None])).clamp(-448, 448).to(FP8)
        raw[slots // page, slots % page] = code.view(torch.uint8)
        s[n + "_scale"].view(torch.uint8).copy_((k + 127).to(torch.uint8).view(pages, blocks, H_kv))
    return {"k": s["cache_k"], "v": s["cache_v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attn8(s):
    """Every request's pages gathered side by side and brought to 32 bits, scores of all its new tokens, a softmax."""
    B, H, H_kv, d, page, block = s["B"], s["H"], s["H_kv"], s["d"], s["page"], s["block"]
    table, kv_lens, cu = s["table"][:, :s["max_pages"]].long(), s["kv_lens"].long(), s["cu_q"].long()
    pages, M, K = s["cache_k"].shape[0], s["max_q"], s["max_pages"] * page
    t = torch.arange(s["tokens"], device=DEV)
    of = torch.searchsorted(cu[1:].contiguous(), t, right=True)      # each token's request
    row = t - cu[of]                                                 # and its row in it
    there = (table >= 0) & (table < pages)
    key = torch.arange(K, device=DEV)
    exists = there.repeat_interleave(page, 1) & (key[None] < kv_lens[:, None])
    hide = ~exists[:, :, None, None]
    at = table.clamp(0, pages - 1)

    def gather(n):
        scale = _pow2(s[n + "_scale"].view(torch.uint8)[at].int() - 127).reshape(B, K // block, 1, H_kv, 1)
        x = s["cache_" + n].view(torch.uint8)[at].reshape(B, K // block, block, H_kv, d).view(FP8).float()
        return x.mul_(scale).reshape(B, K, H_kv, d).masked_fill_(hide, 0)

    k = gather("k")
    q = torch.zeros(B, M, H, d, device=DEV)
    q[of, row] = s["q"][:s["tokens"]].float()
    q = q.reshape(B, M, H_kv, H // H_kv, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1))                       # [B][H_kv][heads x rows][K]
    del k
    x = x.view(B, H_kv, H // H_kv, M, K).mul_(1.0 / math.sqrt(d))
    allowed = exists[:, None, :]
    if s["mask"] == "causal":
        pos = (kv_lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(M, device=DEV)[None]
        allowed = allowed & (key[None, None] <= pos[:, :, None])
        if s["window"]:
            allowed = allowed & (key[None, None] > pos[:, :, None] - s["window"])
    x.masked_fill_(~allowed[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H_kv, -1, K), gather("v").permute(0, 2, 1, 3)).view(B, H_kv, H // H_kv, M, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, M, H, d)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, M, H)
    s["o"][:s["tokens"]] = o[of, row].to(torch.bfloat16)
    s["lse"][:, :s["tokens"]] = lse[of, row].t()
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "norm_rope": _exact_rope, "append8": _exact_append8, "attn8": _exact_attn8}[case["op"]](case, s)


def _exact_rope(case, s):
    """Pairs as complex numbers, rows a slab at a time."""
    rot, inter, d = case["rot"], case["inter"], case["d"]
    if case["form"] == "rows":
        new, old = _lengths(case)
        pos = torch.tensor([c + i for n, c in zip(new, old) for i in range(n)], device=DEV)
        if case["given"]:
            pos = torch.cat([pos, pos.new_zeros(case["pad"])])
    else:
        m = torch.arange(case["P"] * case["B"] * case["Lp"] * (case["P"] if case["head"] else 1), device=DEV)
        L = case["P"] * case["Lp"]
        pos = case["pos0"] + (m % L if case["head"] else m // (case["B"] * case["Lp"]) * case["Lp"] + m % case["Lp"])

    def spin(x, at, sign):  # [rows, heads, d] in 64 bits
        turn = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device=DEV), sign * at.double()[:, None] * s["freq"])[:, None]
        if inter:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            y = torch.cat([z.real, z.imag], -1)
        return torch.cat([y, x[..., rot:]], -1)

    out = {}
    for n in ("q", "k"):
        w = None if s["w_" + n] is None else s["w_" + n].double()
        src = s["d" + n + "_out"] if case["form"] == "bwd" else s[n]
        flat = src.reshape(-1, *src.shape[-2:])
        got = torch.zeros(flat.shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(d, dtype=torch.float64, device=DEV)
        for a in range(0, pos.numel(), 4096):
            at = pos[a:a + 4096]
            e = a + at.numel()
            x = flat[a:e].double()
            if case["form"] == "bwd":
                z = spin(x, at, -1.0)
                if w is not None:
                    x = s[n].reshape(flat.shape)[a:e].double()
                    r = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
                    dw += (z * x / r).sum((0, 1))
                    z = z * w / r - x * ((z * w * x).sum(-1, keepdim=True) / (d * r ** 3))
                got[a:e] = z
            else:
                if w is not None:
                    x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w
                got[a:e] = spin(x, at, 1.0)
        if case["form"] == "bwd":
            out["d" + n] = got.view(src.shape)
            if w is not None:
                out["dw_" + n] = dw
        else:
            out[n] = got.view(src.shape)
    return out


def _exact_append8(case, s):
    """Block by block on the host for the scales; the codes that 64-bit values would have, before any rounding."""
    block, H_kv, d, rows = case["block"], case["H_kv"], case["d"], case["T"] - case["pad"]
    slots = s["slots"][:rows].long()
    host = slots.cpu().numpy()
    out = {}
    for n in ("k", "v"):
        x = s[n][:rows].double()
        top = x.abs().amax(-1).cpu().numpy()                                     # [rows][H_kv]
        byte = s[n + "_scale"].view(torch.uint8).reshape(-1, H_kv).cpu().numpy().astype(np.int64)
        was = byte.copy()
        order = np.argsort(host // block, kind="stable")
        marks = np.flatnonzero(np.diff(host[order] // block)) + 1
        for run in np.split(order, marks):
            b = host[run[0]] // block
            largest = top[run].max(0)
            k = np.array([-117 if t == 0 else min(119, max(-117, math.ceil(math.log2(t / 448.0) - 1e-9))) for t in largest]) + 127
            byte[b] = k if (host[run] % block == 0).any() else np.maximum(k, was[b])
        pool = s["cache_" + n].double()
        codes = pool.reshape(-1, block, H_kv, d)
        fresh = np.zeros(len(byte), bool)
        fresh[host[host % block == 0] // block] = True
        grown = (byte != was) & ~fresh[:, None]
        codes *= torch.tensor(np.where(grown, 2.0 ** (was - byte), 1.0), device=DEV)[:, None, :, None]
        flat = codes.reshape(-1, H_kv, d)
        flat[slots] = x / torch.tensor(2.0 ** (byte[host // block] - 127.0), device=DEV)[..., None]
        out[n] = flat.reshape(pool.shape)
        out[n + "_scale"] = torch.tensor(2.0 ** (byte - 127.0), device=DEV).reshape(s[n + "_scale"].shape)
    return out


def _exact_attn8(case, s):
    H, H_kv, d, page, block = case["H"], case["H_kv"], case["d"], case["page"], case["block"]
    o, lse = s["o"].double(), s["lse"].double()
    cu, kv_lens, table = s["cu_q"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
    sizes = {n: 2.0 ** (s[n + "_scale"].view(torch.uint8).double() - 127) for n in ("k", "v")}
    for b in range(case["B"]):
        n, kv = cu[b + 1] - cu[b], kv_lens[b]
        if n == 0:
            continue
        ids = table[b][:-(-kv // page)]
        lost = sum(1 for p in ids if p < 0)            # pages before the window, never seen
        at = torch.tensor(ids[lost:], device=DEV)
        k, v = ((s["cache_" + n].view(torch.uint8)[at].view(FP8).double().unflatten(1, (-1, block)) * sizes[n][at][:, :, None, :, None])
                .reshape(-1, H_kv, d)[:kv - lost * page] for n in ("k", "v"))
        where = torch.arange(lost * page, kv, device=DEV)
        for a in range(0, n, 1024):
            e = min(n, a + 1024)
            pos = torch.arange(kv - n + a, kv - n + e, device=DEV)[:, None]
            bad = torch.zeros(e - a, kv - lost * page, dtype=torch.bool, device=DEV)
            if case["mask"] == "causal":
                bad |= where[None] > pos
                if case["window"]:
                    bad |= where[None] <= pos - case["window"]
            for h in range(H):
                kh = h // (H // H_kv)
                z = s["q"][cu[b] + a:cu[b] + e, h].double() @ k[:, kh].t() / d ** 0.5
                z[bad] = -math.inf
                norm = torch.logsumexp(z, 1)
                lse[h, cu[b] + a:cu[b] + e] = norm
                o[cu[b] + a:cu[b] + e, h] = torch.exp(z - norm[:, None]) @ v[:, kh]
    return {"o": o, "lse": lse}
