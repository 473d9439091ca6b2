"""What is measured of the paged-cache operators, on one GPU, with PyTorch holding the memory.

Three operators that serve a trained attention block from a paged key/value cache:

- ``page_plan``: block tables and slot maps of a batch, built on the GPU from request lengths;
- ``kv_append``: the new tokens' keys and values written to the pages that the slot map names;
- ``paged_attn``: attention of each request's new tokens (one for decoding, a chunk for
  prefilling) over its pages, the chunk itself among them.

``run`` is either the operators' plain form in elementary torch operations (``own`` false) or
the calls that a user makes of the package (``own`` true). ``exact`` says in 64 bits what the
outputs are.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a captured decoding step: 48 requests add one token each, the batch padded to 64 rows
        {"name": "plan_decode", "op": "page_plan", "B": 48, "T": 64, "page": 16, "width": 512, "lens": 1,
         "new_lo": 1, "new_hi": 1, "old_lo": 1, "old_hi": 8000, "idle": False},
        # a bulk admission: 1500 requests, prompts of very different lengths, some with nothing new
        {"name": "plan_prefill", "op": "page_plan", "B": 1500, "T": 131072, "page": 64, "width": 256, "lens": 2,
         "new_lo": 1, "new_hi": 170, "old_lo": 0, "old_hi": 12000, "idle": True},
        # a decoding step's keys and values: 64 rows, the last of them padding
        {"name": "append_decode", "op": "kv_append", "T": 64, "pad": 13, "H_kv": 8, "d": 128, "page": 16, "pages": 1024,
         "head_major": False, "fused": False},
        # keys and values cut out of rows of a fused QKV product, 64-wide heads, a head-major cache
        {"name": "append_odd", "op": "kv_append", "T": 3001, "pad": 0, "H_kv": 2, "d": 64, "page": 32, "pages": 200,
         "head_major": True, "fused": True},
        # a long prompt (the 32768 tokens of the GPT-7B-like layer with 8 key/value heads)
        {"name": "append_prefill", "op": "kv_append", "T": 32768, "pad": 0, "H_kv": 8, "d": 128, "page": 128, "pages": 320,
         "head_major": False, "fused": False},
        # one request decoding: latency
        {"name": "decode_one", "op": "paged_attn", "B": 1, "H": 32, "H_kv": 8, "d": 128, "page": 16, "mask": "causal",
         "window": 0, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 1499, "old_hi": 1499, "idle": False, "pad": 0,
         "head_major": False, "lens": 3},
        # a full decoding batch: 64 requests of 64 to 8192 tokens, grouped heads
        {"name": "decode_batch", "op": "paged_attn", "B": 64, "H": 32, "H_kv": 8, "d": 128, "page": 16, "mask": "causal",
         "window": 0, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 64, "old_hi": 8191, "idle": False, "pad": 0,
         "head_major": False, "lens": 4},
        # a few long requests, one key/value head to each of 16 query heads, larger pages
        {"name": "decode_long_mha", "op": "paged_attn", "B": 3, "H": 16, "H_kv": 16, "d": 128, "page": 64, "mask": "causal",
         "window": 0, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 9000, "old_hi": 32767, "idle": False, "pad": 0,
         "head_major": False, "lens": 5},
        # many short requests, 64-wide heads, a sliding window whose older pages are gone, a padded
        # batch with requests that add nothing, a head-major cache
        {"name": "decode_window_d64", "op": "paged_attn", "B": 200, "H": 8, "H_kv": 2, "d": 64, "page": 32, "mask": "causal",
         "window": 700, "single": 1.0, "q_lo": 1, "q_hi": 1, "old_lo": 0, "old_hi": 1500, "idle": True, "pad": 17,
         "head_major": True, "lens": 6},
        # chunked prefilling: four requests bring 512 tokens each over contexts up to 16384
        {"name": "chunk", "op": "paged_attn", "B": 4, "H": 32, "H_kv": 8, "d": 128, "page": 64, "mask": "causal",
         "window": 0, "single": 0.0, "q_lo": 512, "q_hi": 512, "old_lo": 1000, "old_hi": 15872, "idle": False, "pad": 0,
         "head_major": False, "lens": 7},
        # a mixed step: mostly decoding, a few odd chunks, some requests idle
        {"name": "mixed", "op": "paged_attn", "B": 24, "H": 32, "H_kv": 8, "d": 128, "page": 16, "mask": "causal",
         "window": 0, "single": 0.8, "q_lo": 33, "q_hi": 301, "old_lo": 0, "old_hi": 4000, "idle": True, "pad": 5,
         "head_major": False, "lens": 8},
        # the second half of a 16384-token prompt, the largest call
        {"name": "prefill", "op": "paged_attn", "B": 1, "H": 32, "H_kv": 8, "d": 128, "page": 128, "mask": "causal",
         "window": 0, "single": 0.0, "q_lo": 8192, "q_hi": 8192, "old_lo": 8192, "old_hi": 8192, "idle": False, "pad": 0,
         "head_major": False, "lens": 9},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["page_plan", "kv_append", "paged_attn", "paged_attn", "paged_attn", "paged_attn"])
    lens = rng.randrange(1, 1 << 20)
    if op == "page_plan":
        B = _log_int(rng, 1, 1500)
        hi = _log_int(rng, 1, max(1, 131072 // B))
        page = rng.choice([16, 32, 64, 128])
        old = _log_int(rng, 1, 12000)
        c = {"op": op, "B": B, "T": B * hi + rng.randrange(0, 40), "page": page, "width": (old + hi) // page + rng.randrange(1, 9),
             "lens": lens, "new_lo": rng.choice([1, (hi + 1) // 2]), "new_hi": hi, "old_lo": 0, "old_hi": old,
             "idle": rng.random() < 0.5}
        return c
    if op == "kv_append":
        T = _log_int(rng, 1, 32768)
        H_kv, d, page = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        return {"op": op, "T": T, "pad": min(T - 1, rng.choice([0, 0, 3, 20])), "H_kv": H_kv, "d": d, "page": page,
                "pages": T // page + rng.randrange(2, 60), "head_major": rng.random() < 0.3, "fused": rng.random() < 0.4}
    while True:
        kind = rng.choice(["decode", "decode", "few", "chunk", "mixed"])
        G = rng.choice([1, 2, 3, 4, 5, 8, 16])
        H_kv = rng.choice([1, 2, 4, 8, 16])
        B = _log_int(rng, 1, 128 if kind == "decode" else 16)
        old = _log_int(rng, 16, 32000)
        new = {"decode": 1, "few": _log_int(rng, 2, 8), "chunk": _log_int(rng, 9, 4096), "mixed": _log_int(rng, 9, 512)}[kind]
        mask = "none" if rng.random() < 0.15 else "causal"
        c = {"op": op, "B": B, "H": G * H_kv, "H_kv": H_kv, "d": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128, 256]),
             "mask": mask, "window": _log_int(rng, 20, 8000) if mask == "causal" and rng.random() < 0.25 else 0,
             "single": {"decode": 1.0, "mixed": 0.75}.get(kind, 0.0), "q_lo": (new + 1) // 2, "q_hi": new,
             "old_lo": 0 if rng.random() < 0.5 else old // 2, "old_hi": old, "idle": rng.random() < 0.4,
             "pad": rng.choice([0, 0, 7]), "head_major": rng.random() < 0.3, "lens": lens}
        scores = c["B"] * c["H"] * new * (old + new)        # what the plain form holds
        w = work(c)
        if c["H"] <= 64 and scores <= 1.5e9 and w["bytes"] <= 8e8 and w["flops"] <= 1.2e12 and B * (old + new) * H_kv * c["d"] <= 5e8:
            return c


def _lengths(case):
    """(new tokens, cached tokens) of each request: part of the case, not of its seed."""
    r = random.Random(case["lens"])
    new, old = [], []
    for i in range(case["B"]):
        if case["op"] == "page_plan":
            n = r.randint(case["new_lo"], case["new_hi"])
        else:
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
    if case["op"] == "page_plan":
        new, old = _lengths(case)
        page, B = case["page"], case["B"]
        fresh = sum(-(-(c + n) // page) - -(-c // page) for n, c in zip(new, old))
        # lengths in, row starts and lengths out, the slot map, the entries that tokens on old pages
        # read, and the new pages: taken from the list and written to the table
        return {"bytes": 4 * (2 * B + (B + 1) + B + case["T"] + B + 2 * fresh), "flops": 0}
    if case["op"] == "kv_append":
        rows = case["T"] - case["pad"]
        return {"bytes": 2 * 2 * rows * case["H_kv"] * case["d"] * 2 + 4 * case["T"], "flops": 0}
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
    row = case["H"] * case["d"]
    return {"bytes": 2 * 2 * tokens * row + 4 * tokens * case["H"] + 2 * 2 * keys * case["H_kv"] * case["d"]
            + 4 * (keys // case["page"] + 2 * case["B"]), "flops": 4 * pairs * row}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(g, pages, page, H_kv, d, head_major):
    """Keys and values of every page, indexed [page][token][head][element] in either order of memory."""
    if head_major:
        return tuple(_randn(g, pages, H_kv, page, d).permute(0, 2, 1, 3) for _ in range(2))
    return tuple(_randn(g, pages, page, H_kv, d) for _ in range(2))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if own:
        import ulysses_sequence_gb300 as U
        s["U"] = U
    if case["op"] == "page_plan":
        new, old = _lengths(case)
        B, page, width = case["B"], case["page"], case["width"]
        held = [-(-c // page) for c in old]
        pages = sum(-(-(c + n) // page) for n, c in zip(new, old)) + 50
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        has = torch.tensor(held, device=DEV)
        at = torch.arange(width, device=DEV)[None]
        first = (has.cumsum(0) - has)[:, None]
        table = torch.where(at < has[:, None], order[(first + at).clamp(max=pages - 1)], -1).to(torch.int32)
        s.update(num_pages=pages, new_lens=_i32(new), cached_lens=_i32(old), table=table,
                 free=order[sum(held):].contiguous(), n_free=_i32([pages - sum(held)]),
                 cu_q=torch.empty(B + 1, dtype=torch.int32, device=DEV), kv_lens=torch.empty(B, dtype=torch.int32, device=DEV),
                 slots=torch.empty(case["T"], dtype=torch.int32, device=DEV), info=torch.empty(4, dtype=torch.int32, device=DEV))
        return s
    if case["op"] == "kv_append":
        T, H_kv, d, page, pages = case["T"], case["H_kv"], case["d"], case["page"], case["pages"]
        s["cache_k"], s["cache_v"] = _cache(g, pages, page, H_kv, d, case["head_major"])
        if case["fused"]:  # the last two thirds of rows [query heads | key heads | value heads]
            rows = _randn(g, T, 3 * H_kv, d)
            s["k"], s["v"] = rows[:, H_kv:2 * H_kv], rows[:, 2 * H_kv:]
        else:
            s["k"], s["v"] = _randn(g, T, H_kv, d), _randn(g, T, H_kv, d)
        # tokens of one request follow one another inside a page; its pages lie anywhere
        at = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        s["slots"] = (at[t // page] * page + t % page).to(torch.int32)
        if case["pad"]:
            s["slots"][T - case["pad"]:] = -1
        if own:
            s["cache"] = s["U"].PagedCache(s["cache_k"], s["cache_v"])
        return s
    new, old = _lengths(case)
    B, page, d, H, H_kv = case["B"], case["page"], case["d"], case["H"], case["H_kv"]
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
    s["cache_k"], s["cache_v"] = _cache(g, pages, page, H_kv, d, case["head_major"])
    s.update(table=table, kv_lens=_i32(kv), cu_q=_i32([0] + list(np.cumsum(new))), tokens=tokens, max_q=max(1, max(new)),
             max_pages=max(held), q=_randn(g, T, H, d), o=torch.zeros(T, H, d, device=DEV, dtype=torch.bfloat16),
             lse=torch.zeros(H, T, device=DEV, dtype=torch.float32))
    if own:
        U = s["U"]
        s["cache"] = U.PagedCache(s["cache_k"], s["cache_v"])
        s["kind"] = U.Mask.causal() if case["mask"] == "causal" else U.Mask.none()
        s["workspace"] = U.paged_attn_workspace(s["q"], s["cache"], s["max_q"])
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"page_plan": _plain_plan, "kv_append": _plain_append, "paged_attn": _plain_attn}[s["op"]](s)


def _own(s):
    U = s["U"]
    if s["op"] == "page_plan":
        U.page_plan(s["cached_lens"], s["new_lens"], s["free"], s["n_free"], s["table"], s["page"], s["num_pages"], s["T"],
                    cu_q=s["cu_q"], kv_lens=s["kv_lens"], slot_map=s["slots"], info=s["info"])
        return {"cu_q": s["cu_q"], "kv_lens": s["kv_lens"], "slots": s["slots"], "table": s["table"], "info": s["info"]}
    if s["op"] == "kv_append":
        U.kv_append(s["k"], s["v"], s["cache"], s["slots"])
        return {"k": s["cache_k"], "v": s["cache_v"]}
    U.paged_attn_fwd(s["q"], s["cache"], s["cu_q"], s["kv_lens"], s["table"], s["max_q"], s["kind"], window=s["window"],
                     o=s["o"], lse=s["lse"], workspace=s["workspace"])
    return {"o": s["o"], "lse": s["lse"]}


def _plain_plan(s):
    """Row starts, lengths, new pages (taken from the end of the free list) and each token's slot."""
    B, T, page, width, num_pages = s["B"], s["T"], s["page"], s["width"], s["num_pages"]
    table, free = s["table"], s["free"]
    old = s["cached_lens"].long().clamp(0, width * page)
    wanted = s["new_lens"].long().clamp(min=0)
    ends = wanted.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends.clamp(max=T)])
    n = cu[1:] - cu[:-1]
    kv = old + n
    has = (old + page - 1) // page
    needs = (kv + page - 1) // page
    fresh = needs.clamp(max=width) - has
    before = fresh.cumsum(0) - fresh
    n_free = s["n_free"].long().clamp(0, free.numel())
    # the table: entry j of request i, from has to has + fresh, is new page number before + j - has
    j = torch.arange(width, device=DEV)[None]
    number = before[:, None] + j - has[:, None]
    is_new = (j >= has[:, None]) & (j < (has + fresh)[:, None])
    took = free[(n_free - 1 - number).clamp(0, max(0, free.numel() - 1))].long()
    took = torch.where((number < n_free) & (took >= 0) & (took < num_pages), took, -1)
    table.copy_(torch.where(is_new, took, table.long()))
    t = torch.arange(T, device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = old[i] + t - cu[i]
    at = pos // page
    entry = table[i, at.clamp(max=width - 1)].long()
    fine = (t < cu[-1]) & (at < width) & (entry >= 0) & (entry < num_pages)
    s["slots"].copy_(torch.where(fine, entry * page + pos % page, -1))
    s["cu_q"].copy_(cu)
    s["kv_lens"].copy_(kv)
    total = fresh.sum()
    missing = (needs - width).clamp(min=0).sum() + (total - n_free[0]).clamp(min=0)
    s["info"].copy_(torch.stack([cu[-1], torch.minimum(total, n_free[0]), missing, ends[-1] - cu[-1]]))
    return {"cu_q": s["cu_q"], "kv_lens": s["kv_lens"], "slots": s["slots"], "table": table, "info": s["info"]}


def _plain_append(s):
    rows = s["T"] - s["pad"]
    slots = s["slots"][:rows].long()
    at, token = slots // s["page"], slots % s["page"]
    s["cache_k"][at, token] = s["k"][:rows]
    s["cache_v"][at, token] = s["v"][:rows]
    return {"k": s["cache_k"], "v": s["cache_v"]}


def _plain_attn(s):
    """Every request's pages gathered side by side, scores of all its new tokens, a softmax."""
    B, H, H_kv, d, page = s["B"], s["H"], s["H_kv"], s["d"], s["page"]
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
    k = s["cache_k"][at].reshape(B, K, H_kv, d).float().masked_fill_(hide, 0)
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
    v = s["cache_v"][at].reshape(B, K, H_kv, d).float().masked_fill_(hide, 0)
    o = torch.matmul(x.view(B, H_kv, -1, K), v.permute(0, 2, 1, 3)).view(B, H_kv, H // H_kv, M, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, M, H, d)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, M, H)
    s["o"][:s["tokens"]] = o[of, row].to(torch.bfloat16)
    s["lse"][:, :s["tokens"]] = lse[of, row].t()
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "page_plan":
        return None  # whole numbers: they are compared for equality
    s = prepare(case, seed)
    if case["op"] == "kv_append":
        out = {}
        for name, pool, x in (("k", s["cache_k"], s["k"]), ("v", s["cache_v"], s["v"])):
            full = pool.double()
            flat = full.reshape(-1, case["H_kv"], case["d"])
            for a in range(0, case["T"], 4096):
                part = s["slots"][a:a + 4096].long()
                keep = part >= 0
                flat[part[keep]] = x[a:a + 4096][keep].double()
            out[name] = flat.reshape(pool.shape)
        return out
    H, H_kv, d, page = case["H"], case["H_kv"], case["d"], case["page"]
    o, lse = s["o"].double(), s["lse"].double()
    cu, kv_lens, table = s["cu_q"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
    for b in range(case["B"]):
        n, kv = cu[b + 1] - cu[b], kv_lens[b]
        if n == 0:
            continue
        ids = table[b][:-(-kv // page)]
        lost = sum(1 for p in ids if p < 0)            # pages before the window, never seen
        k = torch.cat([s["cache_k"][p] for p in ids[lost:]])[:kv - lost * page].double()
        v = torch.cat([s["cache_v"][p] for p in ids[lost:]])[:kv - lost * page].double()
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
