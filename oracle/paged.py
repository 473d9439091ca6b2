"""Oracle of the paged-cache calls -- TEST INFRASTRUCTURE ONLY (see the package docstring).

Plain loops and fp64 numpy over host arrays, written from the definitions in
``include/ulysses.h`` ("Serving from a paged key/value cache"):

* ``page_plan``  -- block tables and slot maps from request lengths, request by request, token by
  token;
* ``kv_append``  -- rows copied to their slots;
* ``paged_attention`` -- softmax attention of each request's new tokens over the keys that its
  block table names, and, beside o and lse, what an error bound needs: the sum of weight x |v|
  behind every element of o, the largest sum of |q||k| behind a row's scores, and the row's number
  of keys.
"""

from __future__ import annotations

import numpy as np


def page_plan(cached, new, free_pages, n_free, table, page, num_pages, T):
    """Returns (cu_q, kv_lens, slot_map, info, new table)."""
    table = np.array(table, dtype=np.int64, copy=True)
    B, width = table.shape
    n_free = min(max(int(n_free), 0), len(free_pages))
    cu, kv, slots = [0], [], np.full(T, -1, dtype=np.int64)
    taken = missing = dropped = 0
    for i in range(B):
        c = min(max(int(cached[i]), 0), width * page)
        want = max(int(new[i]), 0)
        n = min(want, T - cu[-1])
        dropped += want - n
        has, need = -(-c // page), -(-(c + n) // page)
        for j in range(has, need):
            if j >= width:
                missing += 1
                continue
            if taken < n_free:
                e = int(free_pages[n_free - 1 - taken])
            else:
                e = -1
                missing += 1
            taken += 1
            table[i, j] = e if 0 <= e < num_pages else -1
        for t in range(n):
            j = (c + t) // page
            if j < width and 0 <= table[i, j] < num_pages:
                slots[cu[-1] + t] = table[i, j] * page + (c + t) % page
        cu.append(cu[-1] + n)
        kv.append(c + n)
    info = [cu[-1], min(taken, n_free), missing, min(dropped, 2 ** 31 - 1)]
    return np.array(cu), np.array(kv, dtype=np.int64), slots, np.array(info), table


def kv_append(pool, x, slots):
    """pool [num_pages][page][H][d] with row t of x [T][H][d] at slots[t]; others unchanged."""
    out = np.array(pool, copy=True)
    page = pool.shape[1]
    for t, s in enumerate(slots):
        if 0 <= s < pool.shape[0] * page:
            out[s // page, s % page] = x[t]
    return out


def permitted(row_pos, keys, causal, window):
    """Which of `keys` (positions) the row at position row_pos may see."""
    ok = np.ones(len(keys), dtype=bool)
    if causal:
        ok &= keys <= row_pos
        if window > 0:
            ok &= keys > row_pos - window
    return ok


def paged_attention(q, k_pool, v_pool, cu_q, kv_lens, table, causal, window=0, scale=0.0):
    """q [T][H][d] and the pools [num_pages][page][H_kv][d], all fp64. Returns a dict with o [T][H][d],
    lse [H][T], owned [T] (rows of some request), absv (like o), sqk and keys (like lse)."""
    T, H, d = q.shape
    pages, page, Hkv, _ = k_pool.shape
    B, width = table.shape
    scale = scale if scale > 0 else 1.0 / np.sqrt(d)
    G = H // Hkv
    out = {"o": np.zeros((T, H, d)), "lse": np.zeros((H, T)), "owned": np.zeros(T, dtype=bool), "absv": np.zeros((T, H, d)),
           "sqk": np.zeros((H, T)), "keys": np.zeros((H, T))}
    for b in range(B):
        r0 = min(max(int(cu_q[b]), 0), T)
        n = max(0, min(int(cu_q[b + 1]), T) - r0)
        kv = max(0, int(kv_lens[b]))
        pos = np.arange(min(kv, width * page))
        entry = table[b, pos // page] if len(pos) else np.zeros(0, dtype=np.int64)
        pos = pos[(entry >= 0) & (entry < pages)]
        entry = entry[(entry >= 0) & (entry < pages)]
        k, v = k_pool[entry, pos % page], v_pool[entry, pos % page]
        for t in range(n):
            row = r0 + t
            out["owned"][row] = True
            ok = permitted(kv - n + t, pos, causal, window)
            for h in range(H):
                kk, vv = k[ok, h // G], v[ok, h // G]
                if len(kk) == 0:
                    out["lse"][h, row] = -np.inf
                    continue
                s = kk @ q[row, h] * scale
                m = s.max()
                e = np.exp(s - m)
                out["lse"][h, row] = m + np.log(e.sum())
                out["o"][row, h] = (e @ vv) / e.sum()
                out["absv"][row, h] = (e @ np.abs(vv)) / e.sum()
                out["sqk"][h, row] = (np.abs(kk) @ np.abs(q[row, h])).max() * scale
                out["keys"][h, row] = len(kk)
    return out
