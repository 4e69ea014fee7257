"""Paged KV cache and attention, in float64.
TEST INFRASTRUCTURE ONLY (see oracle/__init__.py for the page key).

The pages keep the attention layers' KV cache in FP8 ([P1] 접근 방법) and say
nothing of its layout; block tables, slots and the attention itself follow
their textbook definitions:

  * request r with cached_r tokens held and new_r added fills the pages
    0 .. ceil((cached_r + new_r) / page) - 1 of its row of the block table;
    those from ceil(cached_r / page) on come from the free list, requests in
    order; the token at position p has slot table[p // page] * page + p % page;
  * a token at position p sees the keys j < length, j <= p if causal,
    j > p - window if a window is set, and its output is
    sum_j softmax_j(scale q.k_j) v_j, zero if it sees none.
"""
import numpy as np


def page_tables(new, cached, table, free, page, n_tokens):
    """(table, cu, kv, positions, slots, used) by plain loops."""
    table = np.array(table, dtype=np.int64)
    cols = table.shape[1]
    cu, kv, positions, slots, used = [0], [], [], [], 0
    for r, (n, c) in enumerate(zip(new, cached)):
        n, c = max(int(n), 0), max(int(c), 0)
        kv.append(n + c)
        cu.append(cu[-1] + n)
        for b in range(-(-c // page), min(-(-(c + n) // page), cols)):
            table[r, b] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            positions.append(p)
            b = p // page
            held = table[r, b] if b < cols else -1
            slots.append(held * page + p % page if held >= 0 else -1)
    pad = n_tokens - len(positions)
    return (table, np.array(cu), np.array(kv), np.array(positions + [-1] * pad, dtype=np.int64),
            np.array(slots + [-1] * pad, dtype=np.int64), used)


def attention(q, k, v, scale, causal=True, window=0):
    """One request: q [new, heads, d] at the last positions of k, v
    [length, kv_heads, d].  Returns (o, mean_abs, reach): the output, the
    weighted mean of |v| of each output element, and for each row and head
    the largest scale * sum |q_i k_i| over the keys it sees (what bounds the
    rounding of its scores)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    new, heads, d = q.shape
    length, kv_heads, _ = k.shape
    o = np.zeros((new, heads, d))
    mean_abs, reach = np.zeros((new, heads, d)), np.zeros((new, heads))
    for i in range(new):
        p = length - new + i
        hi = min(length, p + 1) if causal else length
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(heads):
            g = h // (heads // kv_heads)
            s = scale * (k[lo:hi, g] @ q[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            o[i, h] = w @ v[lo:hi, g]
            mean_abs[i, h] = w @ np.abs(v[lo:hi, g])
            reach[i, h] = scale * (np.abs(k[lo:hi, g]) @ np.abs(q[i, h])).max()
    return o, mean_abs, reach
