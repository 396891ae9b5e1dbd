"""Plain models of the paged cache calls, row by row and in 64 bits."""

from __future__ import annotations

import numpy as np


def tables_model(want, lens, table, free, page, n_pages, max_tokens):
    """dv_page_tables, one request after another (`free`: the stack's free entries)."""
    W = len(table[0])
    pages = lambda n: -(-n // page)  # noqa: E731
    table, stack, lens = [list(r) for r in table], list(free), list(lens)
    fits = [w <= W * page and 0 <= n <= W * page for w, n in zip(want, lens)]
    for r, w in enumerate(want):
        if fits[r] and 0 <= w < lens[r]:
            stack += table[r][pages(w):pages(lens[r])]
    avail, need_sum, tok_sum = len(stack), 0, 0
    top, offsets, slots, granted, new = avail, [0], [], [], []
    for r, w in enumerate(want):
        n, ok, goal = lens[r], fits[r], lens[r]
        if ok and w >= 0:
            goal = w
            need, add = max(0, pages(w) - pages(n)), max(0, w - n)
            need_sum, tok_sum = need_sum + need, tok_sum + add
            ok = (need == 0 or need_sum <= avail) and (add == 0 or tok_sum <= max_tokens)
            if not ok:
                goal = n
        granted.append(int(ok))
        new.append(goal)
        for p in range(pages(n), pages(goal)):
            top -= 1
            table[r][p] = stack[top]
        for pos in range(n, goal):
            slots.append(table[r][pos // page] * page + pos % page)
        offsets.append(len(slots))
    return dict(lens=new, table=table, stack=stack, free_count=top, granted=granted, offsets=offsets,
                slots=slots + [-1] * (max_tokens - len(slots)))


def attn_model(q, K, V, table, lens, scale, heads=None):
    """Softmax attention of q [B][rows][dh] (float64) over each row's pages:
    (out, lse, bound) with bound the largest |scale| sum |q| |k| of any score,
    which the rounding of the scores goes by."""
    B, rows, dh = q.shape
    page = K.shape[2]
    heads = list(range(K.shape[1])) if heads is None else list(heads)
    G = rows // len(heads)
    out, lse, bound = np.zeros(q.shape), np.full((B, rows), -np.inf), 0.0
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pages = [int(p) for p in table[b][: -(-n // page)]]
        for j, i in enumerate(heads):
            k = np.concatenate([K[p, i] for p in pages])[:n]
            v = np.concatenate([V[p, i] for p in pages])[:n]
            for r in range(j * G, (j + 1) * G):
                z = scale * (k @ q[b, r])
                bound = max(bound, abs(scale) * float(np.max(np.abs(k) @ np.abs(q[b, r]))))
                m = z.max()
                e = np.exp(z - m)
                out[b, r] = (e @ v) / e.sum()
                lse[b, r] = m + np.log(e.sum())
    return out, lse, bound
