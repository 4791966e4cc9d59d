"""Absorbed attention of a chunk of new tokens over a paged cache, in float64,
one sequence and one head at a time, from the definition."""
import numpy as np


def visible(n, cached, i, mask_row):
    """Positions that new token i of n sees."""
    new = [m for m in range(n) if (m <= i if mask_row is None else mask_row >> m & 1)]
    return np.concatenate([np.arange(cached), cached + np.array(new, dtype=int)]).astype(int)


def chunk_attention(q, kv, table, page_size, w_uk, w_uv, iro, cached, scale, mask=None, sink=None):
    """(out, lse, slack): rows of tokens outside every sequence are NaN.

    kv: [rows][576] cache rows; mask: for every token a whole number whose bit m
    is new token m, or None for causal; slack bounds |error of a score| per unit
    of relative error in the projected query: scale * sum |q_lat c|, the largest
    over the row's keys."""
    T, H = q.shape[:2]
    out, lse = np.full((T, H, 128), np.nan), np.full((T, H), np.nan)
    slack = np.zeros((T, H))
    for b in range(len(cached)):
        a, n = int(iro[b]), int(iro[b + 1]) - int(iro[b])
        j = np.arange(cached[b] + n)
        c = kv[table[b, j // page_size] * page_size + j % page_size]
        for i in range(n):
            see = visible(n, cached[b], i, None if mask is None else mask[a + i])
            for h in range(H):
                lat = w_uk[h] @ q[a + i, h, :128]
                s = scale * (c[see, :512] @ lat + c[see, 512:] @ q[a + i, h, 128:])
                slack[a + i, h] = scale * (np.abs(c[see, :512]) @ np.abs(lat)).max(initial=0.0)
                extra = -np.inf if sink is None else sink[b]
                top = max(s.max(initial=-np.inf), extra)
                if top == -np.inf:
                    out[a + i, h], lse[a + i, h] = 0.0, -np.inf
                    continue
                e = np.exp(s - top)
                total = e.sum() + np.exp(extra - top)
                out[a + i, h] = w_uv[h] @ (e @ c[see, :512] / total)
                lse[a + i, h] = top + np.log(total)
    return out, lse, slack
