"""References and layouts shared by the tests of attention with a window or a
tree mask: the definition in float64 over an explicit table of which query sees
which key."""
import numpy as np
import torch

import oracle
import workloads as W


def window_seen(n_q, n, window, sinks):
    """[n_q, n] bool: queries at the last n_q of n positions."""
    p = np.arange(n - n_q, n)[:, None]
    j = np.arange(n)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def masked_ref(q, k, v, seen, scale):
    """q [n_q, h, d], k and v [n, h_kv, d] (float64), seen [n_q, n]: outputs
    [n_q, h, d] and log-sum-exps [n_q, h]. A key that is not seen takes no part,
    whatever it and its value hold; a query that sees none gives 0 and -inf."""
    n_q, h, d = q.shape
    g = h // k.shape[1]
    O, L = np.zeros((n_q, h, d)), np.full((n_q, h), -np.inf)
    if k.shape[0] == 0:
        return O, L
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if np.isfinite(k).all() and np.isfinite(v).all() and np.isfinite(q).all():
            for hq in range(h):
                s = np.where(seen, q[:, hq] @ k[:, hq // g].T * scale, -np.inf)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - np.where(np.isinf(m), 0.0, m))
                l = p.sum(-1, keepdims=True)
                O[:, hq] = (p @ v[:, hq // g]) / np.where(l == 0, 1.0, l)
                L[:, hq] = np.where(l == 0, -np.inf, m + np.log(np.where(l == 0, 1.0, l)))[:, 0]
        else:  # a query at a time over the keys it sees
            for i in range(n_q):
                at = np.nonzero(seen[i])[0]
                if len(at):
                    o, l = oracle.attention_ref(q[i][:, None], k[at].transpose(1, 0, 2), v[at].transpose(1, 0, 2), scale)
                    O[i], L[i] = o[:, 0], l[:, 0]
    return O, L


def row_keys(cache, table_row, n):
    """The first n keys of a row of a bf16 cache in float64, [n, h_kv, d]; pages
    without an entry read as NaN."""
    pages = table_row[:(n + 15) // 16].long()
    out = (pages < 0) | (pages >= cache.shape[0])
    x = oracle.to_f64(cache[torch.where(out, 0, pages)])
    x[out.numpy()] = np.nan
    return x.reshape(-1, *cache.shape[2:])[:n]


def hide_pages(table, lens, n_qs, window, sinks, value=-1):
    """Table without entries for the pages that no query of a row sees."""
    t = table.clone()
    for b, (n, m) in enumerate(zip(lens, n_qs)):
        first = n - m + 1 - window
        for p in range(t.shape[1]):
            if (p + 1) * 16 <= first and p * 16 >= sinks or p * 16 >= n:
                t[b, p] = value
    return t


def cache_inputs(lens, h_kv, d, seed, qk_mult=1.0):
    """Table and bf16 caches for rows of the given lengths (CPU)."""
    table, nb = W.paged_layout(list(lens), seed, spare_pages=2)
    k = W.normal((nb, 16, h_kv, d), seed * 5 + 2, torch.bfloat16, mult=qk_mult)
    v = W.normal((nb, 16, h_kv, d), seed * 5 + 3, torch.bfloat16)
    return table, k, v


def i32(x):
    return torch.tensor(x, dtype=torch.int32)
