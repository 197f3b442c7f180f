"""Values that carry their position, for caches whose rows are cut into many parts.

Page p of a row (in the order of its keys) has a_p > 0 in column p mod d and 0 in the
others, a_p one of 8 numbers in [1, 2). Every output is then the weight of the few
pages of its column, times a_p: with n pages a row, n / d of them, each a share of about
d / n of the output. A page or a partial state that is lost, counted twice or joined
with another's weight moves its column's output by that share, 3 % for 4400 pages of
128 columns, against an error bound of 2^-8 + 2^-11 + 2^-13 = 0.45 % of it. (With
values from N(0, 1) a whole key tile of 40000 keys is within 2e-3 of nothing.)"""
import numpy as np
import torch

BOUND = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13


def page_values(n_pages, d, first=0):
    """[n_pages, d] float64 rows for pages first, first + 1, ... of a row."""
    p = np.arange(first, first + n_pages)
    x = np.zeros((n_pages, d))
    x[np.arange(n_pages), p % d] = 1.0 + ((p * 5 + p // d * 3) % 8) / 8.0
    return x


def check(o, O):
    """The output's rounding (2^-8), a weight's (one fp16 number, 2^-11) and what is
    done in 32 bits (2^-13); every product is positive, so the sum of magnitudes is
    the output itself. A column without a page is 0 exactly."""
    err = np.abs(np.asarray(o, np.float64) - O)
    assert (err <= BOUND * O).all(), (float((err / np.maximum(O, 1e-30)).max()), int((err > BOUND * O).sum()))


def shared_case(prefix, lens, h_kv, g, d, seed):
    """case() of test_gpu_decode_shared with page values: the prefix's pages, then a
    row's own."""
    from test_gpu_decode_shared import case

    args = case(prefix, lens, h_kv, g, d, seed)
    v, ptab, tab = args[2], args[3], args[5]
    v.zero_()

    def put(pages, n, first):
        x = torch.from_numpy(page_values(n, d, first)).to(torch.bfloat16)
        v[pages[:n].long()] = x[:, None, None, :].expand(n, 16, h_kv, d)

    n = (prefix + 15) // 16
    put(ptab, n, 0)
    for b, length in enumerate(lens):
        put(tab[b], (length + 15) // 16, n)
    return args


def e4m3_case(lens, h_kv, g, d, seed):
    """decode_case() of e4m3_cases with page values (numbers of four bits: stored as
    they are)."""
    from e4m3_cases import cache_from, decode_case

    q, kc, vc, ks, vs, table, n = decode_case(lens, h_kv, g, d, seed)
    v64 = np.zeros((vc.shape[0], h_kv, 16, d))
    for b, length in enumerate(lens):
        k = (length + 15) // 16
        v64[table[b, :k].long().numpy()] = page_values(k, d)[:, None, None, :]
    vc, vs = cache_from(v64)
    return q, kc, vc, ks, vs, table, n


SHARED = [(20000, [100, 1000], 8, 4, 128), (40000, [0, 17, 3000], 1, 4, 128), (9000, [100 + 37 * i % 900 for i in range(70)], 3, 4, 64),
          (0, [30000, 16], 2, 4, 128), (12000, [500 * (i % 3) for i in range(40)], 2, 8, 128)]
E4M3 = [([70000], 2, 4, 128), ([70000], 1, 8, 64), ([5000], 2, 4, 128), ([100, 0, 9000] * 7, 2, 4, 128), ([33000, 20000, 1], 2, 5, 64)]
