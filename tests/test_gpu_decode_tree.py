"""attn_decode_paged_tree against the definition in float64. Tolerances are those
of parity.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle
import workloads as W
from masked_cases import cache_inputs, i32, masked_ref, row_keys
from parity import check_lse, check_lse_nonfinite, check_nonfinite, check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def tree(n, seed, kind="tree"):
    """[n, n] bool: which draft sees which."""
    rng = np.random.default_rng(seed)
    if kind == "random":
        return rng.random((n, n)) < 0.3
    seen = np.eye(n, dtype=bool)
    for i in range(n):
        p = i - 1 if kind == "chain" else int(rng.integers(-1, i)) if i else -1
        if p >= 0:
            seen[i] |= seen[p]
    return seen


def pack(blocks, words):
    """Rows' masks [n, n] as int32 words [total, words]."""
    out = []
    for m in blocks:
        bits = np.zeros((m.shape[0], words * 32), np.uint8)
        bits[:, :m.shape[1]] = m
        out.append(np.packbits(bits, axis=1, bitorder="little").view("<u4"))
    x = np.concatenate(out) if out else np.zeros((0, words), np.uint32)
    return torch.from_numpy(x.view(np.int32).copy())


class Case:
    """Rows of `old` keys and `new` drafts (CPU)."""

    def __init__(self, old, new, h_kv, g, d, seed, kind="tree", qk_mult=1.0, words=None):
        self.new, self.lens = list(new), [a + b for a, b in zip(old, new)]
        self.table, self.k, self.v = cache_inputs(self.lens, h_kv, d, seed, qk_mult)
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.q = W.normal((self.cu[-1], h_kv * g, d), seed * 5 + 1, torch.bfloat16, mult=qk_mult)
        self.seen = [tree(n, seed + b, kind) for b, n in enumerate(new)]
        self.max_q = max(1, max(new))
        self.words = words or (self.max_q + 31) // 32
        self.mask = pack(self.seen, self.words)

    def reference(self, rows=None):
        T, h, d = self.q.shape
        O, L = np.zeros((T, h, d)), np.full((T, h), -np.inf)
        for b in range(len(self.lens)) if rows is None else rows:
            n, m = self.lens[b], self.new[b]
            seen = np.concatenate([np.ones((m, n - m), bool), self.seen[b]], 1)
            s = slice(self.cu[b], self.cu[b + 1])
            O[s], L[s] = masked_ref(oracle.to_f64(self.q[s]), row_keys(self.k, self.table[b], n),
                                    row_keys(self.v, self.table[b], n), seen, d ** -0.5)
        return O, L

    def args(self):
        return [t.cuda() for t in (self.q, self.k, self.v, self.table, i32(self.cu), i32(self.lens), self.mask)]

    def run(self, **kw):
        return attn.attn_decode_paged_tree(*self.args(), self.max_q, **kw)

    def tokens(self, rows):
        return [t for b in rows for t in range(self.cu[b], self.cu[b + 1])]

    def check(self, rows=None, **kw):
        O, L = self.reference(rows)
        o, lse = self.run(**kw)
        at = slice(None) if rows is None else self.tokens(rows)
        check_out(o[at], O[at], torch.bfloat16)
        check_lse(lse[at], L[at])
        assert attn.attn_get_device_error() == 0
        return o, lse


@pytest.mark.parametrize("h_kv,g", [(2, 1), (1, 4), (2, 5), (1, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("draft", [1, 2, 7, 26, 33])
def test_lengths_around_tiles(h_kv, g, d, draft):
    old = [0, 1, 15, 16, 100, 127 - draft if draft < 127 else 0, 128 - draft, 128, 129, 255, 400]
    Case(old, [draft] * len(old), h_kv, g, d, seed=draft + g + d).check()


@pytest.mark.parametrize("g,draft", [(4, 31), (4, 32), (4, 33), (4, 63), (4, 64), (4, 65), (4, 130), (5, 25), (5, 26), (5, 51),
                                     (1, 127), (1, 128), (1, 129), (1, 257), (3, 86), (128, 1), (128, 3), (100, 2), (16, 9)])
def test_row_blocks(g, draft):
    """Query rows at and around one tile, a block of two, several blocks."""
    Case([300, 10, 0], [draft, 1, max(1, draft // 2)], 1, g, 64, seed=g + draft).check()


@pytest.mark.parametrize("kind", ["chain", "random", "tree"])
def test_mask_kinds_and_wide_masks(kind):
    Case([40, 90, 0, 33], [70, 33, 100, 0], 2, 4, 128, seed=3, kind=kind, words=9).check()


def test_chain_equals_causal_prefill():
    c = Case([100, 3, 0], [40, 17, 5], 2, 4, 128, seed=4, kind="chain")
    o, lse = c.run()
    q, k, v, table, cu, n, _ = c.args()
    o2, lse2 = attn.attn_prefill_paged(q, k, v, table, cu, n, 40, True)
    assert ((o.float() - o2.float()).abs() <= 4e-3 + o2.float().abs() * 2.0 ** -7).all()
    assert (lse - lse2).abs().max() <= 2e-4


@pytest.mark.parametrize("B,old,draft,h_kv,d", [(1, 32768, 26, 8, 128), (2, 20000, 64, 3, 128), (64, 2000, 24, 8, 64),
                                               (300, 60, 5, 8, 128), (3, 9000, 200, 2, 64)])
def test_batches_cut_over_the_gpu(B, old, draft, h_kv, d):
    g = torch.Generator().manual_seed(B)
    olds = torch.randint(0, old + 1, (B,), generator=g).tolist()
    olds[-1] = old
    news = torch.randint(0, draft + 1, (B,), generator=g).tolist()
    news[-1] = draft
    c = Case(olds, news, h_kv, 4, d, seed=B)
    rows = sorted({0, B // 3, B // 2, B - 1})
    o, lse = c.check(rows)
    again, lse2 = c.run()
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B", [31, 32, 33])
def test_rows_around_a_warps_lanes(B):
    """At most 32 rows are planned by one warp, a row a lane."""
    g = torch.Generator().manual_seed(B)
    olds = torch.randint(0, 900, (B,), generator=g).tolist()
    news = torch.randint(0, 12, (B,), generator=g).tolist()
    news[-1], olds[-1] = 9, 700
    Case(olds, news, 2, 4, 128, seed=B).check()


def test_many_rows():
    """More rows than a CTA has threads; most without a draft."""
    B = 1000
    c = Case([i % 40 for i in range(B)], [1 if i % 7 == 0 else 0 for i in range(B)], 2, 4, 64, seed=5)
    c.check([0, 7, 497, 994])


def test_tokens_that_see_nothing():
    c = Case([0, 0, 20], [6, 40, 3], 2, 4, 128, seed=6)
    for m in c.seen:
        m[::2] = False  # every other draft sees no draft
    c.mask = pack(c.seen, c.words)
    o, lse = c.check()
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_bits_behind_the_drafts_are_ignored():
    c = Case([20, 130], [6, 40], 2, 4, 64, seed=7, words=3)
    O, L = c.reference()
    for b, n in enumerate(c.new):
        for t in range(c.cu[b], c.cu[b + 1]):
            for w in range(3):
                c.mask[t, w] |= -1 if w * 32 >= n else -1 << (n - w * 32) if n - w * 32 < 32 else 0
    o, lse = c.run()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_outliers_force_the_reference_up():
    """One key that outweighs the rest: in the context's middle, its last tile,
    among the drafts; logits of standard deviation 9 elsewhere."""
    for j in (300, 880, 905):
        c = Case([900, 900], [30, 60], 2, 4, 128, seed=8, qk_mult=3.0)
        c.k[int(c.table[0, j // 16]), j % 16] = (c.q[3].view(2, 4, 128)[:, 0] * 2).to(torch.bfloat16)
        c.check()


@pytest.mark.parametrize("mult", [1e5, 2.0 ** -20, 2.0 ** 60])
def test_value_magnitudes(mult):
    c = Case([400, 33], [20, 40], 1, 4, 128, seed=9)
    c.v = (c.v.float() * mult).to(torch.bfloat16)
    O, L = c.reference()
    o, lse = c.run()
    check_out((o.double() / mult).cpu(), O / mult, torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("exp", [10, 21, 30, 100])
def test_large_logits(exp):
    """One key leads by 2^(exp - 3) or more: the row is that key's value."""
    c = Case([700, 20], [20, 40], 2, 4, 64, seed=10)
    c.q.zero_()
    c.q[:, :, 0] = 2.0 ** exp
    c.k.zero_()
    c.k[..., 0] = torch.randint(-8, 8, c.k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for b, j in ((0, 650), (1, 3)):
        c.k[int(c.table[b, j // 16]), j % 16, :, 0] = 8
    O, L = c.reference()
    o, lse = c.run()
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()


def put(c, cache, b, j, value, kv=slice(None), e=slice(None)):
    cache[int(c.table[b, j // 16]), j % 16, kv, e] = value


def test_slots_past_the_lengths_never_reach_a_row():
    c = Case([133, 1, 250], [10, 3, 40], 2, 4, 128, seed=11)
    O, L = c.reference()
    for b, n in enumerate(c.lens):
        for j in range(n, (n + 15) // 16 * 16):
            put(c, c.k, b, j, float("nan"))
            put(c, c.v, b, j, float("nan" if j % 2 else "inf"))
    o, lse = c.run()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("old", [[0, 100], [120, 1000], [250, 20000]])
@pytest.mark.parametrize("draft", [9, 40, 70])
def test_nonfinite_drafts_reach_the_tokens_that_see_them_alone(old, draft):
    c = Case(old, [draft] * 2, 2, 4, 64, seed=12)
    c.seen[0][0] = False  # a token of row 0 that sees nothing of the tree
    c.mask = pack(c.seen, c.words)
    for b, i, e, x in ((0, 3, 5, "nan"), (0, draft - 1, 63, "inf"), (1, 2, 0, "-inf"), (1, 5, 33, "nan")):
        put(c, c.v, b, old[b] + i, float(x), kv=1, e=e)
    put(c, c.k, 0, old[0] + 4, float("nan"), kv=0, e=7)
    put(c, c.k, 1, old[1] + 1, float("inf"), kv=0, e=7)
    with np.errstate(invalid="ignore"):
        O, L = c.reference()
    o, lse = c.run()
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)
    assert attn.attn_get_device_error() == 0


def test_nonfinite_keys_and_values_of_the_context():
    c = Case([200, 300], [20, 33], 2, 2, 64, seed=13)
    put(c, c.v, 0, 50, float("nan"), kv=1, e=5)
    put(c, c.k, 1, 290, float("nan"), kv=0, e=0)
    put(c, c.v, 1, 299, float("inf"), kv=1, e=9)  # in the drafts' tile
    with np.errstate(invalid="ignore"):
        O, L = c.reference()
    o, lse = c.run()
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)


def test_bad_pages_lengths_and_offsets_are_flagged():
    c = Case([150, 60, 20], [10, 4, 5], 2, 4, 128, seed=14)
    attn.attn_get_device_error()
    q, k, v, table, cu, n, mask = c.args()
    bad = table.clone()
    bad[0, 1], bad[1, 3] = k.shape[0], -7
    o, lse = attn.attn_decode_paged_tree(q, k, v, bad, cu, n, mask, c.max_q)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    z = c.k.shape[0]
    kept = c.k, c.v, c.table
    c.k, c.v = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (c.k, c.v))
    c.table = c.table.clone()
    c.table[0, 1] = c.table[1, 3] = z
    O, L = c.reference()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    c.k, c.v, c.table = kept
    O, L = c.reference()
    cap = table.shape[1] * 16
    for lens, offs, skipped in (([cap + 1, 64, 25], c.cu, [0]), ([160, 3, 25], c.cu, [1]),  # clamped: other keys
                                ([160, 64, 25], [0, 10, 9, 9], [1, 2]), ([160, 64, 25], [-1, 10, 14, 19], [0]),
                                ([160, 64, 25], [0, 10, 14, 20], [2]), ([160, 64, 25], [0, 10, 14, 2 ** 31 - 1], [2])):
        o = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        attn.attn_decode_paged_tree(q, k, v, table, i32(offs).cuda(), i32(lens).cuda(), mask, c.max_q, o=o, lse=lse)
        assert attn.attn_get_device_error() & attn.ATTN_DEVERR_BAD_SEQ_LEN, (lens, offs)
        for b in range(3):
            s = slice(c.cu[b], c.cu[b + 1])
            if b not in skipped:
                check_out(o[s], O[s], torch.bfloat16)
            elif offs != c.cu:
                assert (o[s] == 7).all() and (lse[s] == 7).all()
    # More drafts in a row than the call allows for: the row is left out.
    o = torch.full_like(q, 7.0)
    attn.attn_decode_paged_tree(q, k, v, table, cu, n, mask, 9, o=o)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    assert (o[:10] == 7).all()
    check_out(o[10:], O[10:], torch.bfloat16)


def test_outputs_and_workspace_stay_in_bounds():
    for old, new in (([5, 0, 3000], [3, 9, 40]), ([40] * 70, [5] * 70)):
        c = Case(old, new, 2, 4, 128, seed=15)
        O, L = c.reference()
        T, h, d = c.q.shape
        need = attn.attn_decode_tree_workspace_bytes(len(old), h, 2, d)
        ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")  # NaN where not written
        buf = torch.full((T * h * d + 2048,), float("nan"), dtype=torch.bfloat16, device="cuda")
        o = buf[1024:-1024].view(T, h, d)
        lbuf = torch.full((T * h + 8,), 7.0, device="cuda")
        lse = lbuf[4:-4].view(T, h)
        c.run(workspace=ws[:need], o=o, lse=lse)
        torch.cuda.synchronize()
        assert torch.isnan(buf[:1024].float()).all() and torch.isnan(buf[-1024:].float()).all()
        assert (lbuf[:4] == 7).all() and (lbuf[-4:] == 7).all() and (ws[need:] == 0xff).all()
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
        o2, none = c.run(return_lse=False)
        assert none is None and torch.equal(o, o2)


def test_tokens_outside_the_rows_are_left_as_they_are():
    """A padded batch: tokens in front of the first row and behind the last."""
    c = Case([40, 300], [6, 12], 2, 4, 64, seed=16)
    O, L = c.reference()
    q, k, v, table, cu, n, mask = c.args()
    pad = lambda x, a, b: torch.cat([x.new_full((a, *x.shape[1:]), 3), x, x.new_full((b, *x.shape[1:]), 3)])
    o, lse = torch.full((28, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((28, 8), 7.0, device="cuda")
    attn.attn_decode_paged_tree(pad(q, 3, 7), k, v, table, cu + 3, n, pad(mask, 3, 7), c.max_q, o=o, lse=lse)
    check_out(o[3:21], O, torch.bfloat16)
    check_lse(lse[3:21], L)
    for x in (o, lse):
        assert (x[:3] == 7).all() and (x[21:] == 7).all()


def test_captured_and_replayed_with_new_trees():
    c = Case([700, 100, 300], [20, 20, 20], 2, 4, 128, seed=17, words=2)
    q, k, v, table, cu, n, mask = c.args()
    ws = torch.empty(attn.attn_decode_tree_workspace_bytes(3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((60, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.attn_decode_paged_tree(q, k, v, table, cu, n, mask, 40, workspace=ws, o=o, lse=lse)
    for new, lens in (([20, 20, 20], c.lens), ([1, 0, 33], [1, 77, 320]), ([40, 9, 11], [720, 9, 100])):
        c.new, c.lens = new, lens
        c.cu = [0, new[0], new[0] + new[1], sum(new)]
        c.seen = [tree(m, 50 + m) for m in new]
        part = pack(c.seen, c.words)
        mask[:part.shape[0]] = part.cuda()
        cu.copy_(i32(c.cu))
        n.copy_(i32(lens))
        o.fill_(7.0)
        graph.replay()
        O, L = c.reference()
        T = c.cu[-1]
        check_out(o[:T], O[:T], torch.bfloat16)
        check_lse(lse[:T], L[:T])
        assert (o[T:] == 7).all()
    assert attn.attn_get_device_error() == 0


def test_two_streams_at_once():
    a, b = Case([3000] * 5, [10] * 5, 2, 4, 128, seed=18), Case([300] * 50, [40] * 50, 2, 4, 128, seed=19)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    args_a, args_b = a.args(), b.args()
    torch.cuda.synchronize()
    got = [(attn.attn_decode_paged_tree(*args_a, a.max_q, stream=s1), attn.attn_decode_paged_tree(*args_b, b.max_q, stream=s2))
           for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(y[0], want[1][0])


def test_far_pages_beyond_32_bit_offsets():
    nb, h_kv, d = 140000, 8, 128
    assert nb * h_kv * 16 * d > 2 ** 31
    c = Case([40, 20], [10, 3], h_kv, 4, d, seed=20)
    q, k, v, table, cu, n, mask = c.args()
    far_k = torch.empty((nb, 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
    far_v = torch.empty_like(far_k)
    for page in range(k.shape[0]):
        far_k[nb - 1 - page] = k[page]
        far_v[nb - 1 - page] = v[page]
    O, L = c.reference()
    o, lse = attn.attn_decode_paged_tree(q, far_k, far_v, torch.where(table < 0, table, nb - 1 - table), cu, n, mask, c.max_q)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


def test_inputs_rewritten_just_before():
    """The kernel in front lets the call start at once and rewrites one of offsets,
    lengths, table and mask 50 us later."""
    c = Case([200, 0, 33], [10, 20, 3], 2, 4, 128, seed=21)
    O, L = c.reference()
    dev = c.args()
    for i in (3, 4, 5, 6):
        old = torch.zeros_like(dev[i])
        now = dev[:i] + [old] + dev[i + 1:]
        attn.attn_decode_paged_tree(*now, c.max_q)  # warm: lines of the old contents
        attn.attn_selftest_delayed_copy(old.view(-1), dev[i].view(-1), delay_us=50)
        o, lse = attn.attn_decode_paged_tree(*now, c.max_q)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
    attn.attn_get_device_error()  # (the warm calls' rows may be shorter than their drafts)


def test_a_speculating_loop():
    """Drafts' keys enter the cache behind the context, the tree is verified, the
    accepted path is moved up, and the next step's context holds it: each step is the
    definition over the accepted tokens and the tree."""
    h_kv, g, d, steps, n = 2, 4, 128, 6, 12
    k = torch.zeros((20, 16, h_kv, d), dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None]
    slot = lambda p: (int(table[0, p // 16]), p % 16)
    rng, ctx = np.random.default_rng(2), 0
    for step in range(steps):
        c = Case([ctx], [n], h_kv, g, d, seed=30 + step)
        kv = W.normal((n, 2, h_kv, d), 60 + step, torch.bfloat16)
        for i in range(n):
            k[slot(ctx + i)], v[slot(ctx + i)] = kv[i, 0], kv[i, 1]
        c.k, c.v, c.table = k, v, table
        c.check()
        path = np.nonzero(c.seen[0][int(rng.integers(n))])[0]  # a token and its ancestors
        for to, i in enumerate(path):
            k[slot(ctx + to)], v[slot(ctx + to)] = kv[i, 0], kv[i, 1]
        ctx += len(path)


def test_binding_refuses():
    c = Case([3, 20], [4, 5], 2, 4, 64, seed=22)
    q, k, v, table, cu, n, mask = c.args()
    good = dict(q=q, k_cache=k, v_cache=v, block_table=table, cu_seqlens_q=cu, seq_lens=n, tree_mask=mask, max_q_len=5)
    attn.attn_decode_paged_tree(**good)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=k.float()), dict(v_cache=v[:1]), dict(k_cache=k[..., :32]),
               dict(block_table=table[:1]), dict(block_table=table.long()), dict(cu_seqlens_q=cu[:2]), dict(seq_lens=n[:1]),
               dict(seq_lens=n.cpu()), dict(tree_mask=mask[:3]), dict(tree_mask=mask.long()), dict(tree_mask=mask[:, 0]),
               dict(o=q.float()), dict(lse=torch.empty((2, 9), device="cuda"))):
        with pytest.raises(ValueError):
            attn.attn_decode_paged_tree(**{**good, **kw})
    for kw in (dict(max_q_len=0), dict(max_q_len=33), dict(scale=-1.0),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(attn.AttnError):
            attn.attn_decode_paged_tree(**{**good, **kw})
    assert attn.attn_get_device_error() == 0
