"""attn_prefill_paged_window against the definition in float64. Tolerances are
those of parity.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle
import workloads as W
from masked_cases import cache_inputs, hide_pages, i32, masked_ref, row_keys, window_seen
from parity import check_lse, check_lse_nonfinite, check_nonfinite, check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


class Case:
    """Rows of `old` keys and `new` queries (CPU); pages out of sight have no entry."""

    def __init__(self, old, new, h_kv, g, d, seed, window, sinks, qk_mult=1.0, hide=True):
        self.new, self.lens = list(new), [a + b for a, b in zip(old, new)]
        self.window, self.sinks = window, sinks
        self.table, self.k, self.v = cache_inputs(self.lens, h_kv, d, seed, qk_mult)
        if hide:
            self.table = hide_pages(self.table, self.lens, self.new, window, sinks)
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.q = W.normal((self.cu[-1], h_kv * g, d), seed * 5 + 1, torch.bfloat16, mult=qk_mult)
        self.max_q = max(1, max(new))

    def reference(self, rows=None):
        T, h, d = self.q.shape
        O, L = np.zeros((T, h, d)), np.full((T, h), -np.inf)
        for b in range(len(self.lens)) if rows is None else rows:
            n, m = self.lens[b], self.new[b]
            s = slice(self.cu[b], self.cu[b + 1])
            seen = window_seen(m, n, self.window, self.sinks)
            some = seen.any(0)  # (pages out of sight read as NaN)
            O[s], L[s] = masked_ref(oracle.to_f64(self.q[s]), row_keys(self.k, self.table[b], n)[some],
                                    row_keys(self.v, self.table[b], n)[some], seen[:, some], d ** -0.5)
        return O, L

    def args(self):
        return [t.cuda() for t in (self.q, self.k, self.v, self.table, i32(self.cu), i32(self.lens))]

    def run(self, **kw):
        return attn.attn_prefill_paged_window(*self.args(), self.window, self.sinks, self.max_q, **kw)

    def check(self, rows=None, **kw):
        O, L = self.reference(rows)
        o, lse = self.run(**kw)
        at = slice(None) if rows is None else [t for b in rows for t in range(self.cu[b], self.cu[b + 1])]
        check_out(o[at], O[at], torch.bfloat16)
        check_lse(lse[at], L[at])
        assert attn.attn_get_device_error() == 0
        return o, lse


@pytest.mark.parametrize("h_kv,g", [(2, 1), (1, 4), (1, 3), (2, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (100, 0), (128, 16), (129, 130), (300, 3),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_windows_and_sinks(h_kv, g, d, window, sinks):
    Case([0, 3, 128, 500, 40, 255], [1, 128, 129, 60, 300, 0], h_kv, g, d, window % 97 + sinks % 89, window, sinks).check()


@pytest.mark.parametrize("sinks", [0, 1, 127, 128, 129, 400])
@pytest.mark.parametrize("window", [1, 127, 128, 129, 255, 256, 257])
def test_bounds_around_tiles(window, sinks):
    Case([0, 640, 513], [400, 130, 257], 1, 2, 64, 3, window, sinks).check()


def test_window_beyond_the_rows_is_causal_prefill():
    c = Case([100, 3, 0], [140, 17, 300], 2, 4, 128, 4, 10 ** 6, 0)
    o, lse = c.run()
    o2, lse2 = attn.attn_prefill_paged(*c.args(), c.max_q, True, decode_splits=0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("old,new,window,sinks", [([0], [5000], 1024, 4), ([3000, 9000, 100], [600, 257, 33], 2000, 0),
                                                  ([700] * 40, [70] * 40, 333, 20)])
def test_long_rows(old, new, window, sinks):
    c = Case(old, new, 2, 4, 128, 5, window, sinks)
    o, lse = c.check([0] if len(old) == 1 else [1, len(old) - 1])
    again, lse2 = c.run()
    assert torch.equal(o, again) and torch.equal(lse, lse2)


def test_outliers_force_the_reference_up():
    for j in (2, 150, 290):  # a sink, inside the windows, a late key
        c = Case([100], [200], 2, 4, 128, 6, 90, 5, qk_mult=3.0)
        c.k[int(c.table[0, j // 16]), j % 16] = (c.q[195].view(2, 4, 128)[:, 0] * 2).to(torch.bfloat16)
        c.check()


@pytest.mark.parametrize("mult", [1e5, 2.0 ** -13, 3e8])
def test_value_magnitudes(mult):
    """Values that fp16 does not hold take the two-term weights, masks included.
    (2^-13: some turn fp16 subnormals, each within 2^-25.)"""
    c = Case([300, 0], [150, 140], 1, 4, 128, 7, 100, 3)
    c.v = (c.v.float() * mult).to(torch.bfloat16)
    O, L = c.reference()
    o, lse = c.run()
    if mult < 1:
        # Half a bf16 step of the output; a weight's 2^-11 twice (fp16, and the sum of
        # unrounded ones) of values below 6 * 2^-13; 2^-25 from the values.
        tol = 2.0 ** -9 * np.abs(O) + 2.0 ** -10 * 6 * mult + 2.0 ** -25
        assert (np.abs(o.double().cpu().numpy() - O) <= tol).all()
    else:
        check_out((o.double() / mult).cpu(), O / mult, torch.bfloat16)
    check_lse(lse, L)


def test_one_large_value_in_an_edge_tile():
    c = Case([200], [200], 2, 2, 64, 8, 130, 4)
    c.v[int(c.table[0, 20]), 3, 1, 7] = 3e5
    O, L = c.reference()
    a = Case([200], [200], 2, 2, 64, 8, 130, 4)
    a.v = c.v.abs()
    o, lse = c.run()
    check_out(o, O, torch.bfloat16, mag=a.reference()[0])
    check_lse(lse, L)


def test_keys_out_of_sight_never_reach_a_query():
    """NaN and infinities in the gap, in the pages where sinks end and windows
    begin, and behind the rows' ends."""
    window, sinks = 90, 5
    c = Case([300, 450, 0], [40, 150, 20], 2, 4, 128, 9, window, sinks, hide=False)
    O, L = c.reference()
    for b, n in enumerate(c.lens):
        some = window_seen(c.new[b], n, window, sinks).any(0)
        for j in range((n + 15) // 16 * 16):
            if j >= n or not some[j]:
                c.k[int(c.table[b, j // 16]), j % 16] = float("nan") if j % 2 else float("inf")
                c.v[int(c.table[b, j // 16]), j % 16] = float("inf") if j % 3 else float("nan")
    o, lse = c.run()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("d,g", [(64, 1), (128, 4)])
@pytest.mark.parametrize("window,sinks", [(60, 3), (200, 0), (130, 140)])
def test_nonfinite_keys_and_values_reach_the_queries_that_see_them_alone(window, sinks, d, g):
    c = Case([100, 300], [260, 140], 2, g, d, 10, window, sinks, hide=False)
    for b, j, e, x in ((0, 1, 5, "nan"), (0, 200, 63, "inf"), (0, 359, 1, "nan"), (0, 128, 9, "nan"), (1, 300, 0, "-inf"),
                       (1, 255, 33, "nan")):
        c.v[int(c.table[b, j // 16]), j % 16, 1, e] = float(x)
    c.v[int(c.table[1, 1]), 3] = 1e6  # a finite value that fp16 does not hold
    c.k[int(c.table[0, 15]), 4, 0, 7] = float("nan")
    c.k[int(c.table[1, 20]), 4, 0, 7] = float("inf")
    with np.errstate(invalid="ignore"):
        O, L = c.reference()
    keep = ~np.isfinite(O) | (np.abs(O) < 8)  # (the 1e6 sets its rows' own scale)
    o, lse = c.run()
    o, O = np.where(keep, o.double().cpu().numpy(), 0.0), np.where(keep, O, 0.0)
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)
    assert attn.attn_get_device_error() == 0


def test_only_visible_pages_are_looked_up():
    window, sinks = 50, 20
    c = Case([300, 90], [60, 30], 2, 4, 64, 11, window, sinks)
    want, lse_w = c.run()
    c.table = hide_pages(c.table, c.lens, c.new, window, sinks, value=2 ** 31 - 1)
    o, lse = c.run()
    assert torch.equal(o, want) and torch.equal(lse, lse_w)
    assert attn.attn_get_device_error() == 0
    c.table[0, 1] = -5  # a sink page
    o, lse = c.run()
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    z = c.k.shape[0]
    c.k, c.v = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (c.k, c.v))
    c.table[0, 1] = z
    O, L = c.reference()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_bad_lengths_and_offsets_are_flagged():
    c = Case([150, 60, 20], [10, 4, 5], 2, 4, 128, 12, 70, 3, hide=False)
    O, L = c.reference()
    q, k, v, table, cu, n = c.args()
    cap = table.shape[1] * 16
    for lens, offs, skipped in (([cap + 1, 64, 25], c.cu, [0]), ([160, 3, 25], c.cu, [1]),  # clamped: other keys
                                ([160, 64, 25], [0, 10, 9, 9], [1, 2]), ([160, 64, 25], [-1, 10, 14, 19], [0]),
                                ([160, 64, 25], [0, 10, 14, 20], [2]), ([160, 64, 25], [0, 10, 14, 2 ** 31 - 1], [2])):
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        attn.attn_prefill_paged_window(q, k, v, table, i32(offs).cuda(), i32(lens).cuda(), 70, 3, c.max_q, o=o, lse=lse)
        assert attn.attn_get_device_error() & attn.ATTN_DEVERR_BAD_SEQ_LEN, (lens, offs)
        for b in range(3):
            s = slice(c.cu[b], c.cu[b + 1])
            if b not in skipped:
                check_out(o[s], O[s], torch.bfloat16)
            elif offs != c.cu:
                assert (o[s] == 7).all() and (lse[s] == 7).all()
    o = torch.full_like(q, 7.0)
    attn.attn_prefill_paged_window(q, k, v, table, cu, n, 70, 3, 9, o=o)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    assert (o[:10] == 7).all()
    check_out(o[10:], O[10:], torch.bfloat16)


def test_outputs_and_workspace_stay_in_bounds():
    c = Case([5, 0, 500], [3, 9, 200], 2, 4, 128, 13, 100, 4)
    O, L = c.reference()
    T, h, d = c.q.shape
    need = attn.attn_prefill_window_workspace_bytes(3, c.table.shape[1], 2, d)
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
    c = Case([40, 300], [60, 12], 2, 4, 64, 14, 50, 2)
    O, L = c.reference()
    q, k, v, table, cu, n = c.args()
    pad = lambda x: torch.cat([x.new_full((3, *x.shape[1:]), 3), x, x.new_full((200, *x.shape[1:]), 3)])
    o, lse = torch.full((275, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((275, 8), 7.0, device="cuda")
    attn.attn_prefill_paged_window(pad(q), k, v, table, cu + 3, n, 50, 2, c.max_q, o=o, lse=lse)
    check_out(o[3:75], O, torch.bfloat16)
    check_lse(lse[3:75], L)
    for x in (o, lse):
        assert (x[:3] == 7).all() and (x[75:] == 7).all()


def test_captured_and_replayed_with_new_rows():
    c = Case([700, 100, 300], [100, 200, 20], 2, 4, 128, 15, 130, 4, hide=False)
    q, k, v, table, cu, n = c.args()
    ws = torch.empty(attn.attn_prefill_window_workspace_bytes(3, table.shape[1], 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((320, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.attn_prefill_paged_window(q, k, v, table, cu, n, 130, 4, 300, workspace=ws, o=o, lse=lse)
    for new, lens in (([100, 200, 20], c.lens), ([1, 0, 290], [1, 77, 320]), ([40, 130, 11], [720, 300, 100])):
        c.new, c.lens = new, lens
        c.cu = [0, new[0], new[0] + new[1], sum(new)]
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


def test_inputs_rewritten_just_before():
    """The kernel in front lets the call start at once and rewrites one of q, the
    caches, table, offsets and lengths 50 us later."""
    c = Case([300, 0, 33], [40, 200, 3], 2, 4, 128, seed=22, window=150, sinks=4)
    O, L = c.reference()
    dev = c.args()
    words = lambda t: t.reshape(-1).view(torch.int32)
    for i in range(6):
        old = torch.zeros_like(dev[i])
        now = dev[:i] + [old] + dev[i + 1:]
        attn.attn_prefill_paged_window(*now, 150, 4, c.max_q)  # warm: lines of the old contents
        attn.attn_selftest_delayed_copy(words(old), words(dev[i]), delay_us=50)
        o, lse = attn.attn_prefill_paged_window(*now, 150, 4, c.max_q)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
    attn.attn_get_device_error()  # (the warm calls' rows may be shorter than their queries)


def test_two_streams_at_once():
    a, b = Case([3000], [500], 2, 4, 128, 16, 1000, 4), Case([30] * 20, [40] * 20, 2, 4, 128, 17, 33, 1)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    args_a, args_b = a.args(), b.args()
    torch.cuda.synchronize()
    got = [(attn.attn_prefill_paged_window(*args_a, 1000, 4, 500, stream=s1),
            attn.attn_prefill_paged_window(*args_b, 33, 1, 40, stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(y[0], want[1][0])


def test_far_pages_beyond_32_bit_offsets():
    nb, h_kv, d = 140000, 8, 128
    assert nb * h_kv * 16 * d > 2 ** 31
    c = Case([40, 20], [100, 3], h_kv, 4, d, 18, 60, 4)
    q, k, v, table, cu, n = c.args()
    far_k = torch.empty((nb, 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
    far_v = torch.empty_like(far_k)
    for page in range(k.shape[0]):
        far_k[nb - 1 - page] = k[page]
        far_v[nb - 1 - page] = v[page]
    O, L = c.reference()
    o, lse = attn.attn_prefill_paged_window(q, far_k, far_v, torch.where(table < 0, table, nb - 1 - table), cu, n, 60, 4,
                                            c.max_q)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_prefill_then_decode_steps():
    """A prompt in two chunks, then decode steps, all with one window: every token
    is the definition over the whole sequence. Pages are given back as they leave
    the window."""
    h_kv, g, d, window, sinks, T = 2, 4, 128, 70, 5, 300
    k = W.normal((T, h_kv, d), 1, torch.bfloat16)
    v = W.normal((T, h_kv, d), 2, torch.bfloat16)
    q = W.normal((T, h_kv * g, d), 3, torch.bfloat16)
    kc = torch.full((30, 16, h_kv, d), float("nan"), dtype=torch.bfloat16)
    vc = torch.full_like(kc, float("nan"))
    table = torch.full((1, 20), -1, dtype=torch.int32)
    free, outs, at = list(range(29, -1, -1)), [], 0
    for n in [150, 100] + [1] * 50:
        for p in range(sinks // 16 + 1, 20):  # behind the first query's window
            if int(table[0, p]) >= 0 and (p + 1) * 16 <= at + 1 - window:
                page = int(table[0, p])
                kc[page] = vc[page] = float("nan")
                free.append(page)
                table[0, p] = -1
        for t in range(at, at + n):
            if int(table[0, t // 16]) < 0:
                table[0, t // 16] = free.pop(0)
            kc[int(table[0, t // 16]), t % 16], vc[int(table[0, t // 16]), t % 16] = k[t], v[t]
        args = [x.cuda() for x in (q[at:at + n], kc, vc, table)]
        lens = i32([at + n]).cuda()
        if n > 1:
            outs.append(attn.attn_prefill_paged_window(*args, i32([0, n]).cuda(), lens, window, sinks, n))
        else:
            outs.append(attn.attn_decode_paged_window(*args, lens, window, sinks))
        at += n
    O, L = masked_ref(oracle.to_f64(q), oracle.to_f64(k), oracle.to_f64(v), window_seen(T, T, window, sinks), d ** -0.5)
    check_out(torch.cat([o for o, _ in outs]), O, torch.bfloat16)
    check_lse(torch.cat([l for _, l in outs]), L)
    assert attn.attn_get_device_error() == 0


def test_binding_refuses():
    c = Case([3, 20], [4, 5], 2, 4, 64, 22, 10, 1)
    q, k, v, table, cu, n = c.args()
    good = dict(q=q, k_cache=k, v_cache=v, block_table=table, cu_seqlens_q=cu, seq_lens=n, window=10, sinks=1, max_q_len=5)
    attn.attn_prefill_paged_window(**good)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=k.float()), dict(v_cache=v[:1]), dict(k_cache=k[..., :32]),
               dict(block_table=table[:1]), dict(block_table=table.long()), dict(cu_seqlens_q=cu[:2]), dict(seq_lens=n[:1]),
               dict(seq_lens=n.cpu()), dict(o=q.float()), dict(lse=torch.empty((2, 9), device="cuda"))):
        with pytest.raises(ValueError):
            attn.attn_prefill_paged_window(**{**good, **kw})
    for kw in (dict(max_q_len=0), dict(window=0), dict(sinks=-1), dict(scale=-1.0),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(attn.AttnError):
            attn.attn_prefill_paged_window(**{**good, **kw})
    assert attn.attn_get_device_error() == 0
