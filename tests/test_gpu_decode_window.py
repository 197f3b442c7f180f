"""attn_decode_paged_window and attn_decode_paged_window_e4m3 against the
definition in float64 over the keys that each row sees. Tolerances are those of
parity.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle
import workloads as W
from e4m3_cases import decode_case, empty_cache, values
from masked_cases import cache_inputs, hide_pages, i32, masked_ref, row_keys, window_seen
from parity import check_lse, check_lse_nonfinite, check_nonfinite, check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def case(lens, h_kv, g, d, seed, window, sinks, eight=False, qk_mult=1.0):
    """(q, caches..., table, lengths) on the CPU; pages out of sight have no entry."""
    if eight:
        q, kc, vc, ks, vs, table, n = decode_case(lens, h_kv, g, d, seed)
        caches = [kc, vc, ks, vs]
    else:
        table, k, v = cache_inputs(lens, h_kv, d, seed, qk_mult)
        q = W.normal((len(lens), h_kv * g, d), seed * 5 + 1, torch.bfloat16, mult=qk_mult)
        caches, n = [k, v], i32(lens)
    return [q, *caches, hide_pages(table, lens, [1] * len(lens), window, sinks), n]


def reference(args, window, sinks, scale=None, rows=None):
    q, table, n = args[0], args[-2], args[-1]
    if len(args) == 7:
        k, v = (torch.from_numpy(values(args[1 + i], args[3 + i])) for i in (0, 1))
    else:
        k, v = args[1], args[2]
    B, h, d = q.shape
    O, L = np.zeros((B, h, d)), np.full((B, h), -np.inf)
    for b in range(B) if rows is None else rows:
        m = int(n[b])
        if m:
            seen = window_seen(1, m, window, sinks)[0]
            kk, vv = (row_keys(c, table[b], m)[seen] for c in (k, v))
            o, l = masked_ref(oracle.to_f64(q[b:b + 1]), kk, vv, np.ones((1, len(kk)), bool),
                              d ** -0.5 if scale is None else scale)
            O[b], L[b] = o[0], l[0]
    return O, L


def run(args, window, sinks, **kw):
    f = attn.attn_decode_paged_window_e4m3 if len(args) == 7 else attn.attn_decode_paged_window
    return f(*[t.cuda() for t in args], window, sinks, **kw)


def check(args, window, sinks, **kw):
    O, L = reference(args, window, sinks)
    o, lse = run(args, window, sinks, **kw)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


LENS = [0, 1, 5, 15, 16, 17, 31, 33, 64, 100, 333]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (15, 0), (16, 4), (17, 16), (33, 17), (64, 40), (100, 3),
                                          (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 31 - 1)])
def test_lengths_around_pages(window, sinks, d, eight):
    check(case(LENS, 2, 3, d, 7 + window % 100 + sinks % 100, window, sinks, eight), window, sinks)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("h_kv,g", [(1, 1), (2, 2), (8, 4), (3, 5), (1, 8), (2, 9), (1, 20)])
def test_head_layouts(h_kv, g, eight):
    check(case([40, 0, 3, 200], h_kv, g, 128, h_kv + g, 37, 3, eight), 37, 3)


@pytest.mark.parametrize("eight", [False, True])
def test_every_window_and_sink_count_of_a_row(eight):
    """One unit in a cluster: each window start and sink end within two pages."""
    args = case([50], 1, 2, 64, 3, 50, 50, eight)
    for window in range(1, 52, 3):
        for sinks in range(0, 36, 5):
            check(args, window, sinks)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("B,length,window,sinks", [(40, 700, 300, 4), (300, 90, 33, 17), (2, 30000, 20000, 5),
                                                   (20, 5000, 4097, 0)])
def test_batches_cut_over_the_gpu(B, length, window, sinks, eight):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, length + 1, (B,), generator=g).tolist()
    lens[-1] = length
    args = case(lens, 8, 4, 128 if B < 300 else 64, B, window, sinks, eight)
    rows = sorted({0, 1, B // 2, B - 2, B - 1})
    O, L = reference(args, window, sinks, rows=rows)
    o, lse = run(args, window, sinks)
    check_out(o[rows], O[rows], torch.bfloat16)
    check_lse(lse[rows], L[rows])
    again, lse2 = run(args, window, sinks)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("eight", [False, True])
def test_window_beyond_the_rows_is_plain_decode(eight):
    args = [t.cuda() for t in case([500, 3, 0, 77], 2, 4, 128, 9, 10 ** 6, 0, eight)]
    o, lse = run(args, 10 ** 6, 0)
    if eight:
        o2, lse2 = attn.attn_decode_paged_e4m3(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    else:
        o2, lse2 = attn.attn_decode_paged(*args, 3)
        assert ((o.float() - o2.float()).abs() <= 4e-3 + o2.float().abs() * 2.0 ** -7).all()
        m = ~torch.isneginf(lse2)
        assert (lse[m] - lse2[m]).abs().max() <= 2e-4 and torch.equal(torch.isneginf(lse), ~m)


def test_slots_out_of_sight_never_reach_a_row():
    """NaN and infinities between the sinks and the window, in the pages where
    either ends, and behind the row's end."""
    window, sinks = 40, 5
    for lens in ([200, 47, 133], [200] * 20):  # a cluster per unit, and runs
        args = case(lens, 2, 4, 128, 11, 10 ** 6, 0)
        O, L = reference(args, window, sinks)
        q, k, v, tab, n = args
        for b, m in enumerate(lens):
            hidden = ~window_seen(1, m, window, sinks)[0]
            for j in np.nonzero(hidden)[0]:
                k[int(tab[b, j // 16]), j % 16] = float("nan") if j % 2 else float("inf")
                v[int(tab[b, j // 16]), j % 16] = float("inf") if j % 3 else float("nan")
            if m % 16:
                k[int(tab[b, m // 16]), m % 16:] = float("nan")
                v[int(tab[b, m // 16]), m % 16:] = float("nan")
        o, lse = run(args, window, sinks)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)


def test_nonfinite_values_in_sight():
    window, sinks = 30, 3
    args = case([100, 100, 100], 2, 2, 64, 12, window, sinks)
    q, k, v, tab, n = args
    v[int(tab[0, 0]), 2, 1, 5] = float("nan")   # a sink of row 0, KV head 1
    k[int(tab[1, 5]), 3, 0, 0] = float("nan")   # in row 1's window, KV head 0
    v[int(tab[2, 6]), 0, 0, 9] = float("inf")   # in row 2's window
    with np.errstate(invalid="ignore"):
        O, L = reference(args, window, sinks)
    o, lse = run(args, window, sinks)
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)


@pytest.mark.parametrize("eight", [False, True])
def test_only_visible_pages_are_looked_up(eight):
    """Entries of pages out of sight may hold anything; a visible one outside
    the cache reads as zeros and is flagged."""
    window, sinks = 50, 20
    lens = [300, 90, 0]
    args = case(lens, 2, 4, 64, 13, window, sinks, eight)
    want, lse_w = run(args, window, sinks)
    args[-2] = hide_pages(args[-2], lens, [1] * 3, window, sinks, value=2 ** 31 - 1)
    o, lse = run(args, window, sinks)
    assert torch.equal(o, want) and torch.equal(lse, lse_w)
    assert attn.attn_get_device_error() == 0
    args[-2][0, 1] = -5  # a sink page
    o, lse = run(args, window, sinks)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    z = args[1].shape[0]
    fixed = [args[0]] + [torch.cat([c, torch.zeros_like(c[:1])]) for c in args[1:-2]] + [args[-2].clone(), args[-1]]
    fixed[-2][0, 1] = z
    O, L = reference(fixed, window, sinks)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_lengths_outside_the_table_are_clamped():
    window, sinks = 50, 4
    args = case([64, 30], 2, 4, 64, 14, 10 ** 6, 0)
    O, L = reference(args, window, sinks)
    args[-1][0] = 10 ** 9
    args[-1][1] = -1
    o, lse = run(args, window, sinks)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    check_out(o[:1], O[:1], torch.bfloat16)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("eight", [False, True])
def test_outputs_and_workspace_stay_in_bounds(eight):
    for lens in ([5, 0, 300], [40] * 70):
        args = case(lens, 2, 4, 128, 15, 100, 3, eight)
        O, L = reference(args, 100, 3)
        B, h, d = args[0].shape
        need = attn.attn_decode_window_workspace_bytes(B, h, 2, d)
        ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")  # NaN where not written
        buf = torch.full((B * h * d + 2048,), float("nan"), dtype=torch.bfloat16, device="cuda")
        o = buf[1024:-1024].view(B, h, d)
        lbuf = torch.full((B * h + 8,), 7.0, device="cuda")
        lse = lbuf[4:-4].view(B, h)
        run(args, 100, 3, workspace=ws[:need], o=o, lse=lse)
        torch.cuda.synchronize()
        assert torch.isnan(buf[:1024].float()).all() and torch.isnan(buf[-1024:].float()).all()
        assert (lbuf[:4] == 7).all() and (lbuf[-4:] == 7).all() and (ws[need:] == 0xff).all()
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
        o2, none = run(args, 100, 3, return_lse=False)
        assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("B", [2, 40])
def test_captured_and_replayed_with_new_lengths(B):
    window, sinks = 70, 6
    args = [t.cuda() for t in case([400] * B, 2, 4, 128, 16, 10 ** 6, 0)]
    q, n = args[0], args[-1]
    ws = torch.empty(attn.attn_decode_window_workspace_bytes(B, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(args, window, sinks, workspace=ws, o=o, lse=lse)
    for step in (0, 1, 17, 75, 76, 77, 400):
        n.copy_(torch.tensor([max(0, step - 3 * i) for i in range(B)], dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        O, L = reference([t.cpu() for t in args], window, sinks)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)


def test_two_streams_at_once():
    a = [t.cuda() for t in case([3000] * 5, 2, 4, 128, 17, 1000, 4)]
    b = [t.cuda() for t in case([300] * 50, 2, 4, 128, 18, 100, 4)]
    want = [run(a, 1000, 4), run(b, 100, 4)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(run(a, 1000, 4, stream=s1), run(b, 100, 4, stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(y[0], want[1][0])


@pytest.mark.parametrize("exp", [10, 24, 30, 100])
def test_large_logits(exp):
    """One visible key leads by 2^(exp - 3) or more: the row is that key's value."""
    window, sinks = 100, 4
    args = case([300, 80], 2, 4, 64, 19, window, sinks)
    q, k, v, tab, n = args
    q.zero_()
    q[:, :, 0] = 2.0 ** exp
    k.zero_()
    k[..., 0] = torch.randint(-8, 8, k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for b, j in ((0, 250), (1, 40)):
        k[int(tab[b, j // 16]), j % 16, :, 0] = 8
    O, L = reference(args, window, sinks)
    o, lse = run(args, window, sinks)
    if exp >= 10:  # (the others' weights are below e^-128)
        assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()


def test_far_pages_beyond_32_bit_offsets():
    nb, h_kv, d, window, sinks = 140000, 8, 128, 30, 4
    assert nb * h_kv * 16 * d > 2 ** 31
    args = case([70, 20], h_kv, 4, d, 20, window, sinks)
    q, k, v, tab, n = args
    far_k = torch.empty((nb, 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
    far_v = torch.empty_like(far_k)
    for page in range(k.shape[0]):
        far_k[nb - 1 - page] = k[page].cuda()
        far_v[nb - 1 - page] = v[page].cuda()
    O, L = reference(args, window, sinks)
    o, lse = run([q, far_k, far_v, torch.where(tab < 0, tab, nb - 1 - tab), n], window, sinks)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_lengths_and_tables_rewritten_just_before():
    """The kernel in front lets the decode start at once and rewrites the
    lengths or the table 50 us later."""
    window, sinks = 100, 4
    for lens in ([200, 0, 33], [200] * 40):
        args = case(lens, 2, 4, 128, 21, 10 ** 6, 0)
        O, L = reference(args, window, sinks)
        dev = [t.cuda() for t in args]
        for i in (3, 4):
            old = torch.zeros_like(dev[i])
            now = dev[:i] + [old] + dev[i + 1:]
            run(now, window, sinks)  # warm: lines of the old contents
            attn.attn_selftest_delayed_copy(old.view(-1), dev[i].view(-1), delay_us=50)
            o, lse = run(now, window, sinks)
            check_out(o, O, torch.bfloat16)
            check_lse(lse, L)
        assert attn.attn_get_device_error() == 0


def test_steps_write_and_decode_over_the_8_bit_cache():
    """Tokens enter the 8-bit cache one step at a time and each step's query
    decodes over the window and the sinks, from pages that are given back as
    they leave the window."""
    h_kv, g, d, window, sinks, steps = 2, 4, 128, 40, 3, 90
    kv = W.normal((steps, 2, h_kv, d), 41, torch.bfloat16).cuda()
    q = W.normal((steps, h_kv * g, d), 42, torch.bfloat16).cuda()
    cache = empty_cache(5, h_kv, d)  # 5 pages serve 90 tokens
    table = torch.full((1, 8), -1, dtype=torch.int32)
    free, outs = [4, 2, 0, 3, 1], []
    for t in range(steps):
        if t % 16 == 0:
            for p in range(1, 8):  # pages behind the window, but the sinks'
                if int(table[0, p]) >= 0 and (p + 1) * 16 <= t + 1 - window:
                    free.append(int(table[0, p]))
                    table[0, p] = -1
            table[0, t // 16] = free.pop(0)
        tab, n = table.cuda(), i32([t + 1]).cuda()
        attn.attn_cache_write_e4m3(kv[t:t + 1, 0], kv[t:t + 1, 1], *cache, tab, i32([0, 1]).cuda(), n)
        outs.append(attn.attn_decode_paged_window_e4m3(q[t:t + 1], *cache, tab, n, window, sinks))
    import oracle.cache_e4m3 as fmt

    stored = fmt.values_ref(*fmt.quantise_ref(kv.double().cpu().numpy()))
    O, L = masked_ref(oracle.to_f64(q), stored[:, 0], stored[:, 1], window_seen(steps, steps, window, sinks), d ** -0.5)
    check_out(torch.cat([o for o, _ in outs]), O, torch.bfloat16)
    check_lse(torch.cat([l for _, l in outs]), L)
    assert attn.attn_get_device_error() == 0


def test_binding_refuses():
    q, k, v, tab, n = [t.cuda() for t in case([3, 20], 2, 4, 64, 22, 10, 1)]
    good = dict(q=q, k_cache=k, v_cache=v, block_table=tab, seq_lens=n, window=10, sinks=1)
    attn.attn_decode_paged_window(**good)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=k.float()), dict(v_cache=v[:1]), dict(k_cache=k[..., :32]),
               dict(block_table=tab[:1]), dict(block_table=tab.long()), dict(seq_lens=n[:1]), dict(seq_lens=n.cpu()),
               dict(o=q.float()), dict(lse=torch.empty((2, 9), device="cuda"))):
        with pytest.raises(ValueError):
            attn.attn_decode_paged_window(**{**good, **kw})
    for kw in (dict(window=0), dict(sinks=-1), dict(scale=-1.0),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(attn.AttnError):
            attn.attn_decode_paged_window(**{**good, **kw})
    for kw in (dict(window=2 ** 31), dict(window=1.5), dict(sinks=None)):
        with pytest.raises((ValueError, TypeError)):
            attn.attn_decode_paged_window(**{**good, **kw})
    assert attn.attn_get_device_error() == 0
