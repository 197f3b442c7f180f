"""attn_decode_paged_shared against the float64 oracle over each row's prefix
and own keys laid end to end. Tolerances are those of parity.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle
import workloads as W
from e4m3_cases import empty_cache
from parity import check_lse, check_nonfinite, check_lse_nonfinite, check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def case(prefix, lens, h_kv, g, d, seed, qk_mult=1.0):
    """q, caches, prefix table and length, block table, lengths (CPU). Prefix
    and own pages are shuffled through one pool."""
    table, nb = W.paged_layout([prefix] + list(lens), seed, spare_pages=2)
    n = (prefix + 15) // 16
    ptab = table[0, :max(n, 1)].clamp(min=0).contiguous()
    width = max([1] + [(x + 15) // 16 for x in lens])
    tab = torch.full((len(lens), width), -1, dtype=torch.int32)
    tab[:, :] = table[1:, :width]
    q = W.normal((len(lens), h_kv * g, d), seed * 5 + 1, torch.bfloat16, mult=qk_mult)
    k = W.normal((nb, 16, h_kv, d), seed * 5 + 2, torch.bfloat16, mult=qk_mult)
    v = W.normal((nb, 16, h_kv, d), seed * 5 + 3, torch.bfloat16)
    return [q, k, v, ptab, torch.tensor([prefix], dtype=torch.int32), tab, torch.tensor(lens, dtype=torch.int32)]


def keys(cache, pages, n):
    return oracle.to_f64(cache[pages.long()]).reshape(-1, *cache.shape[2:])[:n].transpose(1, 0, 2)


def reference(q, k, v, ptab, plen, tab, lens, scale=None, rows=None):
    B, h, d = q.shape
    O, L = np.zeros((B, h, d)), np.full((B, h), -np.inf)
    P = int(plen)
    pk, pv = (keys(c, ptab[:(P + 15) // 16], P) for c in (k, v))
    for b in range(B) if rows is None else rows:
        n = int(lens[b])
        kk, vv = (np.concatenate([p, keys(c, tab[b, :(n + 15) // 16], n)], 1) for p, c in ((pk, k), (pv, v)))
        if kk.shape[1]:
            o, l = oracle.attention_ref(oracle.to_f64(q[b])[:, None], kk, vv, d ** -0.5 if scale is None else scale)
            O[b], L[b] = o[:, 0], l[:, 0]
    return O, L


def run(args, **kw):
    return attn.attn_decode_paged_shared(*[t.cuda() for t in args], **kw)


@pytest.mark.parametrize("h_kv,g", [(2, 1), (1, 2), (3, 4), (2, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 16, 127, 128, 129, 300, 1000])
def test_small_prefixes_and_own_lengths(h_kv, g, d, prefix):
    lens = [0, 1, 15, 16, 17, 40, 333]
    args = case(prefix, lens, h_kv, g, d, seed=g + d + prefix)
    O, L = reference(*args)
    o, lse = run(args)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    if prefix == 0:
        assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("B,g,h_kv", [(1, 1, 1), (16, 8, 1), (17, 8, 2), (32, 4, 2), (33, 4, 1), (64, 4, 2), (65, 4, 1),
                                      (130, 2, 1), (300, 1, 2), (200, 8, 1)])
@pytest.mark.parametrize("prefix", [77, 700])
def test_row_blocks(B, g, h_kv, prefix):
    """Row counts at and around one tile, one block of two tiles, several blocks."""
    lens = [(7 * i) % 23 for i in range(B)]
    args = case(prefix, lens, h_kv, g, 64, seed=B)
    O, L = reference(*args)
    o, lse = run(args)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("B,h_kv,prefix", [(2, 8, 20000), (3, 1, 40000), (70, 3, 9000)])
def test_long_prefixes_cut_over_the_gpu(B, h_kv, prefix):
    lens = [100 + 37 * i % 900 for i in range(B)]
    args = case(prefix, lens, h_kv, 4, 128, seed=B)
    rows = range(B) if B < 10 else [0, 31, 32, 63, 64, 69]
    O, L = reference(*args, rows=rows)
    o, lse = run(args)
    check_out(o[list(rows)], O[list(rows)], torch.bfloat16)
    check_lse(lse[list(rows)], L[list(rows)])
    again, lse2 = run(args)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert attn.attn_get_device_error() == 0


def test_many_row_blocks():
    """More row blocks than the GPU's first wave takes in equal parts."""
    B, lens = 2100, [i % 5 for i in range(2100)]
    args = case(200, lens, 8, 8, 64, seed=1)  # 66 blocks a head
    rows = [0, 31, 32, 1000, 2047, 2048, 2099]
    O, L = reference(*args, rows=rows)
    o, lse = run(args)
    check_out(o[rows], O[rows], torch.bfloat16)
    check_lse(lse[rows], L[rows])


def test_equals_the_decode_over_whole_rows():
    """The prefix's pages in front of every row's own in one table: the same
    keys through attn_decode_paged."""
    prefix, lens = 160, [5, 0, 100, 64]
    args = case(prefix, lens, 2, 4, 128, seed=4)
    q, k, v, ptab, plen, tab, n = [t.cuda() for t in args]
    o, lse = attn.attn_decode_paged_shared(q, k, v, ptab, plen, tab, n)
    full = torch.cat([ptab[None].expand(len(lens), -1), tab], 1).contiguous()
    o2, lse2 = attn.attn_decode_paged(q, k, v, full, (n + prefix).to(torch.int32), 3)
    assert ((o.float() - o2.float()).abs() <= 4e-3 + o2.float().abs() * 2.0 ** -7).all()
    assert (lse - lse2).abs().max() <= 2e-4


@pytest.mark.parametrize("where", ["prefix", "own", "middle"])
def test_outliers_force_the_reference_up(where):
    """One key that outweighs the rest, late in the prefix, in its middle, or
    among a row's own keys; logits of standard deviation 9 elsewhere."""
    prefix, lens = 900, [60, 61]
    args = case(prefix, lens, 2, 4, 128, seed=6, qk_mult=3.0)
    q, k, v, ptab, plen, tab, n = args
    one = (q[0].view(2, 4, 128)[:, 0] * 2).to(torch.bfloat16)
    if where == "own":
        k[int(tab[0, 3]), 11] = one
    else:
        pos = 899 if where == "prefix" else 300
        k[int(ptab[pos // 16]), pos % 16] = one
    O, L = reference(*args)
    o, lse = run(args)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("mult", [1.0, 1e5, 2.0 ** -20, 2.0 ** 30])
def test_value_magnitudes(mult):
    """Values of every size (fp16 holds neither the large nor the small ones);
    one tile of ordinary values among them."""
    prefix, lens = 400, [33, 0]
    args = case(prefix, lens, 1, 4, 128, seed=8)
    args[2] = (args[2].float() * mult).to(torch.bfloat16)
    O, L = reference(*args)
    o, lse = run(args)
    check_out((o.double() / mult).cpu(), O / mult, torch.bfloat16)
    check_lse(lse, L)


def test_mixed_magnitudes_between_tiles():
    """Large values in one key tile and one column only."""
    prefix, lens = 700, [3] * 40
    args = case(prefix, lens, 2, 4, 64, seed=9)
    page = int(args[3][20])
    args[2][page, 3, 1, 7] = 3e5
    O, L = reference(*args)
    mag, _ = reference(args[0], args[1], args[2].abs(), *args[3:])
    o, lse = run(args)
    check_out(o, O, torch.bfloat16, mag=mag)
    check_lse(lse, L)


def test_slots_past_the_lengths_never_reach_a_row():
    prefix, lens = 133, [17, 1, 0]
    args = case(prefix, lens, 2, 4, 128, seed=10)
    O, L = reference(*args)
    q, k, v, ptab, plen, tab, n = args
    for c in (k, v):
        c[int(ptab[-1]), prefix % 16:] = float("nan")
        c[int(tab[0, 1]), 1:] = float("inf")
        c[int(tab[1, 0]), 1:] = float("nan")
    o, lse = run(args)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_nonfinite_keys_and_values_of_the_prefix_and_of_a_row():
    prefix, lens = 200, [20, 20, 20]
    args = case(prefix, lens, 2, 2, 64, seed=11)
    q, k, v, ptab, plen, tab, n = args
    v[int(ptab[3]), 2, 1, 5] = float("nan")   # every row, KV head 1, column 5
    k[int(tab[1, 0]), 3, 0, 0] = float("nan")  # row 1, KV head 0
    v[int(tab[2, 1]), 0, 0, 9] = float("inf")  # row 2, KV head 0, column 9
    with np.errstate(invalid="ignore"):
        O, L = reference(*args)
    o, lse = run(args)
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)


def test_bad_pages_and_lengths_are_flagged():
    prefix, lens = 64, [20, 33]
    args = case(prefix, lens, 2, 4, 128, seed=12)
    attn.attn_get_device_error()
    bad = [t.clone() for t in args]
    bad[3][1] = args[1].shape[0] + 3
    bad[5][1, 2] = -7
    o, lse = run(bad)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    z = args[1].shape[0]  # a page of zeros
    zero = torch.zeros_like(args[1][:1])
    fixed = [args[0], torch.cat([args[1], zero]), torch.cat([args[2], zero]), bad[3].clone(), args[4], bad[5].clone(), args[6]]
    fixed[3][1] = fixed[5][1, 2] = z
    O, L = reference(*fixed)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    bad = [t.clone() for t in args]
    bad[4][0] = 10 ** 9
    o, lse = run(bad)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    O, L = reference(*args)  # clamped to the table: its 64 keys
    check_out(o, O, torch.bfloat16)
    bad[4][0] = -3
    bad[6][0] = -1
    o, lse = run(bad)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_outputs_and_workspace_stay_in_bounds():
    for lens, prefix in (([5, 0, 300], 500), ([4] * 70, 150)):
        args = case(prefix, lens, 2, 4, 128, seed=13)
        O, L = reference(*args)
        B, h, d = args[0].shape
        need = attn.attn_decode_shared_workspace_bytes(B, h, 2, d)
        ws = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")  # NaN where not written
        buf = torch.full((B * h * d + 2048,), float("nan"), dtype=torch.bfloat16, device="cuda")
        o = buf[1024:-1024].view(B, h, d)
        lbuf = torch.full((B * h + 8,), 7.0, device="cuda")
        lse = lbuf[4:-4].view(B, h)
        run(args, workspace=ws[:need], o=o, lse=lse)
        torch.cuda.synchronize()
        assert torch.isnan(buf[:1024].float()).all() and torch.isnan(buf[-1024:].float()).all()
        assert (lbuf[:4] == 7).all() and (lbuf[-4:] == 7).all() and (ws[need:] == 0xff).all()
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
        o2, none = run(args, return_lse=False)
        assert none is None and torch.equal(o, o2)


def test_captured_and_replayed_with_new_lengths():
    args = [t.cuda() for t in case(1000, [300, 0, 500, 17], 2, 4, 128, seed=14)]
    q, k, v, ptab, plen, tab, n = args
    ws = torch.empty(attn.attn_decode_shared_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.attn_decode_paged_shared(*args, workspace=ws, o=o, lse=lse)
    for P, new in ((1000, [300, 0, 500, 17]), (0, [1, 0, 17, 0]), (129, [300, 0, 497, 16]), (960, [0, 0, 0, 0])):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        plen.fill_(P)
        o.fill_(float("nan"))
        graph.replay()
        O, L = reference(*[t.cpu() for t in args])
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)


def test_two_streams_at_once():
    a = [t.cuda() for t in case(3000, [100] * 5, 2, 4, 128, seed=15)]
    b = [t.cuda() for t in case(500, [10] * 90, 2, 4, 128, seed=16)]
    want = [attn.attn_decode_paged_shared(*x) for x in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(attn.attn_decode_paged_shared(*a, stream=s1), attn.attn_decode_paged_shared(*b, stream=s2))
           for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(y[0], want[1][0])


def test_prefix_read_back_from_the_8_bit_cache():
    """A prompt written to the 8-bit cache and read back as bf16 pages serves
    as the shared prefix; rows of the 8-bit decode over prompt and own keys give
    the same."""
    h_kv, g, d, P, B = 2, 4, 128, 200, 3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    own = [10, 33, 1]
    x = W.normal((P, 2, h_kv, d), 31, torch.bfloat16).cuda()
    y = [W.normal((n, 2, h_kv, d), 32 + n, torch.bfloat16).cuda() for n in own]
    # each row's whole sequence in the 8-bit cache
    tab, nb = W.paged_layout([P + n for n in own], 3)
    cache = empty_cache(nb, h_kv, d)
    seqs = torch.cat([torch.cat([x, t]) for t in y])
    cu = [0]
    for n in own:
        cu.append(cu[-1] + P + n)
    lens = i32([P + n for n in own])
    attn.attn_cache_write_e4m3(seqs[:, 0], seqs[:, 1], *cache, tab.cuda(), i32(cu), lens)
    q = W.normal((B, h_kv * g, d), 40, torch.bfloat16).cuda()
    o8, l8 = attn.attn_decode_paged_e4m3(q, *cache, tab.cuda(), lens)
    # the prefix (row 0's first P tokens) and each row's own tokens, read back into bf16 pages
    pages = (P + 15) // 16
    kc = torch.zeros((pages + 16, 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    flat = lambda c: c.view(-1, h_kv, d)
    attn.attn_cache_read_e4m3(*cache, tab[:1].cuda(), i32([0, P]), i32([P]), flat(kc)[:P], flat(vc)[:P])
    btab, at = [], pages
    for b, n in enumerate(own):
        m = (n + 15) // 16
        sl = slice(at * 16, at * 16 + n)
        attn.attn_cache_read_e4m3(*cache, tab[b:b + 1].cuda(), i32([0, n]), i32([P + n]), flat(kc)[sl], flat(vc)[sl])
        btab.append(list(range(at, at + m)) + [-1] * (3 - m))
        at += m
    o, lse = attn.attn_decode_paged_shared(q, kc, vc, i32(list(range(pages))), i32([P]), i32(btab), i32(own))
    assert ((o.float() - o8.float()).abs() <= 4e-3 + o8.float().abs() * 2.0 ** -7).all()
    assert (lse - l8).abs().max() <= 2e-4
    assert attn.attn_get_device_error() == 0


def test_binding_refuses():
    """What the compiled binding checks before it calls the library."""
    q, k, v, ptab, plen, tab, n = [t.cuda() for t in case(40, [3, 20], 2, 4, 64, seed=21)]
    good = dict(q=q, k_cache=k, v_cache=v, prefix_table=ptab, prefix_len=plen, block_table=tab, seq_lens=n)
    attn.attn_decode_paged_shared(**good)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(k_cache=k.float()), dict(v_cache=v[:2]), dict(k_cache=k[..., :32]),
               dict(prefix_table=ptab[None]), dict(prefix_table=ptab.long()), dict(prefix_len=plen[0]),
               dict(prefix_len=torch.cat([plen, plen])), dict(prefix_len=plen.cpu()), dict(block_table=tab[:1]),
               dict(seq_lens=n[:1]), dict(o=q.float()), dict(lse=torch.empty((2, 9), device="cuda"))):
        with pytest.raises(ValueError):
            attn.attn_decode_paged_shared(**{**good, **kw})
    with pytest.raises(attn.AttnError):
        attn.attn_decode_paged_shared(**good, scale=-1.0)
    with pytest.raises(attn.AttnError):
        attn.attn_decode_paged_shared(**good, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert attn.attn_get_device_error() == 0


def test_far_pages_beyond_32_bit_offsets():
    """Prefix and own pages whose elements lie past 2^31."""
    nb, h_kv, d = 140000, 8, 128
    assert nb * h_kv * 16 * d > 2 ** 31
    args = case(40, [20, 0], h_kv, 4, d, seed=22)
    q, k, v, ptab, plen, tab, n = args
    far_k = torch.empty((nb, 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
    far_v = torch.empty_like(far_k)
    move = lambda t: torch.where(t < 0, t, nb - 1 - t)
    for page in range(k.shape[0]):
        far_k[nb - 1 - page] = k[page].cuda()
        far_v[nb - 1 - page] = v[page].cuda()
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_shared(q.cuda(), far_k, far_v, move(ptab).cuda(), plen.cuda(), move(tab).cuda(), n.cuda())
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("v_mult", [1.0, 1e6])
@pytest.mark.parametrize("shift", [0, -16])
@pytest.mark.parametrize("exp", [16, 21, 24, 27, 30, 40, 110])
def test_logits_beyond_the_precision_of_differences(exp, shift, v_mult, where):
    """Logits up to 2^exp in magnitude, exact up to the factor log2(e): one key
    leads by 2^(exp - 3) or more, so the row is that key's value. In fp32 the
    logits' spacing passes the weights' range (2^15) from 2^27 on."""
    prefix, lens = 700, [500, 20]
    args = case(prefix, lens, 2, 4, 64, seed=23)
    q, k, v, ptab, plen, tab, n = args
    q.zero_()
    q[:, :, 0] = 2.0 ** exp  # scale 1/8: the leading key's logit is 2^exp (or -2^exp)
    k.zero_()
    g = torch.Generator().manual_seed(1)
    k[..., 0] = torch.randint(-8, 8, k.shape[:-1], generator=g).to(torch.bfloat16) + shift
    v *= v_mult
    if where == "prefix":
        k[int(ptab[20]), 3, :, 0] = 8 + shift
    else:
        for b in range(2):
            k[int(tab[b, 1]), 3, :, 0] = 8 + shift
    O, L = reference(*args)
    o, lse = run(args)
    # The weights besides the leading one's are 0; the output rounds once, and V
    # (fp16 in the prefix: within 2^-25) and the accumulation far below that.
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()


def test_lengths_and_tables_rewritten_just_before():
    """The kernel in front lets the decode start at once and rewrites one of
    lengths and tables 50 us later."""
    args = case(300, [200, 0, 33], 2, 4, 128, seed=24)
    O, L = reference(*args)
    dev = [t.cuda() for t in args]
    for i in (3, 4, 5, 6):
        old = torch.zeros_like(dev[i])
        now = dev[:i] + [old] + dev[i + 1:]
        attn.attn_decode_paged_shared(*now)  # warm: lines of the old contents
        attn.attn_selftest_delayed_copy(old.view(-1), dev[i].view(-1), delay_us=50)
        o, lse = attn.attn_decode_paged_shared(*now)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
    assert attn.attn_get_device_error() == 0
