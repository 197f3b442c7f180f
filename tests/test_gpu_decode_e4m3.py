"""attn_decode_paged_e4m3 against the float64 oracle over the stored values.
Tolerances are those of parity.py: the stored values are exact inputs, q and the
weights are rounded as in the bf16 decode or finer (fp16 weights, relative 2^-11)."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle
import workloads as W
from e4m3_cases import cache_from, decode_case, empty_cache, values
from parity import check_lse, check_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def cuda(*ts):
    return [t.cuda() for t in ts]


def reference(q, kc, vc, ks, vs, table, lens, scale=None):
    return oracle.decode_paged_ref(q, values(kc, ks), values(vc, vs), table, lens,
                                   q.shape[-1] ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("h_kv,g", [(2, 1), (2, 2), (3, 3), (2, 4), (1, 5), (2, 7), (1, 8), (2, 12), (1, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_around_pages(h_kv, g, d):
    lens = [0, 1, 15, 16, 17, 40, 333, 1000, 0]
    args = decode_case(lens, h_kv, g, d, seed=g + d)
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("lens", [[1], [16], [128], [129], [5000], [70000], [3] * 400, [100, 0, 9000] * 20])
def test_runs_of_every_kind(lens):
    """One page, one CTA's pages and one more, rows cut over many CTAs, many
    rows in one CTA, more rows than threads in a CTA."""
    args = decode_case(lens, 2, 4, 128, seed=len(lens))
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    again, lse2 = attn.attn_decode_paged_e4m3(*cuda(*args))
    assert torch.equal(o, again) and torch.equal(lse, lse2)  # no order of arrival in the result


def test_no_rows_with_keys():
    args = decode_case([0, 0, 0], 2, 2, 64, seed=1)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("v_mult", [2.0 ** -60, 2.0 ** 40])
def test_value_magnitudes(v_mult):
    """V far from 1: results scale with it."""
    lens = [700, 33]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 4, 128, seed=3, v_mult=v_mult)
    O, L = reference(q, kc, vc, ks, vs, table, n)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kc, vc, ks, vs, table, n))
    check_out((o.double() / v_mult).cpu(), O / v_mult, torch.bfloat16)  # division by 2^n: exact
    check_lse(lse, L)


def test_mixed_value_scales():
    """Values of one row spread over 2^40, the heavy keys among the small ones
    (attention sinks): the sum is right relative to its own size."""
    lens = [2000]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 1, 4, 128, seed=5)
    g = torch.Generator().manual_seed(1)
    vs = (vs.int() + torch.randint(-40, 1, vs.shape, generator=g)).to(torch.uint8)
    O, L = reference(q, kc, vc, ks, vs, table, n)
    Omag, _ = oracle.decode_paged_ref(q, values(kc, ks), np.abs(values(vc, vs)), table, n, 128 ** -0.5)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kc, vc, ks, vs, table, n))
    # each fp16 weight is within 2^-12 of its value, the output within half a bf16 step, 2^-9
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= 2.0 ** -11 * Omag + 2.0 ** -8 * np.abs(O)).all()
    check_lse(lse, L)


def test_zero_value_rows_of_a_dominant_key():
    """A key that takes nearly all the weight and has a zero value (its
    exponent is the smallest there is): what is left comes from the rest."""
    lens = [3000]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 1, 1, 128, seed=6)
    k64 = values(kc, ks)
    page, slot = int(table[0, 40]), 5
    one = q[0, 0].double().numpy() * 2.0
    k64[page, slot, 0] = one
    kc, ks = cache_from(k64.transpose(0, 2, 1, 3))
    v64 = values(vc, vs)
    v64[page, slot, 0] = 0.0
    vc, vs = cache_from(v64.transpose(0, 2, 1, 3))
    assert vs[page, 0, slot] == 10
    O, L = reference(q, kc, vc, ks, vs, table, n)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kc, vc, ks, vs, table, n))
    Omag, _ = oracle.decode_paged_ref(q, values(kc, ks), np.abs(values(vc, vs)), table, n, 128 ** -0.5)
    err = np.abs(o.double().cpu().numpy() - O)
    assert (err <= 2.0 ** -11 * Omag + 2.0 ** -8 * np.abs(O)).all()
    check_lse(lse, L)


def test_flat_tail_under_a_heavy_key():
    """60000 keys of weight 2^-17 of the heaviest: together nearly half the sum."""
    lens = [60000]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 1, 1, 64, seed=7)
    q = torch.zeros_like(q)
    q[0, 0, 0] = 1.0
    k64 = np.zeros_like(values(kc, ks))
    page = int(table[0, 17])
    k64[page, 3, 0, 0] = 8.0 * 17 * np.log(2.0) * 1.0
    kc, ks = cache_from(k64.transpose(0, 2, 1, 3))
    v64 = np.ones_like(k64)
    v64[page, 3] = -1.0
    vc, vs = cache_from(v64.transpose(0, 2, 1, 3))
    args = (q, kc, vc, ks, vs, table, n)
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_extreme_queries():
    """Queries from 2^-100 to 2^60 against ordinary keys at a scale that keeps
    the logits ordinary, and rows of zeros."""
    lens = [200, 200, 200]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 1, 4, 128, seed=8)
    q[1] = 0
    for e in (-100, 60):
        qq = (q.float() * 2.0 ** e).to(torch.bfloat16)
        s = 2.0 ** (-e) * 128 ** -0.5
        O, L = reference(qq, kc, vc, ks, vs, table, n, scale=s)
        o, lse = attn.attn_decode_paged_e4m3(*cuda(qq, kc, vc, ks, vs, table, n), scale=s)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)


def test_large_logits_force_the_reference_up():
    lens = [900, 901]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 4, 128, seed=9)
    ks = (ks.int() + 4).to(torch.uint8)  # logits 16 times as wide
    O, L = reference(q, kc, vc, ks, vs, table, n)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kc, vc, ks, vs, table, n))
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_slots_past_the_length_never_reach_a_row():
    lens = [17, 1, 31]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 4, 128, seed=10)
    O, L = reference(q, kc, vc, ks, vs, table, n)
    kb, vb = kc.view(torch.uint8).clone(), vc.view(torch.uint8).clone()
    for b, ln in enumerate(lens):
        page = int(table[b, (ln - 1) // 16])
        for t, e in ((kb, ks), (vb, vs)):
            t[page, :, ln % 16 or 16:] = 0x7f  # NaN codes
            e[page, :, ln % 16 or 16:] = 255   # and an exponent no write makes
    f8 = torch.float8_e4m3fn
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kb.view(f8), vb.view(f8), ks, vs, table, n))
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)


def test_nan_codes_reach_their_rows_only():
    lens = [50, 50]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 2, 64, seed=11)
    vb = vc.view(torch.uint8).clone()
    vb[int(table[0, 1]), 1, 4, 9] = 0x7f   # row 0, KV head 1, column 9
    kb = kc.view(torch.uint8).clone()
    kb[int(table[1, 2]), 0, 1, 3] = 0xff   # row 1, KV head 0
    f8 = torch.float8_e4m3fn
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kb.view(f8), vb.view(f8), ks, vs, table, n))
    o, lse = o.float().cpu(), lse.cpu()
    want = torch.zeros(2, 4, 64, dtype=torch.bool)
    want[0, 2:, 9] = True
    want[1, :2] = True
    assert torch.equal(torch.isnan(o), want)
    assert torch.isnan(lse).tolist() == [[False] * 4, [True, True, False, False]]


def test_bad_pages_and_lengths_are_flagged():
    lens = [40, 20]
    q, kc, vc, ks, vs, table, n = cuda(*decode_case(lens, 2, 4, 128, seed=12))
    attn.attn_get_device_error()
    bad = table.clone()
    bad[0, 1] = kc.shape[0] + 5
    bad[1, 0] = -2
    ks2 = ks.clone()
    ks2[0] = 255  # the exponents of a page that must not be read instead
    o, lse = attn.attn_decode_paged_e4m3(q, kc, vc, ks, vs, bad, n)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    zeroed = values(kc, ks), values(vc, vs)
    zk, zv = (np.concatenate([x, np.zeros_like(x[:1])]) for x in zeroed)
    fixed = bad.clone()
    fixed[0, 1] = fixed[1, 0] = kc.shape[0]  # a page of zeros
    O, L = oracle.decode_paged_ref(q.cpu(), zk, zv, fixed.cpu(), n.cpu(), 128 ** -0.5)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    long = n.clone()
    long[1] = 10 ** 9
    long[0] = -5
    o, lse = attn.attn_decode_paged_e4m3(q, kc, vc, ks, vs, table.clamp(min=0), long)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    assert (o[0] == 0).all() and torch.isfinite(o.float()).all()


def test_outputs_and_workspace_stay_in_bounds():
    lens = [5, 0, 3000]
    args = decode_case(lens, 2, 4, 128, seed=13)
    O, L = reference(*args)
    B, h, d = args[0].shape
    need = attn.attn_decode_e4m3_workspace_bytes(B, h, 2, d)
    ws = torch.full((need + 512,), 0xab, dtype=torch.uint8, device="cuda")
    buf = torch.full((B * h * d + 2048,), float("nan"), dtype=torch.bfloat16, device="cuda")
    o = buf[1024:-1024].view(B, h, d)
    lbuf = torch.full((B * h + 8,), 7.0, device="cuda")
    lse = lbuf[4:-4].view(B, h)
    attn.attn_decode_paged_e4m3(*cuda(*args), workspace=ws[:need], o=o, lse=lse)
    torch.cuda.synchronize()
    assert torch.isnan(buf[:1024].float()).all() and torch.isnan(buf[-1024:].float()).all()
    assert (lbuf[:4] == 7).all() and (lbuf[-4:] == 7).all() and (ws[need:] == 0xab).all()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    o2, none = attn.attn_decode_paged_e4m3(*cuda(*args), return_lse=False)
    assert none is None and torch.equal(o, o2)


def test_captured_and_replayed_with_new_lengths():
    lens = [300, 0, 5000, 17]
    q, kc, vc, ks, vs, table, n = cuda(*decode_case(lens, 2, 4, 128, seed=14))
    ws = torch.empty(attn.attn_decode_e4m3_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.attn_decode_paged_e4m3(q, kc, vc, ks, vs, table, n, workspace=ws, o=o, lse=lse)
    for new in ([300, 0, 5000, 17], [1, 0, 17, 0], [300, 0, 4097, 16], [0, 0, 0, 0]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        O, L = reference(q.cpu(), kc, vc, ks, vs, table.cpu(), n.cpu())
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)


def test_two_streams_at_once():
    a = cuda(*decode_case([4000, 10], 2, 4, 128, seed=15))
    b = cuda(*decode_case([100] * 30, 2, 4, 128, seed=16))
    want = [attn.attn_decode_paged_e4m3(*x) for x in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((attn.attn_decode_paged_e4m3(*a, stream=s1), attn.attn_decode_paged_e4m3(*b, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], want[0][0]) and torch.equal(x[1], want[0][1])
        assert torch.equal(y[0], want[1][0]) and torch.equal(y[1], want[1][1])


def test_write_decode_and_read_together():
    """A prompt and then tokens one at a time enter the 8-bit cache; each step's
    decode agrees with the bf16 decode over the same tokens read back."""
    h_kv, g, d, B = 2, 4, 128, 3
    final = [70, 33, 130]
    table, nb = W.paged_layout(final, 1)
    tab = table.cuda()
    cache = empty_cache(nb, h_kv, d)
    steps = 5
    x = W.normal((sum(final), 2, h_kv, d), 21, torch.bfloat16).cuda()
    start = [0, final[0], final[0] + final[1]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    prompt = [n - steps for n in final]
    cu = [0, prompt[0], prompt[0] + prompt[1], sum(prompt)]
    rows = torch.cat([x[s:s + p] for s, p in zip(start, prompt)])
    attn.attn_cache_write_e4m3(rows[:, 0], rows[:, 1], *cache, tab, i32(cu), i32(prompt))
    for t in range(1, steps + 1):
        new = torch.stack([x[s + p + t - 1] for s, p in zip(start, prompt)])
        lens = i32([p + t for p in prompt])
        attn.attn_cache_write_e4m3(new[:, 0], new[:, 1], *cache, tab, i32([0, 1, 2, 3]), lens)
        q = W.normal((B, h_kv * g, d), 30 + t, torch.bfloat16).cuda()
        o, lse = attn.attn_decode_paged_e4m3(q, *cache, tab, lens)
        for b in range(B):  # row by row: its pages as a bf16 cache
            n = prompt[b] + t
            pages = (n + 15) // 16
            k = torch.zeros((pages * 16, h_kv, d), dtype=torch.bfloat16, device="cuda")
            v = torch.zeros_like(k)
            attn.attn_cache_read_e4m3(*cache, tab[b:b + 1].contiguous(), i32([0, n]), i32([n]), k, v)
            ident = i32([list(range(pages))])
            ob, lb = attn.attn_decode_paged(q[b:b + 1].contiguous(), k.view(pages, 16, h_kv, d),
                                            v.view(pages, 16, h_kv, d), ident, i32([n]), 2)
            # both within the parity bound of the same exact result
            err = (o[b].float() - ob[0].float()).abs()
            assert (err <= 4e-3 + ob[0].float().abs() * 2.0 ** -7).all()
            assert (lse[b] - lb[0]).abs().max() <= 2e-4
    assert attn.attn_get_device_error() == 0


def test_binding_refuses():
    """What the compiled binding checks before it calls the library."""
    lens = [20, 33]
    good = dict(zip(("q", "kc", "vc", "ks", "vs", "table", "lens"), cuda(*decode_case(lens, 2, 4, 64, seed=20))))
    call = lambda **kw: attn.attn_decode_paged_e4m3(**{**dict(
        q=good["q"], k_cache=good["kc"], v_cache=good["vc"], k_scale=good["ks"], v_scale=good["vs"],
        block_table=good["table"], seq_lens=good["lens"]), **kw})
    call()
    bad = [dict(q=good["q"].float()), dict(q=good["q"][0]), dict(q=good["q"].transpose(0, 1)), dict(q=good["q"].cpu()),
           dict(k_cache=good["kc"].view(torch.uint8)), dict(k_cache=good["kc"][:, :1]), dict(k_cache=good["kc"][:-1]),
           dict(v_scale=good["vs"].int()), dict(k_scale=good["ks"][:, :, :8]), dict(k_scale=good["ks"].cpu()),
           dict(block_table=good["table"].long()), dict(block_table=good["table"][:1]),
           dict(block_table=good["table"].t()), dict(seq_lens=good["lens"].long()), dict(seq_lens=good["lens"][:1]),
           dict(o=torch.empty_like(good["q"], dtype=torch.float32)), dict(o=torch.empty_like(good["q"]).cpu()),
           dict(lse=torch.empty((2, 8), dtype=torch.bfloat16, device="cuda")),
           dict(lse=torch.empty((8, 2), device="cuda").t()), dict(lse=torch.empty((2, 7), device="cuda")),
           dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(attn.AttnError):
            call(**kw)
    with pytest.raises((TypeError, ValueError)):
        call(scale="x")
    with pytest.raises((TypeError, ValueError, AttributeError)):
        call(block_table=None)
    assert attn.attn_get_device_error() == 0


def one_hot_keys(shape, seed, shift):
    """Keys of small integers (each one e4m3 and bf16 number) along dim 0 only,
    from -8 to 7 and shifted; the caller places the largest, 8 + shift."""
    x = np.zeros(shape)
    x[..., 0] = np.random.default_rng(seed).integers(-8, 8, shape[:-1]) + shift
    return x


@pytest.mark.parametrize("shift", [0, -16])
@pytest.mark.parametrize("v_mult", [1.0, 2.0 ** 30, 2.0 ** -40])
@pytest.mark.parametrize("exp", [16, 24, 27, 30, 40, 110])
def test_logits_beyond_the_precision_of_differences(exp, v_mult, shift):
    """Logits up to 2^exp in magnitude, exact up to the factor log2(e): one key
    leads by 2^(exp - 3) or more, so the row is that key's value. In fp32 the
    logits' spacing passes the weights' range (2^15) from 2^27 on."""
    lens = [1000, 33]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 4, 64, seed=11, v_mult=v_mult)
    q = torch.zeros_like(q)
    q[:, :, 0] = 2.0 ** exp  # scale 1/8: the leading key's logit is 2^exp (or -2^exp)
    k64 = one_hot_keys(values(kc, ks).shape, 12, shift)
    lead = [(int(table[0, 31]), 7), (int(table[1, 1]), 15)]
    for page, slot in lead:
        k64[page, slot, :, 0] = 8 + shift
    kc, ks = cache_from(k64.transpose(0, 2, 1, 3))
    args = (q, kc, vc, ks, vs, table, n)
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    # The weights besides the leading one's are 0; the output rounds once, the
    # leading weight and the fp32 accumulation below 2^-20.
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O)).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()


def test_large_values_under_a_dominant_key_without_value():
    """Pages of zero values (the smallest exponent) with a key that leaves the
    others no weight, then pages of large values: 0, not 0 * inf."""
    lens = [60000]  # six pages a run
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 2, 64, seed=13, v_mult=2.0 ** 20)
    q = torch.zeros_like(q)
    q[:, :, 0] = 16.0
    k64, v64 = np.zeros_like(values(kc, ks)), values(vc, vs)
    pages = table[0, ::4].long().numpy()
    k64[pages, 2, :, 0] = 96.0  # logit 192
    v64[pages] = 0.0
    kc, ks = cache_from(k64.transpose(0, 2, 1, 3))
    vc, vs = cache_from(v64.transpose(0, 2, 1, 3))
    o, lse = attn.attn_decode_paged_e4m3(*cuda(q, kc, vc, ks, vs, table, n))
    assert (o == 0).all()  # exp(-192) * 2^20 is no fp32 number
    assert (np.abs(lse.double().cpu().numpy() - (192 + np.log(len(pages)))) <= 1e-4).all()


def test_lengths_and_table_rewritten_just_before():
    """The kernel in front lets the decode start at once and rewrites lengths and
    table 50 us later."""
    args = decode_case([900, 40, 300], 2, 4, 128, seed=14)
    O, L = reference(*args)
    dev = cuda(*args)
    for i in (5, 6):
        old = torch.zeros_like(dev[i])
        now = dev[:i] + [old] + dev[i + 1:]
        attn.attn_decode_paged_e4m3(*now)  # warm: lines of the old contents
        attn.attn_selftest_delayed_copy(old.view(-1), dev[i].view(-1), delay_us=50)
        o, lse = attn.attn_decode_paged_e4m3(*now)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
    assert attn.attn_get_device_error() == 0
