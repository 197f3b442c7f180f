"""The 8-bit paged cache: attn_cache_write_e4m3 and attn_cache_read_e4m3 against
the format's definition in 64 bits. The scale is a power of two and each code is
one rounding of an exact product, so every comparison is for equality."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle.cache_e4m3 as ref
import workloads as W
from e4m3_cases import codes_to_f64, empty_cache, token_slots, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def rows_with_edges(shape, seed, dtype):
    """N(0,1) rows with the format's edges among them: zeros, the border
    between two exponents, halfway codes, tiny and huge magnitudes."""
    x = W.normal(shape, seed, torch.float32).view(-1, shape[-1])
    n = x.shape[0]
    x[0 % n] = 0.0
    x[1 % n] = 0.0
    x[1 % n, 3] = 448.0 * 2.0 ** -3                 # exactly the border
    x[2 % n] = x[2 % n].clamp(-1, 1)
    x[2 % n, 5] = 450.0 * 2.0 ** 4                  # just past it
    x[3 % n, :16] = torch.arange(16) + 16.5         # ties between codes once the row max is 448
    x[3 % n, 20] = 448.0
    x[4 % n] *= 2.0 ** -120
    x[5 % n] *= 2.0 ** -130
    x[6 % n] *= 2.0 ** 118
    x[7 % n, 7] = 3.3e38
    return x.view(shape).to(dtype)


def packed(B, new, old, seed):
    """Row lengths, cu, table, total and blocks of a ragged batch."""
    g = torch.Generator().manual_seed(seed)
    n_new = torch.randint(0, new + 1, (B,), generator=g).tolist()
    n_new[0] = new
    n_old = torch.randint(0, old + 1, (B,), generator=g).tolist()
    lens = [a + b for a, b in zip(n_new, n_old)]
    cu = [0]
    for n in n_new:
        cu.append(cu[-1] + n)
    table, nb = W.paged_layout(lens, seed, spare_pages=3)
    return lens, cu, table, nb


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,new,old,h_kv", [(1, 1, 0, 1), (1, 17, 30, 8), (5, 40, 100, 3), (70, 9, 33, 2)])
def test_write_matches_definition(B, new, old, h_kv, d, dtype):
    """Every byte of the four arrays: written slots by the definition, others
    (padding tokens behind the last sequence among the inputs) untouched."""
    lens, cu, table, nb = packed(B, new, old, seed=B + d)
    total = cu[-1] + 5  # five padding tokens
    qkv = rows_with_edges((total, 2 * h_kv + 1, d), 7, dtype).cuda()
    k, v = qkv[:, 1:1 + h_kv], qkv[:, 1 + h_kv:]  # slices of a fused projection
    kc, vc, ks, vs = empty_cache(nb, h_kv, d, fill=0x5a)
    attn.attn_cache_write_e4m3(k, v, kc, vc, ks, vs, table.cuda(), dev(cu), dev(lens))
    assert attn.attn_get_device_error() == 0
    slots = token_slots(cu, lens, table, total)
    for x, c, e in ((k, kc, ks), (v, vc, vs)):
        want_c, want_e = ref.quantise_ref(x.double().cpu().numpy())
        full_c = codes_to_f64(torch.full((nb, h_kv, 16, d), 0x5a, dtype=torch.uint8).view(torch.float8_e4m3fn))
        full_e = np.full((nb, h_kv, 16), 0x5a, np.uint8)
        for t, ps in enumerate(slots):
            if ps is not None:
                full_c[ps[0], :, ps[1]] = want_c[t]
                full_e[ps[0], :, ps[1]] = want_e[t]
        assert np.array_equal(e.cpu().numpy(), full_e)
        assert np.array_equal(codes_to_f64(c), full_c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_nonfinite_become_nan_and_leave_the_scale(dtype):
    x = W.normal((4, 2, 128), 3, dtype)
    x[0, 0, 5] = float("nan")
    x[1, 1, 7] = float("inf")
    x[2, 0, 9] = float("-inf")
    x[3, 1] = float("nan")
    kc, vc, ks, vs = empty_cache(1, 2, 128)
    attn.attn_cache_write_e4m3(x.cuda(), x.cuda(), kc, vc, ks, vs, dev([[0]]), dev([0, 4]), dev([4]))
    want_c, want_e = ref.quantise_ref(x.double().numpy())
    for c, e in ((kc, ks), (vc, vs)):
        got = codes_to_f64(c)[0].transpose(1, 0, 2)[:4]
        assert np.array_equal(np.isnan(got), np.isnan(want_c))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want_c))
        assert np.array_equal(e.cpu().numpy()[0].T[:4], want_e)


def test_write_bad_pages_and_positions_are_dropped_and_flagged():
    kc, vc, ks, vs = empty_cache(4, 1, 64, fill=1)
    x = W.normal((6, 1, 64), 1, torch.bfloat16).cuda()
    attn.attn_get_device_error()
    table = dev([[2, 9], [-3, 1]])  # row 0's second page and row 1's first lie outside the cache
    attn.attn_cache_write_e4m3(x, x, kc, vc, ks, vs, table, dev([0, 3, 6]), dev([17, 18]))
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    touched = (ks.cpu() != 1).nonzero().tolist()
    assert [t for t in touched if t[0] not in (1, 2)] == []
    assert touched == [[1, 0, 0], [1, 0, 1], [2, 0, 14], [2, 0, 15]]
    # positions before the row's start and past its table row
    kc, vc, ks, vs = empty_cache(4, 1, 64, fill=1)
    attn.attn_cache_write_e4m3(x, x, kc, vc, ks, vs, dev([[0, 1], [2, 3]]), dev([0, 3, 6]), dev([2, 34]))
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_SEQ_LEN
    assert (ks.cpu() != 1).nonzero().tolist() == [[0, 0, 0], [0, 0, 1], [3, 0, 15]]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("head_major", [False, True])
def test_read_returns_stored_values(d, dtype, head_major):
    """All codes with all kinds of exponents, tails of ragged rows; tokens
    behind the last sequence stay as they were."""
    B, h_kv = 6, 3
    lens, cu, table, nb = packed(B, 50, 40, seed=d)
    g = torch.Generator().manual_seed(5)
    kc, vc, ks, vs = empty_cache(nb, h_kv, d)
    for c, e in ((kc, ks), (vc, vs)):
        u = torch.randint(0, 256, c.shape, generator=g, dtype=torch.int64).to(torch.uint8)
        c.view(torch.uint8).copy_(torch.where((u & 0x7f) == 0x7f, torch.zeros_like(u), u))  # no NaN here
        e.copy_(torch.randint(10, 247, e.shape, generator=g).to(torch.uint8))
    total = cu[-1] + 4
    shape = (h_kv, total, d) if head_major else (total, h_kv, d)
    k, v = (torch.full(shape, -7.0, dtype=dtype, device="cuda") for _ in range(2))
    kk, vv = (t.transpose(0, 1) if head_major else t for t in (k, v))
    attn.attn_cache_read_e4m3(kc, vc, ks, vs, table.cuda(), dev(cu), dev(lens), kk, vv)
    assert attn.attn_get_device_error() == 0
    for out, c, e in ((kk, kc, ks), (vv, vc, vs)):
        val = values(c, e)
        want = np.full((total, h_kv, d), -7.0)
        for t, ps in enumerate(token_slots(cu, lens, table, total)):
            if ps is not None:
                want[t] = val[ps[0], ps[1]]
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_read_bad_page_reads_zeros_and_nan_codes_stay_nan():
    kc, vc, ks, vs = empty_cache(2, 1, 64, fill=0x7f)  # NaN codes, scale 1
    k = torch.full((34, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    attn.attn_get_device_error()
    attn.attn_cache_read_e4m3(kc, vc, ks, vs, dev([[0, 7, 1]]), dev([0, 34]), dev([34]), k, v)
    assert attn.attn_get_device_error() == attn.ATTN_DEVERR_BAD_PAGE
    for t in (k, v):
        assert torch.isnan(t[:16].float()).all() and torch.isnan(t[32:].float()).all()
        assert (t[16:32] == 0).all()


def test_write_then_read_is_the_nearest_stored_value():
    """Through both calls a value moves by at most half an e4m3 step, 2^-4 of
    it, or half the smallest step 2^(e - 10); written values read back and
    written again do not move."""
    x = W.normal((100, 4, 128), 9, torch.bfloat16).cuda()
    table, nb = W.paged_layout([100], 2)
    cu, lens, table = dev([0, 100]), dev([100]), table.cuda()
    cache = empty_cache(nb, 4, 128)
    attn.attn_cache_write_e4m3(x, x, *cache, table, cu, lens)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    attn.attn_cache_read_e4m3(*cache, table, cu, lens, y, y2)
    assert torch.equal(y, y2)
    e = torch.log2(x.float().abs().amax(-1, keepdim=True) / 448).ceil()
    assert ((x.float() - y.float()).abs() <= torch.maximum(x.float().abs() * 2.0 ** -4, 2.0 ** (e - 10))).all()
    again = empty_cache(nb, 4, 128)
    attn.attn_cache_write_e4m3(y, y, *again, table, cu, lens)
    z, z2 = torch.empty_like(x), torch.empty_like(x)
    attn.attn_cache_read_e4m3(*again, table, cu, lens, z, z2)
    assert torch.equal(y, z) and torch.equal(y, z2)


def test_far_pages_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^31 (and 2^32 elements over both heads' runs)."""
    nb, h_kv, d = 150000, 8, 128
    assert nb * h_kv * 16 * d > 2 ** 31
    kc = torch.empty((nb, h_kv, 16, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks = torch.empty((nb, h_kv, 16), dtype=torch.uint8, device="cuda")
    vc, vs = torch.empty_like(kc), torch.empty_like(ks)
    x = W.normal((40, h_kv, d), 11, torch.bfloat16).cuda()
    table = dev([[nb - 1, 3, nb - 2]])
    attn.attn_cache_write_e4m3(x, x, kc, vc, ks, vs, table, dev([0, 40]), dev([40]))
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    attn.attn_cache_read_e4m3(kc, vc, ks, vs, table, dev([0, 40]), dev([40]), y, y2)
    c, e = ref.quantise_ref(x.double().cpu().numpy())
    want = ref.values_ref(c, e)
    assert np.array_equal(y.double().cpu().numpy(), want) and np.array_equal(y2.double().cpu().numpy(), want)
    q = W.normal((1, 32, d), 12, torch.bfloat16)
    o, lse = attn.attn_decode_paged_e4m3(q.cuda(), kc, vc, ks, vs, table, dev([40]))
    s = np.einsum("hgd,nhd->hgn", q[0].double().numpy().reshape(h_kv, 4, d), want) / d ** 0.5
    p = np.exp(s - s.max(-1, keepdims=True))
    from parity import check_lse, check_out

    check_out(o[0], (np.einsum("hgn,nhd->hgd", p, want) / p.sum(-1)[..., None]).reshape(32, d), torch.bfloat16)
    check_lse(lse[0], (s.max(-1) + np.log(p.sum(-1))).reshape(32))
    assert attn.attn_get_device_error() == 0


def test_binding_refuses():
    """What the compiled binding checks before it calls the library."""
    x = W.normal((20, 2, 64), 1, torch.bfloat16).cuda()
    kc, vc, ks, vs = empty_cache(3, 2, 64)
    good = dict(k=x, v=x, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=dev([[0, 2]]),
                cu_seqlens=dev([0, 20]), seq_lens=dev([20]))
    for fn in (attn.attn_cache_write_e4m3, attn.attn_cache_read_e4m3):
        fn(**good)
        wide = torch.zeros((20, 2, 128), dtype=torch.bfloat16, device="cuda")
        for kw in (dict(k=x.half()), dict(v=x.float()), dict(k=x.cpu()), dict(k=x[:, :1]), dict(k=x[:10]),
                   dict(k=wide[:, :, ::2], v=wide[:, :, ::2]), dict(k_cache=kc.view(torch.uint8)),
                   dict(v_cache=vc[:2]), dict(k_scale=ks[:, :1]), dict(v_scale=vs.cpu()),
                   dict(block_table=dev([0, 2])), dict(cu_seqlens=dev([0, 20, 20])), dict(cu_seqlens=dev([0, 20]).long()),
                   dict(seq_lens=dev([[20]]))):
            with pytest.raises(ValueError):
                fn(**{**good, **kw})
        odd = torch.zeros(20 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 2560].view(20, 2, 64)
        with pytest.raises(attn.AttnError):  # rows not on 16 bytes
            fn(**{**good, "k": odd})
        loose = torch.zeros((20, 2, 68), dtype=torch.bfloat16, device="cuda")[:, :, :64]
        with pytest.raises(attn.AttnError):
            fn(**{**good, "v": loose})
    assert attn.attn_get_device_error() == 0


def test_offsets_lengths_and_table_rewritten_just_before():
    """The kernel in front lets the write (the read) start at once and rewrites
    one of table, offsets and lengths 50 us later."""
    lens, h_kv, d = [40, 100, 7], 2, 128
    table, nb = W.paged_layout(lens, seed=31)
    cu = torch.tensor([0, 40, 140, 147], dtype=torch.int32)
    where = [table.cuda(), cu.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()]
    k, v = (W.normal((147, h_kv, d), 40 + i, torch.bfloat16).cuda() for i in range(2))
    cache = empty_cache(nb, h_kv, d)
    attn.attn_cache_write_e4m3(k, v, *cache, *where)
    back = attn.attn_cache_read_e4m3(*cache, *where, torch.empty_like(k), torch.empty_like(v))
    for i in range(3):
        for read in (False, True):
            old = torch.zeros_like(where[i])
            now = where[:i] + [old] + where[i + 1:]
            fresh = empty_cache(nb, h_kv, d)
            out = [torch.zeros_like(k), torch.zeros_like(v)]
            attn.attn_cache_read_e4m3(*cache, *now, torch.empty_like(k), torch.empty_like(v))  # warm
            attn.attn_get_device_error()
            attn.attn_selftest_delayed_copy(old.view(-1), where[i].view(-1), delay_us=50)
            if read:
                attn.attn_cache_read_e4m3(*cache, *now, *out)
                assert torch.equal(out[0], back[0]) and torch.equal(out[1], back[1])
            else:
                attn.attn_cache_write_e4m3(k, v, *fresh, *now)
                for a, b in zip(fresh, cache):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert attn.attn_get_device_error() == 0


def test_more_tokens_than_one_grid_dimension_holds():
    """Two rows of over half a million tokens each, the same thousand repeated:
    written and read back through blocks beyond 65535."""
    base, n = 1000, 65535 * 16 + 1000
    k0, v0 = (W.normal((base, 1, 64), 60 + i, torch.bfloat16) for i in range(2))
    k, v = (t.repeat(n // base + 1, 1, 1)[:n].contiguous().cuda() for t in (k0, v0))
    lens = [n // 2 + 3, n - n // 2 - 3]
    pages = [(x + 15) // 16 for x in lens]
    table = torch.full((2, max(pages)), -1, dtype=torch.int32)
    table[0, :pages[0]] = torch.arange(pages[0], dtype=torch.int32)
    table[1, :pages[1]] = torch.arange(pages[0], sum(pages), dtype=torch.int32).flip(0)
    cache = empty_cache(sum(pages), 1, 64)
    where = (table.cuda(), torch.tensor([0, lens[0], n], dtype=torch.int32).cuda(),
             torch.tensor(lens, dtype=torch.int32).cuda())
    attn.attn_cache_write_e4m3(k, v, *cache, *where)
    outs = attn.attn_cache_read_e4m3(*cache, *where, torch.empty_like(k), torch.empty_like(v))
    for x0, out in zip((k0, v0), outs):
        want = torch.from_numpy(ref.values_ref(*ref.quantise_ref(x0.double().numpy()))).to(torch.bfloat16).cuda()
        assert torch.equal(out, want.repeat(n // base + 1, 1, 1)[:n])
    assert attn.attn_get_device_error() == 0
