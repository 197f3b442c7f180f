"""attn_cache_write_e4m3 and attn_cache_read_e4m3 at the edges of what their
arguments allow. Comparisons are for equality, as in test_gpu_cache_e4m3.py."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
import workloads as W
from e4m3_cases import empty_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
def test_inputs_rewritten_just_before(d):
    """The kernel in front lets the read (the write) start at once and rewrites
    codes or exponents (keys or values) 50 us later."""
    lens, h_kv = [40, 100, 7], 2
    table, nb = W.paged_layout(lens, seed=31)
    where = [table.cuda(), dev([0, 40, 140, 147]), dev(lens)]
    k, v = (W.normal((147, h_kv, d), 40 + i, torch.bfloat16).cuda() for i in range(2))
    cache = empty_cache(nb, h_kv, d)
    attn.attn_cache_write_e4m3(k, v, *cache, *where)
    back = attn.attn_cache_read_e4m3(*cache, *where, torch.empty_like(k), torch.empty_like(v))
    words = lambda t: t.view(torch.uint8).view(-1).view(torch.int32)
    for i in range(4):
        old = torch.full_like(cache[i].view(torch.uint8), 0x30).view(cache[i].dtype)
        now = list(cache[:i]) + [old] + list(cache[i + 1:])
        out = [torch.zeros_like(k), torch.zeros_like(v)]
        attn.attn_cache_read_e4m3(*now, *where, *out)  # warm: lines of the old contents
        attn.attn_selftest_delayed_copy(words(old), words(cache[i]), delay_us=50)
        attn.attn_cache_read_e4m3(*now, *where, *out)
        assert torch.equal(out[0], back[0]) and torch.equal(out[1], back[1])
    for i in range(2):
        src = [k, v]
        old = torch.full_like(src[i], 3.0)
        now = src[:i] + [old] + src[i + 1:]
        fresh = empty_cache(nb, h_kv, d)
        attn.attn_cache_write_e4m3(*now, *fresh, *where)
        attn.attn_selftest_delayed_copy(words(old), words(src[i]), delay_us=50)
        attn.attn_cache_write_e4m3(*now, *fresh, *where)
        for a, b in zip(fresh, cache):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("B", [1, 31, 32, 33, 64, 1024, 1025, 5000])
@pytest.mark.parametrize("most", [1, 3, 40])
def test_many_rows_with_and_without_tokens(B, most):
    """Rows of 0 to `most` tokens, runs of over a hundred rows without any: each
    token's values at its row's last positions, none elsewhere."""
    g = torch.Generator().manual_seed(B + most)
    new = torch.randint(0, most + 1, (B,), generator=g)
    for at in range(0, B, 300):
        new[at + 20:at + 150] = 0
    new[-1] = 1
    old = torch.randint(0, 20, (B,), generator=g)
    lens = new + old
    table, nb = W.paged_layout(lens.tolist(), seed=3, spare_pages=1)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    total = int(cu[-1])
    # every token its own value: one code per digit of its number, scale 2^0 by a largest of 448
    x = torch.zeros((total + 5, 1, 64))
    n = torch.arange(total + 5)
    for i in range(5):
        x[:, 0, i] = (n // 8 ** i) % 8
    x[:, 0, 5] = 448.0
    x = x.to(torch.bfloat16).cuda()
    cache = empty_cache(nb, 1, 64)
    where = (table.cuda(), cu.to(torch.int32).cuda(), lens.to(torch.int32).cuda())
    attn.attn_cache_write_e4m3(x, -x, *cache, *where)
    row = torch.repeat_interleave(torch.arange(B), new)
    pos = lens[row] - cu[row + 1] + torch.arange(total)
    page = table[row, pos // 16].long()
    want = torch.zeros((nb, 16, 64))
    want[page, pos % 16] = x[:total, 0].float().cpu()
    assert torch.equal(cache[0][:, 0].float().cpu(), want)
    assert torch.equal(cache[1][:, 0].float().cpu(), -want)
    k, v = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    attn.attn_cache_read_e4m3(*cache, *where, k, v)
    assert torch.equal(k[:total], x[:total]) and torch.equal(v[:total], -x[:total])
    assert (k[total:] == 9).all() and (v[total:] == 9).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("total,h_kv", [(1, 3), (20, 1), (1, 1)])
def test_strides_of_dimensions_of_one_element(total, h_kv, dtype):
    """Where there is one token (one head) its stride is never used: any value does,
    as in a slice of a wider or padded tensor."""
    d = 64
    x = W.normal((total, h_kv, d), 5, dtype).cuda()
    tok = h_kv * d if total > 1 else 1021
    head = d if h_kv > 1 else 333
    odd = lambda t: torch.as_strided(t, t.shape, (tok, head, 1))
    where = (dev([[1, 0]]), dev([0, total]), dev([total]))
    want, got = empty_cache(2, h_kv, d), empty_cache(2, h_kv, d)
    attn.attn_cache_write_e4m3(x, -x, *want, *where)
    attn.attn_cache_write_e4m3(odd(x.clone()), odd(-x), *got, *where)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    k, v = torch.empty_like(x), torch.empty_like(x)
    attn.attn_cache_read_e4m3(*want, *where, k, v)
    k2, v2 = torch.empty_like(x), torch.empty_like(x)
    attn.attn_cache_read_e4m3(*want, *where, odd(k2), odd(v2))
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert attn.attn_get_device_error() == 0
