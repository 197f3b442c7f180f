"""attn_prefill_paged_window at its numbers' and sizes' ends, against the definition in
float64: logits of any size, values of any size, many tiles with values that fp16 does
not hold, tables much wider than the rows. Where parity.py's tolerances do not serve,
the bound is derived beside the check."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
from masked_cases import i32
from parity import check_lse, check_out
from test_gpu_prefill_window import Case, _built  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu


def put(c, cache, b, j, value, kv=slice(None), e=slice(None)):
    cache[int(c.table[b, j // 16]), j % 16, kv, e] = value


def leading(exp, leads, mult, window, sinks, d, seed=20):
    """Row 0: 720 keys, 20 queries; row 1: 60 keys, 40 queries. Keys' logits are integers
    times 2^exp * mult; those of `leads` (row, key) are all rows' largest."""
    c = Case([700, 20], [20, 40], 2, 4, d, seed, window, sinks)
    c.q.zero_()
    c.q[:, :, 0] = mult * 2.0 ** exp
    c.k.zero_()
    low, high = (-8, 8) if mult > 0 else (2, 9)
    c.k[..., 0] = torch.randint(low, high, c.k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for b, j in leads:
        put(c, c.k, b, j, 8 if mult > 0 else 1, e=0)
    return c


@pytest.mark.parametrize("exp", [10, 25, 27, 28, 29, 30, 33, 60, 100])
@pytest.mark.parametrize("mult", [1, -1, 1.25])
@pytest.mark.parametrize("window,sinks,flagged", [(300, 4, False), (300, 4, True), (300, 40, False), (1000, 0, False),
                                                  (1000, 0, True)])
def test_large_logits(exp, mult, window, sinks, flagged):
    """One key leads by 2^(exp - 3) or more: the row is that key's value. (With 4 sinks the
    first tile is a narrow one; `flagged`: tiles that keep two-term weights.)"""
    c = leading(exp, ((0, 650), (1, 3)), mult, window, sinks, 64)
    if flagged:  # values that weigh nothing
        put(c, c.v, 0, 500, 3e5)
        put(c, c.v, 0, 1, -3e5)
        put(c, c.v, 1, 1, 3e5)
    O, L = c.reference()
    o, lse = c.run()
    # (Half a bf16 step is up to 2^-8 of a number; a weight's rounding, 2^-12, moves the one
    # that the row is by less.)
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("exp", [10, 26, 27, 28, 31, 100])
@pytest.mark.parametrize("flagged", [False, True])
@pytest.mark.parametrize("window,sinks,leads", [(300, 4, ((0, 2), (0, 650))), (300, 40, ((0, 2), (0, 650))),
                                                (1000, 0, ((0, 100), (0, 300), (0, 650)))])
def test_large_logits_that_are_equal(exp, window, sinks, leads, flagged):
    """Leading keys in several tiles, their weights equal whatever the logits' size."""
    c = leading(exp, leads + ((1, 3),), 1, window, sinks, 128)
    if flagged:
        put(c, c.v, 0, 640, 3e5)
        put(c, c.v, 0, 1, 3e5)
    O, L = c.reference()
    o, lse = c.run()
    # Half a bf16 step of the result, and 2^-11 of the values that are averaged.
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -11 * 6).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L) + 1e-6).all()


@pytest.mark.parametrize("exp", range(24, 34))
@pytest.mark.parametrize("window,sinks,flagged", [(300, 4, False), (300, 40, False), (1000, 0, True)])
def test_large_logits_of_every_mantissa(exp, window, sinks, flagged):
    """160 queries' factors, so that products lie anywhere between two fp32 numbers."""
    c = leading(exp, ((0, 650), (1, 3)), 1, window, sinks, 64)
    c.q[:, :, 0] = ((1 + torch.arange(c.q.shape[0] * 8) % 128 / 128.0) * 2.0 ** exp).view(-1, 8).to(torch.bfloat16)
    if flagged:
        put(c, c.v, 0, 500, 3e5)
        put(c, c.v, 1, 1, 3e5)
    O, L = c.reference()
    o, lse = c.run()
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()  # as above
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()


@pytest.mark.parametrize("exp", range(20, 30))
def test_logits_that_rise_by_steps(exp):
    """Each tile's logits pass the tile before by 15 to 17 in log2 units, at sizes whose
    spacing is 1/8 to 32: weights stay within fp16, and the rows are averages of values."""
    for step in (15, 16, 17):
        c = Case([900], [128], 1, 2, 64, 21, 1000, 0)
        c.q.zero_()
        c.q[:, :, :2] = 1.0
        c.k.zero_()
        for j in range(1028):
            put(c, c.k, 0, j, 2.0 ** exp, e=0)
            put(c, c.k, 0, j, float(step * (j // 128)), e=1)
        o, lse = c.run(scale=float(np.log(2.0)))
        o = o.double().cpu()
        # (2^-11: a weight's rounding and the sum's; 2^-9: bf16's.)
        assert torch.isfinite(o).all() and o.abs().max() <= c.v.double().abs().max() * (1 + 2.0 ** -8), (exp, step)
        want = 2.0 ** exp * np.log(2.0)
        assert ((lse.double().cpu() - want).abs() <= want * 2.0 ** -20 + 130).all(), (exp, step)


def outweighed(window, sinks, lead, gap, steps=0):
    """8300 keys and 40 queries; every key's logit is 0 but the lead's, `gap`, and with
    `steps` one key's in 128, gap - steps. The leads have the value 0, the others 1 in
    column 0."""
    c = Case([8300], [40], 1, 2, 128, 30, window, sinks)
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.k.zero_()
    c.v[..., 0] = 1.0
    for j in range(64, 8300, 128) if steps else ():
        put(c, c.k, 0, j, (gap - steps) * 128 ** 0.5 / 8.0, e=0)
        put(c, c.v, 0, j, 0.0, e=0)
    put(c, c.k, 0, lead, gap * 128 ** 0.5 / 8.0, e=0)
    put(c, c.v, 0, lead, 0.0, e=0)
    return c


@pytest.mark.parametrize("gap", [6, 10, 12, 13, 14, 17])
@pytest.mark.parametrize("window,sinks,lead,steps", [(8192, 4, 1, 0), (8000, 4, 1, 0), (8000, 100, 99, 0), (8192, 0, 300, 0),
                                                     (8000, 0, 8200, 0), (8000, 4, 1, 3), (8192, 0, 300, 3)])
def test_one_key_outweighs_thousands(window, sinks, lead, steps, gap):
    """What thousands of keys hold together is not lost beside one that outweighs each of
    them by e^gap, a sink or any other."""
    c = outweighed(window, sinks, lead, gap, steps)
    O, L = c.reference()
    o, lse = c.run()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    # Half a bf16 step is up to 2^-8 of a number; a weight's rounding to fp16 2^-12 of itself,
    # and at most 2^-29 of the row's largest (2^-25 of a sink's).
    lost = 8192 * 2.0 ** (-25 if lead < sinks else -29)
    o, O = o[..., 0].double().cpu().numpy(), O[..., 0]
    assert (np.abs(o - O) <= (2.0 ** -8 + 2.0 ** -12) * O + lost).all()


@pytest.mark.parametrize("window,sinks", [(700, 3), (2000, 0), (300, 400)])
def test_infinities_that_every_query_of_a_tile_sees(window, sinks):
    """An infinity in a tile that all of a block's queries see reaches them as an
    infinity, also where another tile's NaN is put into their rows at the end."""
    c = Case([1000], [128], 2, 4, 128, 23, window, sinks)
    inside, edge = 640, 1050  # (tile 5 of each query's keys; the tile that ends them)
    put(c, c.v, 0, inside, float("inf"), kv=1, e=7)
    put(c, c.v, 0, edge, float("nan"), kv=1, e=9)
    some = edge - 1000
    put(c, c.v, 0, 1000, 3e5, kv=1, e=11)
    o, lse = c.run()
    o = o.float().cpu()[:, 4:]  # KV head 1
    # (A weight whose second bf16 term is 0, one in 2^8, gives 0 * inf; no other NaN.)
    assert (o[..., 7] == float("inf")).float().mean() > 0.9 and not torch.isfinite(o[..., 7]).any()
    assert torch.isnan(o[some:, :, 9]).all() and torch.isfinite(o[:some, :, 9]).all()
    keep = [e for e in range(128) if e not in (7, 9)]
    assert torch.isfinite(o[..., keep]).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("window,sinks", [(60000, 0), (500, 40000)])
def test_one_nan_among_many_flagged_tiles(window, sinks):
    """Each V tile holds a value that fp16 does not, and one tile that some queries see in
    part a NaN: looked for there alone, in far less than the waits' 2 s."""
    c = Case([60000], [70], 1, 2, 128, 24, window, sinks)
    c.v[:, ::5, :, 3] = 1e5
    put(c, c.v, 0, 60030, float("nan"), e=5)
    o, lse = c.run()
    assert attn.attn_get_device_error() == 0
    o = o.float().cpu()
    assert torch.isnan(o[30:, :, 5]).all() and torch.isfinite(o[:30]).all()
    assert torch.isfinite(o[30:][..., [e for e in range(128) if e != 5]]).all()
    e0, e1 = torch.cuda.Event(True), torch.cuda.Event(True)
    args = c.args()
    e0.record()
    attn.attn_prefill_paged_window(*args, c.window, c.sinks, c.max_q)
    e1.record()
    torch.cuda.synchronize()
    assert e0.elapsed_time(e1) < 100


@pytest.mark.parametrize("exp", [-120, -60, -30, -22, -20, -16, 7, 9, 60, 64, 66, 100, 118])
@pytest.mark.parametrize("window,sinks", [(100, 3), (400, 0)])
def test_values_of_any_size(exp, window, sinks):
    """Values enter exactly: the same bound at every magnitude."""
    c = Case([300, 0], [150, 140], 1, 4, 128, 25, window, sinks)
    c.v = (c.v.double() * 2.0 ** exp).to(torch.bfloat16)
    O, L = c.reference()
    o, lse = c.run()
    check_out(o.double().cpu() * 2.0 ** -exp, O * 2.0 ** -exp, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("low,high", [(-30, 0), (-60, 3), (-24, 12), (-100, 100), (0, 118), (-25, 8)])
def test_columns_of_different_size(low, high):
    """Every other column 2^low, the others 2^high: each within its own bound."""
    c = Case([500, 30], [200, 140], 2, 2, 64, 26, 300, 4)
    size = torch.full((64,), 2.0 ** high, dtype=torch.float64)
    size[::2] = 2.0 ** low
    c.v = (c.v.double() * size).to(torch.bfloat16)
    O, L = c.reference()
    o, lse = c.run()
    check_out(o.double().cpu() / size, O / size.numpy(), torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("lead", [2, 640])
@pytest.mark.parametrize("exp", [-118, -40, -24, -20, 0, 30, 120])
@pytest.mark.parametrize("gap", [10, 13])
def test_the_leading_key_alone_has_a_small_or_large_value(lead, exp, gap):
    """A row is its leading key's value, whatever the others' sizes."""
    c = leading(gap, ((0, lead), (1, 3)), 1, 300, 4, 128)
    c.v = (c.v.float() * torch.where(torch.arange(16) % 3 == 0, 1e4, 1e-3)[:, None, None]).to(torch.bfloat16)
    for b, j in ((0, lead), (1, 3)):
        put(c, c.v, b, j, (torch.linspace(-1.9, 1.9, 128) * 2.0 ** exp).to(torch.bfloat16))
    O, L = c.reference()
    o, lse = c.run()
    # (As for large logits.) The other keys' logits are 2^gap / sqrt(128) or more below, so
    # their weights are zeros in fp16: at most 720 values of 4.5e4 at e^-that are lost (2^10:
    # e^-90.5, 2e-32 in all).
    lost = 720 * 4.5e4 * np.exp(-2.0 ** gap / 128 ** 0.5)
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + lost).all()


@pytest.mark.parametrize("exp", [17, 63, 64, 120])
def test_one_large_value_leaves_the_other_columns_alone(exp):
    c = Case([200], [200], 2, 2, 64, 27, 130, 4)
    O, L = c.reference()
    for j in (1, 150, 330, 399):
        put(c, c.v, 0, j, 2.0 ** exp, kv=1, e=7)
    o, lse = c.run()
    others = [e for e in range(64) if e != 7]
    check_out(o[..., others], O[..., others], torch.bfloat16)
    check_out(o[:, :2], O[:, :2], torch.bfloat16)
    check_lse(lse, L)
    P, _ = c.reference()
    o = o[..., 7].double().cpu().numpy()
    assert (np.abs(o - P[..., 7])[:, 2:] <= 2.0 ** -7 * np.abs(P[..., 7])[:, 2:] + 4e-3).all()


def test_every_bf16_number_as_a_value():
    """All 65280 finite numbers, each the only key that its query weighs."""
    c = Case([0], [4], 1, 1, 64, 28, 1, 0)
    n = 1020
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7f80) != 0x7f80].to(torch.int16).view(torch.bfloat16)
    v = bits.view(n, 64)
    pages = (n + 15) // 16
    vc = torch.zeros((pages * 16, 1, 64), dtype=torch.bfloat16)
    vc[:n, 0] = v
    kc = torch.zeros((pages, 16, 1, 64), dtype=torch.bfloat16).cuda()
    q = torch.zeros((n, 1, 64), dtype=torch.bfloat16).cuda()
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    o, lse = attn.attn_prefill_paged_window(q, kc, vc.view(pages, 16, 1, 64).cuda(), table, i32([0, n]).cuda(),
                                            i32([n]).cuda(), 1, 0, n)
    o, want = o[:, 0].double().cpu(), v.double()
    normal = want.abs() >= 2.0 ** -126  # (bf16 subnormals may come out as zeros)
    assert torch.equal(o[normal], want[normal])
    assert (o[~normal].abs() <= 2.0 ** -126).all()
    assert torch.equal(lse.cpu(), torch.zeros_like(lse.cpu()))


def test_table_much_wider_than_the_rows():
    """Rows of 1 to 2000 keys in a table of 8192 pages: the results of a tight table."""
    c = Case([700, 0, 1500, 33], [300, 1, 500, 7], 1, 4, 128, 29, 1024, 4)
    want, lse_w = c.check()
    c.table = torch.cat([c.table, c.table.new_full((4, 8192 - c.table.shape[1]), 2 ** 31 - 1)], 1)
    o, lse = c.run()
    assert torch.equal(o, want) and torch.equal(lse, lse_w)
    assert attn.attn_get_device_error() == 0
