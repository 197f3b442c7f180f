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
    # The weight's rounding (2^-12) cancels in part against the sum's; bf16's is 2^-9.
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
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -9 * np.abs(O) + 2.0 ** -11 * 6).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L) + 1e-6).all()


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
