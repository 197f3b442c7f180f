"""attn_decode_paged_window_e4m3 with NaN codes and any exponents in and out of sight,
and both windowed decodes over tables much wider than the rows, in either form of the
kernel (few rows: a cluster per unit; many: runs)."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
from masked_cases import window_seen
from parity import check_lse, check_lse_nonfinite, check_nonfinite, check_out
from test_gpu_decode_window import _built, case, reference, run  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu

NAN_CODE = 0x7f


def raw(codes):
    return codes.view(torch.uint8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[200, 47, 133], [200] * 20])
def test_8_bit_slots_out_of_sight_never_reach_a_row(lens, d):
    window, sinks = 40, 5
    args = case(lens, 2, 4, d, 11, 10 ** 6, 0, True)
    O, L = reference(args, window, sinks)
    q, kc, vc, ks, vs, tab, n = args
    for b, m in enumerate(lens):
        hidden = np.append(~window_seen(1, m, window, sinks)[0], [True] * (-m % 16))
        for j in np.nonzero(hidden)[0]:
            page, slot = int(tab[b, j // 16]), j % 16
            raw(kc)[page, :, slot] = NAN_CODE if j % 2 else 0xff
            raw(vc)[page, :, slot] = NAN_CODE if j % 3 else 0x7e
            ks[page, :, slot] = 255 if j % 5 else 0
            vs[page, :, slot] = 255 if j % 7 else 254
    o, lse = run(args, window, sinks)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("lens", [[100] * 3, [100] * 20])
def test_8_bit_nan_codes_in_sight(lens):
    window, sinks = 30, 3
    args = case(lens, 2, 2, 64, 12, window, sinks, True)
    q, kc, vc, ks, vs, tab, n = args
    raw(vc)[int(tab[0, 0]), 1, 2, 5] = NAN_CODE   # a sink of row 0, KV head 1
    raw(kc)[int(tab[1, 5]), 0, 3, 0] = NAN_CODE   # in row 1's window, KV head 0
    raw(vc)[int(tab[2, 6]), 0, 3, 9] = 0xff       # row 2's own key
    with np.errstate(invalid="ignore"):
        O, L = reference(args, window, sinks)
    o, lse = run(args, window, sinks)
    assert check_nonfinite(o, O, torch.bfloat16) > 0
    check_lse_nonfinite(lse, L)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("lens", [[2000, 0, 33], [700, 1500] * 20])
def test_table_much_wider_than_the_rows(lens, eight):
    window, sinks = 500, 4
    args = case(lens, 1, 4, 128, 13, window, sinks, eight)
    O, L = reference(args, window, sinks)
    tab = args[-2]
    args[-2] = torch.cat([tab, tab.new_full((len(lens), 8192 - tab.shape[1]), 2 ** 31 - 1)], 1)
    o, lse = run(args, window, sinks)
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("exp", [-110, -40, 40, 110])
@pytest.mark.parametrize("lens", [[300, 80], [300, 80] * 10])
def test_values_of_any_size(exp, lens):
    """The bf16 cache's values enter as they are."""
    window, sinks = 100, 4
    args = case(lens, 2, 4, 64, 14, window, sinks)
    args[2] = (args[2].double() * 2.0 ** exp).to(torch.bfloat16)
    O, L = reference(args, window, sinks)
    o, lse = run(args, window, sinks)
    check_out(o.double().cpu() * 2.0 ** -exp, O * 2.0 ** -exp, torch.bfloat16)
    check_lse(lse, L)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("exp", [24, 28, 30, 31, 32, 35, 60, 100])
@pytest.mark.parametrize("rows", [1, 16])
def test_large_logits_of_every_mantissa(exp, rows, eight):
    """Queries' factors with every mantissa, so that products lie anywhere between two fp32
    numbers. One visible key leads: a row is that key's value."""
    window, sinks, n = 600, 4, 1000
    for at in range(0, 128, 8 * rows):
        args = case([n] * rows, 2, 4, 64, 15, 10 ** 6, 0, eight)
        q, k = args[0], args[1]
        q.zero_()
        q[:, :, 0] = ((1 + (at + torch.arange(rows * 8)).view(rows, 8) / 128.0) * 2.0 ** exp).to(torch.bfloat16)
        lead = args[-2][:, 950 // 16].long()
        if eight:  # codes 0 to 7 and 8, exponent 0
            codes = torch.zeros(k.shape)
            codes[..., 0] = torch.randint(-8, 8, k.shape[:-1], generator=torch.Generator().manual_seed(1)).float()
            codes[lead, :, 950 % 16, 0] = 8
            args[1] = codes.to(torch.float8_e4m3fn)
            args[3].fill_(127)
        else:
            k.zero_()
            k[..., 0] = torch.randint(-8, 8, k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
            k[lead, 950 % 16, :, 0] = 8
        O, L = reference(args, window, sinks)
        o, lse = run(args, window, sinks)
        # (Half a bf16 step is up to 2^-8 of a number; a weight's rounding moves the one that
        # the row is by less.)
        assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
        # Factor, product, ln 2 and the product with it, the keys' exponent: 6 roundings of 2^-24.
        assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()
