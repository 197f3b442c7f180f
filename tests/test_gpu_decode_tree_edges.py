"""attn_decode_paged_tree with logits, weights and values at their numbers' ends, against
the definition in float64."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
from parity import check_lse, check_out
from test_gpu_decode_tree import Case, _built, put  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exp", [24, 27, 28, 29, 30, 31, 32, 35, 60, 100])
@pytest.mark.parametrize("g,draft", [(4, 20), (4, 50), (1, 100)])
def test_large_logits_of_every_mantissa(exp, g, draft):
    """Queries' factors with every mantissa, so that products lie anywhere between two fp32
    numbers. One key leads by 2^(exp - 3) or more: a row is that key's value."""
    c = Case([700, 3000], [draft, draft], 2, g, 64, seed=31)
    q = torch.arange(c.q.shape[0] * c.q.shape[1]).view(c.q.shape[:2])
    c.q.zero_()
    c.q[:, :, 0] = ((1 + q % 128 / 128.0) * 2.0 ** exp).to(torch.bfloat16)
    c.k.zero_()
    c.k[..., 0] = torch.randint(-8, 8, c.k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for b, j in ((0, 650), (1, 3)):
        put(c, c.k, b, j, 8, e=0)
    O, L = c.reference()
    o, lse = c.run()
    # (Half a bf16 step is up to 2^-8 of a number; a weight's rounding, 2^-15, moves the one
    # that the row is by less.)
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -24).all()
    # Factor, product, ln 2 and the product with it: 5 roundings of 2^-24.
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("exp", [10, 28, 31, 100])
def test_large_logits_that_are_equal(exp):
    """Leading keys in several tiles, of both streams and of several CTAs."""
    c = Case([20000], [20], 2, 4, 128, seed=32)
    q = torch.arange(160).view(20, 8)
    c.q.zero_()
    c.q[:, :, 0] = ((1 + q % 128 / 128.0) * 2.0 ** exp).to(torch.bfloat16)
    c.k.zero_()
    c.k[..., 0] = torch.randint(-8, 8, c.k.shape[:-1], generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for j in (100, 300, 350, 9000, 19990):
        put(c, c.k, 0, j, 8, e=0)
    O, L = c.reference()
    o, lse = c.run()
    # Half a bf16 step of the result, and 2^-14 of the values that are averaged.
    assert (np.abs(o.double().cpu().numpy() - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -14 * 6).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L) + 1e-6).all()


@pytest.mark.parametrize("gap", [6, 12, 17])
def test_one_key_outweighs_thousands(gap):
    """What thousands of keys hold together is not lost beside one that outweighs each of
    them by e^gap."""
    c = Case([8300], [9], 1, 4, 128, seed=33)
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.k.zero_()
    c.v[..., 0] = 1.0
    put(c, c.k, 0, 300, gap * 128 ** 0.5 / 8.0, e=0)
    put(c, c.v, 0, 300, 0.0, e=0)
    O, L = c.reference()
    o, lse = c.run()
    check_out(o, O, torch.bfloat16)
    check_lse(lse, L)
    # Half a bf16 step is up to 2^-8 of a number; a weight is within 2^-15 of itself.
    o, O = o[..., 0].double().cpu().numpy(), O[..., 0]
    assert (np.abs(o - O) <= (2.0 ** -8 + 2.0 ** -14) * O).all()


@pytest.mark.parametrize("exp", [-110, -60, 60, 105])
def test_values_of_any_size(exp):
    c = Case([300, 0], [15, 40], 2, 4, 64, seed=34)
    c.v = (c.v.double() * 2.0 ** exp).to(torch.bfloat16)
    O, L = c.reference()
    o, lse = c.run()
    check_out(o.double().cpu() * 2.0 ** -exp, O * 2.0 ** -exp, torch.bfloat16)
    check_lse(lse, L)
