"""attn_decode_paged_shared where values of very different sizes meet, and where a
lost or doubled page of values would show. Oracle and cases are those of
test_gpu_decode_shared.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
from parity import check_lse
from test_gpu_decode_shared import case, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def check_by_column(o, O, mag):
    """Relative to each output's own column: mag is the oracle's result over |V|.
    The output's rounding is 2^-8 of it, a weight's 2^-12 (one fp16 number; the
    two-term bf16 form is finer) of its value's share of mag, and q, K, the
    exponential and the sums in 32 bits stay below as much again."""
    err = np.abs(o.double().cpu().numpy() - O)
    tol = 2.0 ** -8 * np.abs(O) + 2.0 ** -11 * mag
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))


def magnitudes(args):
    return reference(args[0], args[1], args[2].abs(), *args[3:])[0]


# 3 rows of 4 heads share the key tiles in turn (two accumulators), 40 rows take two
# row tiles.
ROWS = pytest.mark.parametrize("B", [3, 40])


@ROWS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["all", "first", "middle", "last", "two", "own"])
def test_values_near_the_largest_numbers(where, d, B):
    """Values around 2^120, in every key tile, in some among ordinary ones, or among
    the rows' own keys only: weighted sums stay numbers wherever the result is one."""
    prefix = 900
    args = case(prefix, [33, 0] + [5] * (B - 2), 2, 4, d, seed=31)
    v, ptab, tab = args[2], args[3], args[5]
    big = 2.0 ** 120
    pages = {"all": range(57), "first": [1], "middle": [20], "last": [56], "two": [9, 40], "own": []}[where]
    for p in pages:
        v[int(ptab[p])] *= big
    if where in ("all", "own"):
        v[int(tab[0, 1])] *= big
    O, L = reference(*args)
    o, lse = run(args)
    assert torch.isfinite(o.float()).all()
    check_by_column(o, O, magnitudes(args))
    check_lse(lse, L)


@pytest.mark.parametrize("prefix,own", [(1, 0), (200, 0), (1, 3)])
def test_one_value_next_to_the_largest_number(prefix, own):
    """A key that takes all the weight has the value 1.5 * 2^127 in one column."""
    args = case(prefix, [own, own], 1, 4, 64, seed=33)
    q, k, v, ptab = args[:4]
    q.zero_()
    q[:, :, 0] = 64.0
    k.zero_()
    at = prefix - 1
    k[int(ptab[at // 16]), at % 16, 0, 0] = 64.0  # logit 512 against 0
    v[int(ptab[at // 16]), at % 16, 0, 5] = 1.5 * 2.0 ** 127
    O, L = reference(*args)
    o, lse = run(args)
    assert np.array_equal(o[:, :, 5].double().cpu().numpy(), O[:, :, 5])
    check_by_column(o, O, magnitudes(args))
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0
