"""attn_decode_paged_shared where values of very different sizes meet, and where a
lost or doubled page of values would show. Oracle and cases are those of
test_gpu_decode_shared.py."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import position_cases as PC
from parity import check_lse
from test_gpu_decode_shared import case, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def check_by_column(o, O, mag):
    """Relative to each output's own column: mag is the oracle's result over |V|.
    The output's rounding is 2^-8 of it, a weight's 2^-11 (one fp16 number; the
    two-term bf16 form is finer) of its value's share of mag. What is left are the
    roundings in 32 bits: of a score near the reference (both below 2^5 here but for
    keys that have all the weight) 2^-19, of the exponential 2^-22, of sums over at most
    1000 keys in any order 1000 * 2^-24; 2^-13 covers them."""
    err = np.abs(o.double().cpu().numpy() - O)
    tol = 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -13) * mag
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


@ROWS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exp", [-100, -40, -30, -26, -20, -12, 7, 9, 40])
def test_one_small_or_large_column(exp, d, B):
    """One column of 2^exp beside ordinary ones, in prefix and own keys alike: its
    outputs are right relative to themselves."""
    args = case(700, [33, 0] + [5] * (B - 2), 2, 4, d, seed=41)
    args[2][..., 9] *= 2.0 ** exp
    O, L = reference(*args)
    o, lse = run(args)
    check_by_column(o, O, magnitudes(args))
    check_lse(lse, L)


@pytest.mark.parametrize("exp", [-80, -32, -24, -16, 8, 30])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [3, 130, 690])
def test_dominant_key_with_other_values(at, exp, d):
    """A prefix key that takes all the weight and whose values are 2^exp times the
    others': the rows are that key's values."""
    args = case(700, [33, 0, 2], 2, 4, d, seed=42)
    q, k, v, ptab = args[:4]
    q.zero_()
    q[:, :, 0] = 64.0
    k[..., 0] = 0.0
    page, slot = int(ptab[at // 16]), at % 16
    k[page, slot, :, 0] = 64.0  # logit 512 or 362, others 0
    v[page, slot] *= 2.0 ** exp
    O, L = reference(*args)
    want = v[page, slot].double().repeat_interleave(4, 0).numpy()
    assert (np.abs(O - want) <= 1e-30).all()
    o, lse = run(args)
    check_by_column(o, O, np.abs(O))
    check_lse(lse, L)
    assert torch.equal(o.cpu(), v[page, slot].repeat_interleave(4, 0).expand(3, -1, -1))


@ROWS
@pytest.mark.parametrize("prefix", [128, 700])
@pytest.mark.parametrize("share", [1e-4, 0.3, 1.0])
def test_zeros_among_the_values(share, prefix, B):
    """Exact zeros of either sign here and there, in large parts, or everywhere."""
    args = case(prefix, [33, 0] + [5] * (B - 2), 2, 4, 64, seed=43)
    v = args[2]
    zero = torch.rand(v.shape, generator=torch.Generator().manual_seed(1)) < share
    v[zero] *= 0.0
    O, L = reference(*args)
    o, lse = run(args)
    check_by_column(o, O, magnitudes(args))
    check_lse(lse, L)


def test_every_bf16_number_as_a_value():
    """Each finite bf16 number up to 2^120 once as the value of a key that has all the
    weight: rows return it exactly, whatever the tile's other numbers are (512 rows
    of bits in order, so that the tiles range from all tiny to all large; then
    shuffled)."""
    bits = torch.arange(0, (127 + 120) << 7, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = torch.cat([bits, -bits])
    for shuffle in (False, True):
        if shuffle:
            bits = bits[torch.randperm(bits.numel(), generator=torch.Generator().manual_seed(3))]
        n = (bits.numel() + 63) // 64  # keys of 64 values
        vals = torch.zeros(n * 64, dtype=torch.bfloat16)
        vals[:bits.numel()] = bits
        pages = (n + 15) // 16
        k = torch.zeros((pages, 16, 1, 64), dtype=torch.bfloat16)
        v = torch.zeros_like(k)
        v.view(-1)[:n * 64] = vals
        # key i is +-1 in the 10 dims of its number's bits; a row with the same signs meets it alone at its maximum
        i = torch.arange(pages * 16)
        for b in range(10):
            k.view(-1, 64)[:, b] = ((i >> b) & 1).to(torch.bfloat16) * 2 - 1
        q = torch.zeros((n, 1, 64), dtype=torch.bfloat16)
        q[:, 0] = k.view(-1, 64)[:n] * 512.0  # scale 1: logit 5120, the others 1024 lower or more
        assert n <= 1024
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)
        o, _ = run([q, k, v, torch.arange(pages, dtype=torch.int32), i32([n]), torch.full((n, 1), -1, dtype=torch.int32),
                    torch.zeros(n, dtype=torch.int32)], scale=1.0)
        assert torch.equal(o.cpu().view(-1), vals)


@pytest.mark.parametrize("i", range(len(PC.SHARED)))
def test_every_page_counts_once(i):
    """Long prefixes and rows cut over the GPU, with values that carry their position."""
    args = PC.shared_case(*PC.SHARED[i], seed=71 + i)
    B = args[0].shape[0]
    rows = sorted({0, B // 2, B - 1, int(torch.argmax(args[6]))})
    O, L = reference(*args, rows=rows)
    o, lse = run(args)
    PC.check(o[rows].double().cpu().numpy(), O[rows])
    check_lse(lse[rows], L[rows])
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("shift", [0, -16])
@pytest.mark.parametrize("exp", [16, 21, 24, 27, 28, 30, 110])
@pytest.mark.parametrize("at", [5, 400])
def test_large_logits_and_large_values(at, exp, shift):
    """Logits up to 2^exp, of which one key leads by 2^(exp - 3), and values around 2^100
    from the second key tile on: the row is the leading key's value."""
    args = case(700, [50, 20], 2, 4, 64, seed=44)
    q, k, v, ptab = args[:4]
    q.zero_()
    q[:, :, 0] = 2.0 ** exp
    k.zero_()
    k[..., 0] = torch.randint(-8, 8, k.shape[:-1], generator=torch.Generator().manual_seed(2)).to(torch.bfloat16) + shift
    for p in range(8, 44):
        v[int(ptab[p])] *= 2.0 ** 100
    page, slot = int(ptab[at // 16]), at % 16
    k[page, slot, :, 0] = 8 + shift
    o, lse = run(args)
    assert torch.equal(o.cpu(), v[page, slot].repeat_interleave(4, 0).expand(2, -1, -1))
    L = reference(*args)[1]
    # factor, product, ln 2 and the product with it: 5 roundings of 2^-24
    assert (np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -21 * np.abs(L)).all()
