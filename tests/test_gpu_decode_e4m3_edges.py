"""attn_decode_paged_e4m3 at the far ends of the factors' ranges, and where a lost or
doubled page of values would show. Oracle and cases are those of
test_gpu_decode_e4m3.py; both forms of the call, by the table's width."""
import numpy as np
import pytest
import torch

import online_softmax_attn_gb300 as attn
import position_cases as PC
from e4m3_cases import cache_from, decode_case, values
from parity import check_lse
from test_gpu_decode_e4m3 import cuda, reference
from test_gpu_decode_e4m3_wide import widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


FORMS = pytest.mark.parametrize("call", [attn.attn_decode_paged_e4m3, widened], ids=["one_kernel", "runs"])


@FORMS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qe,ke", [(100, 100), (120, 110), (126, -100), (-100, 118), (60, 60), (-60, -60)])
def test_queries_and_keys_far_from_one(qe, ke, d, call):
    """Queries of 2^qe against keys of 2^ke, in different columns but for one whose
    products are ordinary: scores are numbers although the two sizes' product is not.
    Heads of ordinary queries among them."""
    lens = [300, 20]
    q, kc, vc, ks, vs, table, n = decode_case(lens, 2, 4, d, seed=61)
    q[:, :, 0] = 2.0 ** qe
    q[:, :, 1:] = 0.0
    if qe + ke > -20:  # one column in common, small on one side
        q[:, :, 2] = 2.0 ** max(qe - 12, -100)
    q[:, 1] = 0.0
    q[:, 1, 3] = 1.0
    k64 = np.zeros_like(values(kc, ks))
    k64[..., 1] = 2.0 ** ke
    k64[..., 3] = np.random.default_rng(5).integers(-3, 4, k64.shape[:-1]) * 2.0 ** min(ke, 2)
    kc, ks = cache_from(k64.transpose(0, 2, 1, 3))
    args = (q, kc, vc, ks, vs, table, n)
    O, L = reference(*args)
    assert np.isfinite(L).all()
    o, lse = call(*cuda(*args))
    mag = reference(q, kc, torch.from_numpy(np.abs(vc.float().numpy())).to(vc.dtype), ks, vs, table, n)[0]
    err = np.abs(o.double().cpu().numpy() - O)
    # the output's rounding, a weight's (one fp16 number), and what is done in 32 bits
    assert (err <= 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -13) * mag).all()
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("i", range(len(PC.E4M3)))
def test_every_page_counts_once(i):
    """Rows cut over the GPU, with values that carry their position."""
    args = PC.e4m3_case(*PC.E4M3[i], seed=81 + i)
    O, L = reference(*args)
    o, lse = attn.attn_decode_paged_e4m3(*cuda(*args))
    PC.check(o.double().cpu().numpy(), O)
    check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


@FORMS
@pytest.mark.parametrize("length", [1000, 4096, 16])
def test_every_page_counts_once_in_either_form(length, call):
    args = PC.e4m3_case([length, 20], 2, 4, 64, seed=91)
    O, L = reference(*args)
    o, lse = call(*cuda(*args))
    PC.check(o.double().cpu().numpy(), O)
    check_lse(lse, L)
