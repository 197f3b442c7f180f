"""The abort path of attn_decode_paged_shared, in the debug build and without a fault: a
load that is never requested lets a bounded wait give up after 2 s."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
from parity import check_lse, check_out
from test_gpu_debug_build import debug_library  # noqa: F401  (module fixture)
from test_gpu_decode_shared import case, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [0, 1, 2], ids=["k", "v", "v_again"])
@pytest.mark.parametrize("B,prefix,tile", [(3, 200, 0), (40, 200, 0), (300, 12000, 5), (20, 30000, 1)])
def test_abort_path_after_a_stalled_load(debug_library, B, prefix, tile, what):  # noqa: F811
    """Every role stops (those that wait for the tile, for a stage or for weights),
    drains what it issued, goes through the rows' own pages and ends. The next call on
    the same context, with the stall off, is right."""
    args = case(prefix, [9 * (i % 4) for i in range(B)], 8, 4, 64, seed=51)
    if what == 2:
        args[2][..., 3] = 300.0  # every tile of V stays bf16
    attn.attn_get_device_error()
    attn.attn_selftest_shared_stall(tile, what)
    try:
        run(args)
        bits = attn.attn_get_device_error()
    finally:
        attn.attn_selftest_shared_stall(-1)
    assert bits == attn.ATTN_DEVERR_WAIT_TIMEOUT, f"bits {bits:#x}"
    rows = [0, 1, B - 1]
    O, L = reference(*args, rows=rows)
    o, lse = run(args)
    mag = reference(args[0], args[1], args[2].abs(), *args[3:], rows=rows)[0]
    check_out(o[rows], O[rows], torch.bfloat16, mag=mag[rows])
    check_lse(lse[rows], L[rows])
    assert attn.attn_get_device_error() == 0
