"""The windowed calls and the tree decode against the -DATTN_DEBUG build: index checks on
their kernels' global stores, and the abort paths after a load that is never requested
(a bounded wait gives up after 2 s; no fault)."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
import test_gpu_decode_tree as TD
import test_gpu_decode_window as DW
import test_gpu_prefill_window as PW
from parity import check_lse, check_out
from test_gpu_debug_build import _combinations, debug_library  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu

CASES = [
    (DW, "test_lengths_around_pages"),
    (DW, "test_head_layouts"),
    (DW, "test_batches_cut_over_the_gpu"),
    (DW, "test_slots_out_of_sight_never_reach_a_row"),
    (TD, "test_lengths_around_tiles"),
    (TD, "test_row_blocks"),
    (TD, "test_batches_cut_over_the_gpu"),
    (TD, "test_many_rows"),
    (TD, "test_tokens_outside_the_rows_are_left_as_they_are"),
    (TD, "test_nonfinite_drafts_reach_the_tokens_that_see_them_alone"),
    (PW, "test_bounds_around_tiles"),
    (PW, "test_long_rows"),
    (PW, "test_tokens_outside_the_rows_are_left_as_they_are"),
    (PW, "test_nonfinite_keys_and_values_reach_the_queries_that_see_them_alone"),
]


def _case_list():
    return [pytest.param(getattr(mod, name), kw, id=f"{mod.__name__}.{name}[{i}]")
            for mod, name in CASES for i, kw in enumerate(_combinations(getattr(mod, name)))]


@pytest.mark.parametrize("fn,kw", _case_list())
def test_case_under_debug_checks(fn, kw):
    fn(**kw)
    bits = attn.attn_get_device_error()
    assert bits & attn.ATTN_DEVERR_DEBUG_INDEX == 0, f"debug index check failed (bits {bits:#x})"
    assert bits == 0, f"device error bits {bits:#x}"


def after_a_stall(c, rows, stall):
    """The call with the stall on sets the timeout bit and ends; the next one is right."""
    attn.attn_get_device_error()
    stall(True)
    try:
        c.run()
        bits = attn.attn_get_device_error()
    finally:
        stall(False)
    assert bits == attn.ATTN_DEVERR_WAIT_TIMEOUT, f"bits {bits:#x}"
    O, L = c.reference(rows)
    o, lse = c.run()
    at = [t for b in rows for t in range(c.cu[b], c.cu[b + 1])]
    check_out(o[at], O[at], torch.bfloat16)
    check_lse(lse[at], L[at])
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("what", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("B,old,draft,tile", [(2, 300, 10, 0), (3, 40000, 20, 1), (40, 3000, 50, 6)])
def test_tree_abort_path_after_a_stalled_load(debug_library, B, old, draft, tile, what):  # noqa: F811
    """One row tile and two, a CTA's first tile and a later one, of a later unit too."""
    c = TD.Case([old] * B, [draft] * B, 8, 4, 64, seed=71)
    after_a_stall(c, [0, B - 1], lambda on: attn.attn_selftest_tree_stall(tile if on else -1, what))


@pytest.mark.parametrize("new,tile", [(1000, 2), (5000, 20)])
def test_windowed_prefill_abort_path_after_a_stalled_load(debug_library, new, tile):  # noqa: F811
    """The stall in a CTA's only item, and in a later one."""
    c = PW.Case([0, 300], [new, 40], 8, 4, 128, 72, 700, 4)
    after_a_stall(c, [1], lambda on: attn.attn_selftest_prefill_stall(tile if on else -1))
