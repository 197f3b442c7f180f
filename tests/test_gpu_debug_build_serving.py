"""The 8-bit cache and the shared-prefix decode against the -DATTN_DEBUG build:
their kernels check the indices of their global stores, record a failed check in
the device error word and skip the access. Each case must match its reference, as
in its own module, and leave no error bit set."""
import pytest

import online_softmax_attn_gb300 as attn
import test_gpu_cache_e4m3 as C8
import test_gpu_decode_e4m3 as D8
import test_gpu_decode_shared as DS
from test_gpu_debug_build import _combinations, debug_library  # noqa: F401  (module fixture)

pytestmark = pytest.mark.gpu

CASES = [
    (C8, "test_write_matches_definition"),
    (C8, "test_write_nonfinite_become_nan_and_leave_the_scale"),
    (C8, "test_write_bad_pages_and_positions_are_dropped_and_flagged"),
    (C8, "test_read_returns_stored_values"),
    (D8, "test_lengths_around_pages"),
    (D8, "test_runs_of_every_kind"),
    (D8, "test_bad_pages_and_lengths_are_flagged"),
    (D8, "test_write_decode_and_read_together"),
    (DS, "test_small_prefixes_and_own_lengths"),
    (DS, "test_row_blocks"),
    (DS, "test_many_row_blocks"),
    (DS, "test_mixed_magnitudes_between_tiles"),
    (DS, "test_bad_pages_and_lengths_are_flagged"),
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
