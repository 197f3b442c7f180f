"""Which strides attn_cache_write_e4m3 and attn_cache_read_e4m3 refuse, without a GPU
(accepted calls end with the missing device's error)."""
import pytest

import online_softmax_attn_gb300 as attn
from test_cache_e4m3_args import BAD, lib, read, write  # noqa: F401  (module fixture)


@pytest.mark.parametrize("call", [write, read])
def test_strides_count_where_they_are_used(lib, call):  # noqa: F811
    import torch

    for kw in (dict(kt=1020), dict(vt=4), dict(kh=129), dict(vh=4)):
        assert call(lib, **kw) == BAD, kw
    for kw in (dict(kt=1020, h_kv=1), dict(vh=129, total=1)):  # the other one's
        assert call(lib, **kw) == BAD, kw
    if torch.cuda.is_available():
        return  # the pointers of an accepted call are no memory
    for kw in (dict(kt=1020, total=1), dict(vt=1, total=1), dict(kh=129, h_kv=1), dict(vh=3, h_kv=1, dtype=0),
               dict(kt=5, vt=7, kh=9, vh=11, total=1, h_kv=1)):
        assert call(lib, **kw) == attn.ATTN_ERR_CUDA, kw
