"""What attn_prefill_paged_window refuses, without a GPU."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
from online_softmax_attn_gb300 import build as attn_build

BAD, UNSUP = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
ARGS = dict(q=256, kc=1 << 20, vc=1 << 21, table=768, cu=896, lens=1024, B=2, total=200, h=32, h_kv=8, d=128, page=16,
            nb=100, mb=20, max_q=150, window=64, sinks=4, scale=0.1, ws=4096, wsb=1 << 40, o=8192, lse=None)


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.library()


def call(lib, **kw):
    a = {**ARGS, **kw}
    return lib.attn_prefill_paged_window(*[a[n] for n in ARGS], None)


def test_refuses(lib):
    need = attn.attn_prefill_window_workspace_bytes(2, 20, 8, 128)
    assert need == attn.attn_prefill_paged_workspace_bytes(2, 20, 8, 128, v16=True) + 256 > 256
    for kw in (dict(B=-1), dict(B=65536), dict(total=-1), dict(h=0), dict(h=30), dict(h=65544), dict(h_kv=0), dict(nb=0),
               dict(mb=0), dict(mb=1 << 27), dict(scale=0.0), dict(scale=float("inf")), dict(wsb=need - 1),
               dict(ws=4096 + 16), dict(lse=4098), dict(max_q=0), dict(window=0), dict(window=-5), dict(sinks=-1)):
        assert call(lib, **kw) == BAD, kw
    for name in ("q", "kc", "vc", "table", "cu", "lens", "ws", "o"):
        assert call(lib, **{name: None}) == BAD, name
        assert call(lib, **{name: ARGS[name] + 2}) == BAD, name
    for kw in (dict(d=96), dict(page=32), dict(B=40000, mb=1 << 20), dict(total=2 ** 31 - 1, h=8192)):
        assert call(lib, **kw) == UNSUP, kw
    assert call(lib, B=0, q=None, ws=None, o=None) == 0
    assert call(lib, total=0, q=None, ws=None, o=None) == 0


def test_workspace_bytes(lib):
    f = attn.attn_prefill_window_workspace_bytes
    for bad in ((-1, 20, 8, 128), (2, 0, 8, 128), (2, 20, 0, 128), (2, 20, 8, 96), (40000, 1 << 20, 8, 128)):
        assert f(*bad) == 0, bad


def test_binding_refuses_cpu_tensors():
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_prefill_paged_window(q, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i, 5, 0, 1)


def test_sizes_without_a_workspace_are_unsupported(lib):
    """Where the size function gives 0 a caller holds no workspace: the call says why."""
    big = dict(B=40000, mb=1 << 20)
    assert attn.attn_prefill_window_workspace_bytes(40000, 1 << 20, 8, 128) == 0
    assert call(lib, **big, ws=None, wsb=0) == UNSUP
    assert call(lib, **big, wsb=0) == UNSUP
    assert call(lib, ws=None, wsb=0) == BAD
    assert call(lib, **big, window=0, ws=None) == BAD
