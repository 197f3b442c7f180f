"""What attn_decode_paged_tree refuses, without a GPU."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
from online_softmax_attn_gb300 import build as attn_build

BAD, UNSUP = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
ARGS = dict(q=256, kc=1 << 20, vc=1 << 21, table=768, cu=896, lens=1024, mask=1152, B=2, total=20, h=32, h_kv=8, d=128,
            page=16, nb=100, mb=10, max_q=33, words=2, scale=0.1, ws=4096, wsb=1 << 40, o=8192, lse=None)


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.library()


def call(lib, **kw):
    a = {**ARGS, **kw}
    return lib.attn_decode_paged_tree(*[a[n] for n in ARGS], None)


def test_refuses(lib):
    need = attn.attn_decode_tree_workspace_bytes(2, 32, 8, 128)
    for kw in (dict(B=-1), dict(B=65536), dict(total=-1), dict(total=1 << 27), dict(h=0), dict(h=30), dict(h_kv=0),
               dict(nb=0), dict(mb=0), dict(mb=1 << 27), dict(scale=0.0), dict(scale=float("nan")), dict(wsb=need - 1),
               dict(ws=4096 + 16), dict(lse=4098), dict(max_q=0), dict(max_q=65), dict(words=0), dict(words=-1)):
        assert call(lib, **kw) == BAD, kw
    for name in ("q", "kc", "vc", "table", "cu", "lens", "mask", "ws", "o"):
        assert call(lib, **{name: None}) == BAD, name
        assert call(lib, **{name: ARGS[name] + 2}) == BAD, name
    for kw in (dict(d=96), dict(page=32), dict(h=1032)):
        assert call(lib, **kw) == UNSUP, kw
    assert call(lib, B=0, q=None, ws=None, o=None) == 0
    assert call(lib, total=0, q=None, mask=None, o=None) == 0


def test_workspace_bytes(lib):
    f = attn.attn_decode_tree_workspace_bytes
    # 160 CTAs: 16 bytes each, and two states of two tiles of 128 rows
    assert f(2, 32, 8, 128) == 160 * 16 + 320 * 256 * 130 * 4
    assert f(0, 8, 8, 64) == f(65535, 64, 1, 64) == 160 * 16 + 320 * 256 * 66 * 4
    for bad in ((-1, 32, 8, 128), (2, 30, 8, 128), (2, 32, 0, 128), (2, 32, 8, 96), (2, 129, 1, 64)):
        assert f(*bad) == 0, bad


def test_binding_refuses_cpu_tensors():
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_paged_tree(q, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i, i.view(1, 1), 1)
