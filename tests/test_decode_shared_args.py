"""What attn_decode_paged_shared refuses, and its workspace size, without a GPU."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
from online_softmax_attn_gb300 import build as attn_build

BAD, UNSUP = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
ARGS = dict(q=256, kc=1 << 20, vc=1 << 21, ptab=512, plen=640, table=768, lens=1024, B=2, h=32, h_kv=8, d=128, page=16,
            nb=100, mpb=50, mb=10, scale=0.1, ws=4096, wsb=1 << 40, o=8192, lse=None)


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.library()


def call(lib, **kw):
    a = {**ARGS, **kw}
    return lib.attn_decode_paged_shared(*[a[n] for n in ARGS], None)


def test_refuses(lib):
    need = attn.attn_decode_shared_workspace_bytes(2, 32, 8, 128)
    for kw in (dict(B=-1), dict(B=65536), dict(h=0), dict(h=30), dict(h_kv=0), dict(nb=0), dict(mb=0), dict(mpb=0),
               dict(mb=1 << 27), dict(mpb=1 << 27), dict(scale=0.0), dict(scale=float("nan")), dict(wsb=need - 1),
               dict(ws=4096 + 16), dict(lse=4098)):
        assert call(lib, **kw) == BAD, kw
    for name in ("q", "kc", "vc", "ptab", "plen", "table", "lens", "ws", "o"):
        assert call(lib, **{name: None}) == BAD, name
        assert call(lib, **{name: ARGS[name] + 2}) == BAD, name
    for kw in (dict(d=96), dict(page=32), dict(h=24), dict(h=128)):
        assert call(lib, **kw) == UNSUP, kw
    assert call(lib, B=0, q=None, ws=None, o=None) == 0


def test_workspace_bytes(lib):
    f = attn.attn_decode_shared_workspace_bytes
    a = lambda x: -(-x // 256) * 256
    # 64 rows x 4 heads: one block of two tiles, 152 runs, at most 152 / 8 + 2 on a head
    own = a(a(66 * 8) + 320 * 8 * 130 * 4) + 64 * 32 * 512 + 2 * a(64 * 32 * 4)
    assert f(64, 32, 8, 128) == own + 8 * 21 * 256 * 130 * 4
    assert f(0, 32, 8, 128) == f(1, 32, 8, 128) > 0
    assert f(65535, 8, 1, 64) > f(256, 8, 1, 64)
    for bad in ((-1, 32, 8, 128), (65536, 32, 8, 128), (2, 30, 8, 128), (2, 32, 0, 128), (2, 32, 8, 96), (2, 16, 1, 128)):
        assert f(*bad) == 0, bad


def test_binding_refuses_cpu_tensors():
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_paged_shared(q, c, c, i, i, i.view(1, 1), i)
