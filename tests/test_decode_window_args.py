"""What the windowed decodes refuse, without a GPU."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
from online_softmax_attn_gb300 import build as attn_build

BAD, UNSUP = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
ARGS = dict(q=256, kc=1 << 20, vc=1 << 21, ks=1 << 22, vs=1 << 23, table=768, lens=1024, B=2, h=32, h_kv=8, d=128,
            page=16, nb=100, mb=10, window=64, sinks=4, scale=0.1, ws=4096, wsb=1 << 40, o=8192, lse=None)


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.library()


def call(lib, eight, **kw):
    a = {**ARGS, **kw}
    f = lib.attn_decode_paged_window_e4m3 if eight else lib.attn_decode_paged_window
    return f(*[a[n] for n in ARGS if eight or n not in ("ks", "vs")], None)


@pytest.mark.parametrize("eight", [False, True])
def test_refuses(lib, eight):
    need = attn.attn_decode_window_workspace_bytes(2, 32, 8, 128)
    for kw in (dict(B=-1), dict(B=65536), dict(h=0), dict(h=30), dict(h_kv=0), dict(nb=0), dict(mb=0), dict(mb=1 << 27),
               dict(scale=0.0), dict(scale=float("nan")), dict(wsb=need - 1), dict(ws=4096 + 16), dict(lse=4098),
               dict(window=0), dict(window=-1), dict(sinks=-1)):
        assert call(lib, eight, **kw) == BAD, kw
    for name in ("q", "kc", "vc", "table", "lens", "ws", "o") + (("ks", "vs") if eight else ()):
        assert call(lib, eight, **{name: None}) == BAD, name
        assert call(lib, eight, **{name: ARGS[name] + 2}) == BAD, name
    for kw in (dict(d=96), dict(page=32)):
        assert call(lib, eight, **kw) == UNSUP, kw
    assert call(lib, eight, B=0, q=None, ws=None, o=None) == 0


def test_workspace_bytes(lib):
    f = attn.attn_decode_window_workspace_bytes
    # the run decode's, and 16 bytes for each of 160 CTAs
    assert f(2, 32, 8, 128) == attn.attn_decode_e4m3_workspace_bytes(2, 32, 8, 128) + 160 * 16 > 160 * 16
    for bad in ((-1, 32, 8, 128), (2, 30, 8, 128), (2, 32, 0, 128), (2, 32, 8, 96)):
        assert f(*bad) == 0, bad


def test_binding_refuses_cpu_tensors():
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_paged_window(q, c, c, i.view(1, 1), i, 5)
