"""What attn_cache_write_e4m3, attn_cache_read_e4m3 and attn_decode_paged_e4m3
refuse, without a GPU: the C entry points with pointers that are never
dereferenced, the binding with CPU tensors."""
import ctypes

import pytest
import torch

import online_softmax_attn_gb300 as attn
import oracle.cache_e4m3 as ref
from online_softmax_attn_gb300 import build as attn_build

P = ctypes.c_void_p
BAD, UNSUP = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.library()


TOKENS = dict(k=4096, v=8192, kt=1024, kh=128, vt=1024, vh=128, dtype=1, table=256, cu=512, lens=768, B=2,
              total=10, h_kv=8, d=128, page=16, nb=100, mb=10, kc=1 << 20, vc=1 << 21, ks=1 << 22, vs=1 << 23)


def write(lib, **kw):
    a = {**TOKENS, **kw}
    return lib.attn_cache_write_e4m3(a["k"], a["v"], a["kt"], a["kh"], a["vt"], a["vh"], a["dtype"], a["table"],
                                     a["cu"], a["lens"], a["B"], a["total"], a["h_kv"], a["d"], a["page"], a["nb"],
                                     a["mb"], a["kc"], a["vc"], a["ks"], a["vs"], None)


def read(lib, **kw):
    a = {**TOKENS, **kw}
    return lib.attn_cache_read_e4m3(a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["cu"], a["lens"], a["B"],
                                    a["total"], a["h_kv"], a["d"], a["page"], a["nb"], a["mb"], a["k"], a["v"],
                                    a["kt"], a["kh"], a["vt"], a["vh"], a["dtype"], None)


@pytest.mark.parametrize("call", [write, read])
def test_token_calls_refuse(lib, call):
    for kw in (dict(B=-1), dict(total=-1), dict(h_kv=0), dict(h_kv=65536), dict(nb=0), dict(mb=0), dict(dtype=7),
               dict(mb=1 << 27), dict(kt=1020), dict(vh=129), dict(dtype=0, kh=130)):
        assert call(lib, **kw) == BAD, kw
    for name in ("k", "v", "table", "cu", "lens", "kc", "vc", "ks", "vs"):
        assert call(lib, **{name: None}) == BAD, name
        assert call(lib, **{name: TOKENS[name] + 2}) == BAD, name
    for kw in (dict(d=96), dict(d=256), dict(page=32)):
        assert call(lib, **kw) == UNSUP, kw
    none = {n: None for n in ("k", "v", "table", "cu", "lens", "kc", "vc", "ks", "vs")}
    assert call(lib, total=0, **none) == 0 and call(lib, B=0, **none) == 0  # no-ops


DECODE = dict(q=256, kc=1 << 20, vc=1 << 21, ks=1 << 22, vs=1 << 23, table=512, lens=768, B=2, h=32, h_kv=8, d=128,
              page=16, nb=100, mb=10, scale=0.1, ws=4096, wsb=1 << 40, o=8192, lse=None)


def decode(lib, **kw):
    a = {**DECODE, **kw}
    return lib.attn_decode_paged_e4m3(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"], a["B"],
                                      a["h"], a["h_kv"], a["d"], a["page"], a["nb"], a["mb"], a["scale"], a["ws"],
                                      a["wsb"], a["o"], a["lse"], None)


def test_decode_refuses(lib):
    need = attn.attn_decode_e4m3_workspace_bytes(2, 32, 8, 128)
    for kw in (dict(B=-1), dict(B=65536), dict(h=0), dict(h=30), dict(h_kv=0), dict(nb=0), dict(mb=0), dict(mb=1 << 27),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.0),
               dict(nb=1 << 28), dict(B=65535, h=8 * 8192), dict(wsb=need - 1), dict(ws=4096 + 16)):
        assert decode(lib, **kw) == BAD, kw
    for name in ("q", "kc", "vc", "ks", "vs", "table", "lens", "ws", "o"):
        assert decode(lib, **{name: None}) == BAD, name
        assert decode(lib, **{name: DECODE[name] + 2}) == BAD, name
    assert decode(lib, lse=4098) == BAD
    for kw in (dict(d=96), dict(page=32)):
        assert decode(lib, **kw) == UNSUP, kw
    assert decode(lib, B=0, q=None, ws=None, o=None) == 0


def test_decode_workspace_bytes(lib):
    """Plan (int64: B + 2), then 320 states of 8 heads: d_h + 2 floats each."""
    a = lambda x: -(-x // 256) * 256
    for B, d in ((0, 128), (1, 64), (66, 128), (65535, 64)):
        assert attn.attn_decode_e4m3_workspace_bytes(B, 32, 8, d) == a((B + 2) * 8) + 320 * 8 * (d + 2) * 4
    for bad in ((-1, 32, 8, 128), (2, 0, 8, 128), (2, 30, 8, 128), (2, 32, 0, 128), (2, 32, 8, 96)):
        assert attn.attn_decode_e4m3_workspace_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros((1, 2, 16), dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_cache_write_e4m3(x, x, c, c, e, e, i.view(1, 1), i, i)
    with pytest.raises(ValueError):
        attn.attn_cache_read_e4m3(c, c, e, e, i.view(1, 1), i, i, x, x)
    with pytest.raises(ValueError):
        attn.attn_decode_paged_e4m3(x, c, c, e, e, i.view(1, 1), i)


def test_format_definition():
    """The oracle's own format: border exponents, ties to even, the smallest
    and largest magnitudes."""
    import numpy as np

    c, e = ref.quantise_ref(np.array([[448.0, 1.0, 17.0, 19.0, 0.0, -17.5]]))
    assert e[0] == 127 and c[0].tolist() == [448.0, 1.0, 16.0, 20.0, 0.0, -18.0]
    c, e = ref.quantise_ref(np.array([[449.0, 2.0]]))
    assert e[0] == 128 and c[0].tolist() == [224.0, 1.0]
    c, e = ref.quantise_ref(np.array([[0.0, 0.0]]))
    assert e[0] == 10
    c, e = ref.quantise_ref(np.array([[3.4e38, np.inf]]))
    assert e[0] == 246 and c[0, 0] == 448.0 and np.isnan(c[0, 1])
    # exponent -8, smallest code 2^-9: half of it is a tie that goes to 0
    c, e = ref.quantise_ref(np.array([[1.0, 2.0 ** -18, 1.25 * 2.0 ** -18, 1.5 * 2.0 ** -17]]))
    assert e[0] == 127 - 8 and c[0].tolist() == [256.0, 0.0, 2.0 ** -9, 2.0 ** -8]


def test_format_matches_torch_cast():
    """Every bf16 number in a row whose maximum is 448: the definition agrees
    with torch's rounding to e4m3."""
    import numpy as np

    x = torch.arange(0x0000, 0x43e1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()  # 0 .. 448
    rows = torch.stack([x, torch.full_like(x, 448.0)], -1)
    c, e = ref.quantise_ref(rows.numpy())
    assert (e == 127).all()
    assert np.array_equal(c[:, 0], x.float().to(torch.float8_e4m3fn).double().numpy())
