"""attn_decode_paged_e4m3 with block tables wider than its one-kernel form takes
(256 pages): the small cases of test_gpu_decode_e4m3.py through the other form,
and the two forms on the same inputs."""
import pytest
import torch

import online_softmax_attn_gb300 as attn
import test_gpu_decode_e4m3 as D8
from e4m3_cases import decode_case
from parity import check_lse, check_out
from test_gpu_debug_build import _combinations

pytestmark = pytest.mark.gpu

call = attn.attn_decode_paged_e4m3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from online_softmax_attn_gb300 import build

    build.build()


def widened(q, kc, vc, ks, vs, table, lens, *args, **kw):
    wide = torch.full((table.shape[0], max(table.shape[1], 300)), -1, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return call(q, kc, vc, ks, vs, wide, lens, *args, **kw)


CASES = ["test_lengths_around_pages", "test_no_rows_with_keys", "test_value_magnitudes", "test_mixed_value_scales",
         "test_extreme_queries", "test_large_logits_force_the_reference_up",
         "test_slots_past_the_length_never_reach_a_row", "test_nan_codes_reach_their_rows_only",
         "test_logits_beyond_the_precision_of_differences"]


@pytest.mark.parametrize("name,kw", [pytest.param(n, kw, id=f"{n}[{i}]") for n in CASES
                                     for i, kw in enumerate(_combinations(getattr(D8, n)))])
def test_small_cases_with_a_wide_table(name, kw, monkeypatch):
    monkeypatch.setattr(attn, "attn_decode_paged_e4m3", widened)
    getattr(D8, name)(**kw)


@pytest.mark.parametrize("lens", [[0], [1], [1023], [1024], [1025], [4096], [4095, 1], [0, 700, 0, 16, 129, 2000, 3]])
@pytest.mark.parametrize("h_kv,g,d", [(2, 4, 128), (1, 8, 64), (1, 11, 128), (2, 3, 64)])
def test_both_forms(lens, h_kv, g, d):
    """Lengths at the run borders of a cluster of 64 warps, blocks of more than 8
    heads, empty rows; results and LSE of either form."""
    args = decode_case(lens, h_kv, g, d, seed=40 + len(lens))
    O, L = D8.reference(*args)
    dev = D8.cuda(*args)
    for f in (call, widened):
        o, lse = f(*dev)
        check_out(o, O, torch.bfloat16)
        check_lse(lse, L)
        again, lse2 = f(*dev)
        assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert attn.attn_get_device_error() == 0


def test_one_kernel_form_replayed_with_new_lengths():
    """Captured once, replayed with lengths from 0 to the table's width, two
    calls on one workspace in the graph."""
    lens = [4000, 300]
    q, kc, vc, ks, vs, table, _ = decode_case(lens, 2, 4, 128, seed=50)
    dev = D8.cuda(q, kc, vc, ks, vs, table)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_decode_e4m3_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    q2 = dev[0].flip(0).contiguous()
    outs = [(torch.empty_like(q2), torch.empty(2, 8, device="cuda")) for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(*dev, n, workspace=ws, o=outs[0][0], lse=outs[0][1], stream=s)  # loads the kernel
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for x, (o, lse) in zip((dev[0], q2), outs):
            call(x, *dev[1:], n, workspace=ws, o=o, lse=lse, stream=s)
    for now in ([4000, 300], [0, 1], [1, 0], [17, 299], [2049, 16]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for x, (o, lse) in zip((q, q.flip(0)), outs):
            O, L = D8.reference(x, kc, vc, ks, vs, table, torch.tensor(now, dtype=torch.int32))
            check_out(o, O, torch.bfloat16)
            check_lse(lse, L)
    assert attn.attn_get_device_error() == 0


def test_one_kernel_form_keeps_to_its_outputs():
    """Guard bytes around o, lse and the workspace's end stay."""
    args = D8.cuda(*decode_case([900, 0, 40], 2, 4, 128, seed=51))
    size = attn.attn_decode_e4m3_workspace_bytes(3, 8, 2, 128)
    ws = torch.full((size + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    ob = torch.full((3 * 8 * 128 + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((3 * 8 + 1024,), 7.0, device="cuda")
    o, lse = ob[2048:-2048].view(3, 8, 128), lb[512:-512].view(3, 8)
    call(*args, workspace=ws[:size], o=o, lse=lse)
    want, want_lse = call(*args)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert (ws[size:] == 0x5a).all() and (ob[:2048] == 7).all() and (ob[-2048:] == 7).all()
    assert (lb[:512] == 7).all() and (lb[-512:] == 7).all()
