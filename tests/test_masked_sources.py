"""What the sources of the tree and windowed calls' kernels keep to, without a GPU."""
import os
import re

from online_softmax_attn_gb300 import build as attn_build


def _code(name):
    with open(os.path.join(attn_build.CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_tree_decode_has_no_non_coherent_loads():
    """It is launched while the kernel in front may still write its inputs. A
    non-coherent load is only defined for data that stays as it is for the kernel's
    whole lifetime."""
    assert re.findall(r"__ldg\s*\(|ld\.global\.nc", _code("decode_tree.cu")) == []


def test_windowed_prefill_reads_the_v_pass_coherently():
    """The attention kernel may be resident while the V pass writes the tile flags and
    the rows' tiles: of the flags' two kinds of load, windows take the coherent one."""
    code = _code("prefill_tc.cu")
    body = code[code.index("    prefill_bf16_kernel(") : code.index("    v_to_f16_kernel(")]
    assert re.findall(r"[^\n]*__ldg\s*\([^\n]*", body) == [
        "  auto flag = [](const int* p) { return WIN ? __ldcg(p) : __ldg(p); };"]
