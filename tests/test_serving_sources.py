"""What the sources of the serving calls' kernels keep to, without a GPU."""
import os
import re

import pytest

from online_softmax_attn_gb300 import build as attn_build


@pytest.mark.parametrize("name", ["cache_e4m3.cu", "e4m3.cuh", "decode_runs.cu", "decode_runs.cuh", "decode_shared.cu"])
def test_no_non_coherent_loads(name):
    """These kernels are launched while the kernel in front may still write their
    inputs. A non-coherent load is only defined for data that stays as it is for
    the kernel's whole lifetime."""
    with open(os.path.join(attn_build.CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    assert re.findall(r"__ldg\s*\(|ld\.global\.nc", code) == []
