"""Host-side checks of the attention-side operators beyond tests/test_kv_host.py: how the kernels read what the kernel
before them may have written."""
import os
import re

import pytest


@pytest.fixture(scope="module")
def tg():
    from bit_gemv_tern_b200 import build
    build.build()
    import bit_gemv_tern_b200 as tg
    tg.lib()
    return tg


def test_no_load_goes_through_the_non_coherent_path(tg):
    """What a call reads may have been written by the kernel in front of it, beside which programmatic dependent launch
    starts it; read-only loads are for what nothing writes while the kernel lives. The sources hold none."""
    csrc = os.path.join(os.path.dirname(tg.__file__), "csrc")
    for name in ("tern_kv.cu", "tern_kv.cuh", "tern_attn.cu", "tern_attn.cuh", "tern_attn_tile.cu", "tern_mbar.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code), name
