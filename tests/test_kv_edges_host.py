"""Host-side checks of the attention-side operators beyond tests/test_kv_host.py: calls without rows, and how the
kernels read what the kernel before them may have written."""
import ctypes
import os
import re

import pytest

FAKE = 1 << 40                              # never dereferenced: nothing is launched


@pytest.fixture(scope="module")
def tg():
    from bit_gemv_tern_b200 import build
    build.build()
    import bit_gemv_tern_b200 as tg
    tg.lib()
    return tg


def call(tg, rows):
    """The statuses of the four operators with null row pointers (an empty tensor's) and `rows` rows."""
    L, r = tg.lib(), ctypes.byref
    x = tg._Qkv(None, tg.TERN_ELEM_F32, 32, 8, 128, 48 * 128, FAKE, FAKE, 1e-6, FAKE)
    c, b = tg._KvCache(10, 64, 8, 128, FAKE, FAKE, FAKE, FAKE), tg._KvBatch(4, rows, 16, FAKE, FAKE, FAKE)
    return [L.tern_qk_norm_rope(r(x), rows, None, None, None, 0, None),
            L.tern_kv_append(r(x), r(c), r(b), None, None, 0, None),
            L.tern_kv_read(r(c), r(b), None, None, None, None),
            L.tern_paged_attn(None, 32, 0.1, r(c), r(b), 1, None, None, FAKE, 1 << 30, None, 0, None)]


def test_null_row_pointers_are_fine_without_rows(tg):
    assert call(tg, 0) == [0, 0, 0, 0]
    assert call(tg, 1) == [1, 1, 1, 1]


def test_no_load_goes_through_the_non_coherent_path(tg):
    """What a call reads may have been written by the kernel in front of it, beside which programmatic dependent launch
    starts it; read-only loads are for what nothing writes while the kernel lives. The sources hold none."""
    csrc = os.path.join(os.path.dirname(tg.__file__), "csrc")
    for name in ("tern_kv.cu", "tern_kv.cuh", "tern_attn.cu", "tern_attn.cuh", "tern_attn_tile.cu", "tern_mbar.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code), name
