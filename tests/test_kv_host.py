"""Host-side checks of the attention-side operators that need no GPU: what they refuse, before anything
is launched, through the C ABI and through the Python binding; sizes; the rotation's frequencies."""
import ctypes
import math

import pytest

FAKE = 1 << 40                              # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def tg():
    from bit_gemv_tern_b200 import build
    build.build()
    import bit_gemv_tern_b200 as tg
    tg.lib()
    return tg


def qkv(tg, **kw):
    c = tg._Qkv(FAKE, tg.TERN_ELEM_F32, 32, 8, 128, 48 * 128, FAKE, FAKE, 1e-6, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def cache(tg, **kw):
    c = tg._KvCache(10, 64, 8, 128, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def batch(tg, **kw):
    c = tg._KvBatch(4, 4, 16, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("kw,want", [
    (dict(src_dev=None), 1), (dict(freq_dev=None), 1), (dict(src_dev=FAKE + 8), 1), (dict(freq_dev=FAKE + 4), 1),
    (dict(src_type=2), 1), (dict(q_gain_dev=FAKE + 2), 1), (dict(k_gain_dev=FAKE + 2), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(head_dim=96), 2), (dict(q_heads=0), 2), (dict(q_heads=12), 2), (dict(kv_heads=0), 2), (dict(q_heads=8192), 2),
    (dict(row_stride=40 * 128 - 4), 2), (dict(row_stride=48 * 128 + 2), 2), (dict(row_stride=1 << 33), 2),
])
def test_qkv_refusals(tg, kw, want):
    L = tg.lib()
    assert L.tern_qk_norm_rope(qkv(tg, **kw), 4, FAKE, FAKE, FAKE, 0, None) == want
    assert L.tern_kv_append(qkv(tg, **kw), cache(tg), batch(tg), FAKE, None, 0, None) == want


@pytest.mark.parametrize("ckw,bkw,want", [
    (dict(k_dev=None), {}, 1), (dict(v_dev=None), {}, 1), (dict(k_scale_dev=None), {}, 1), (dict(v_scale_dev=None), {}, 1),
    (dict(k_dev=FAKE + 8), {}, 1), (dict(v_dev=FAKE + 4), {}, 1), (dict(k_scale_dev=FAKE + 2), {}, 1),
    (dict(pages=0), {}, 2), (dict(pages=1 << 23), {}, 2), (dict(page_size=0), {}, 2), (dict(page_size=24), {}, 2), (dict(page_size=65552), {}, 2),
    (dict(head_dim=80), {}, 2), (dict(kv_heads=0), {}, 2), (dict(kv_heads=2000), {}, 2),
    ({}, dict(row_start_dev=None), 1), ({}, dict(kv_len_dev=None), 1), ({}, dict(page_table_dev=None), 1),
    ({}, dict(kv_len_dev=FAKE + 1), 1), ({}, dict(batch=0), 2), ({}, dict(batch=65537), 2), ({}, dict(rows=-1), 2),
    ({}, dict(rows=(1 << 24) + 1), 2), ({}, dict(max_pages=0), 2), ({}, dict(max_pages=1 << 25), 2),
])
def test_cache_and_batch_refusals(tg, ckw, bkw, want):
    L = tg.lib()
    c, b = cache(tg, **ckw), batch(tg, **bkw)
    ws = 1 << 30
    assert L.tern_kv_append(qkv(tg), c, b, FAKE, None, 0, None) == want
    assert L.tern_kv_read(c, b, FAKE, FAKE, None, None) == want
    assert L.tern_paged_attn(FAKE, 32, 0.1, c, b, 1, FAKE, None, FAKE, ws, None, 0, None) == want


def test_call_refusals(tg):
    L, ws = tg.lib(), 1 << 30
    x, c, b = qkv(tg), cache(tg), batch(tg)
    assert L.tern_qk_norm_rope(None, 4, FAKE, FAKE, FAKE, 0, None) == 1
    assert L.tern_qk_norm_rope(x, -1, FAKE, FAKE, FAKE, 0, None) == 2
    assert L.tern_qk_norm_rope(x, 4, None, FAKE, FAKE, 0, None) == 1
    assert L.tern_qk_norm_rope(x, 4, FAKE, FAKE + 8, FAKE, 0, None) == 1
    assert L.tern_qk_norm_rope(x, 4, FAKE, FAKE, None, 0, None) == 1
    assert L.tern_qk_norm_rope(x, 4, FAKE, FAKE, FAKE, 2, None) == 1
    assert L.tern_kv_append(x, None, b, FAKE, None, 0, None) == 1
    assert L.tern_kv_append(x, c, None, FAKE, None, 0, None) == 1
    assert L.tern_kv_append(x, c, b, None, None, 0, None) == 1
    assert L.tern_kv_append(x, c, b, FAKE, FAKE + 2, 0, None) == 1
    assert L.tern_kv_append(x, c, b, FAKE, None, 4, None) == 1
    assert L.tern_kv_append(x, cache(tg, kv_heads=4), b, FAKE, None, 0, None) == 2
    assert L.tern_kv_append(x, cache(tg, head_dim=64), b, FAKE, None, 0, None) == 2
    assert L.tern_kv_read(c, b, None, FAKE, None, None) == 1
    assert L.tern_kv_read(c, b, FAKE, FAKE + 4, None, None) == 1
    ok = dict(q=FAKE, hq=32, scale=0.1, n=1, out=FAKE, lse=None, ws=FAKE, size=ws, flags=0)

    def attn(**kw):
        a = {**ok, **kw}
        return L.tern_paged_attn(a["q"], a["hq"], a["scale"], c, b, a["n"], a["out"], a["lse"], a["ws"], a["size"], None,
                                 a["flags"], None)

    for kw in (dict(q=None), dict(out=None), dict(ws=None), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(lse=FAKE + 1),
               dict(ws=FAKE + 8), dict(scale=math.nan), dict(scale=math.inf), dict(size=16), dict(flags=2)):
        assert attn(**kw) == 1, kw
    for kw in (dict(hq=0), dict(hq=20), dict(hq=4104), dict(n=0)):
        assert attn(**kw) == 2, kw


def test_nothing_to_do_is_fine(tg):
    L = tg.lib()
    b = batch(tg, rows=0)
    assert L.tern_qk_norm_rope(qkv(tg), 0, FAKE, FAKE, FAKE, 0, None) == 0
    assert L.tern_kv_append(qkv(tg), cache(tg), b, FAKE, None, 0, None) == 0
    assert L.tern_kv_read(cache(tg), b, FAKE, FAKE, None, None) == 0
    assert L.tern_paged_attn(FAKE, 32, 0.1, cache(tg), b, 1, FAKE, None, FAKE, 1 << 30, None, 0, None) == 0


def test_workspace_sizes(tg):
    assert tg.tern_paged_attn_workspace_bytes(32, 8, 128) > 0
    assert tg.tern_paged_attn_workspace_bytes(32, 5, 128) == 0
    assert tg.tern_paged_attn_workspace_bytes(32, 8, 100) == 0


def test_frequencies(tg):
    f = tg.tern_rope_freqs(128, 1e6, device="cpu")
    assert f.shape == (64,) and float(f[0]) == 1.0 and abs(float(f[32]) - 1e-3) < 1e-15


def test_python_binding_refuses_other_tensors(tg):
    """Types, shapes, strides and devices: a ValueError before the library is called."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checked where every tensor is on the host")
    f = tg.tern_rope_freqs(128, device="cpu")
    codes, scale = torch.zeros(2, 1, 16, 128, dtype=torch.int8), torch.zeros(2, 1, 1)
    for call in (lambda: tg.QkvSpec(2, 1, 128, f.float()), lambda: tg.QkvSpec(2, 1, 64, f),
                 lambda: tg.KvCache(codes.float(), codes, scale, scale), lambda: tg.KvCache(codes[:, :, :15], codes, scale, scale),
                 lambda: tg.KvBatch(torch.zeros(2), torch.zeros(1), torch.zeros(1, 1), 1),
                 lambda: tg._want(codes, "k", (torch.int8,), (2, 1, 16, 64)),
                 lambda: tg._want(codes.transpose(0, 2), "k", (torch.int8,)),
                 lambda: tg._want(codes, "k", (torch.int8,), device=torch.device("cuda", 0)),
                 lambda: tg._heads_out(torch.zeros(4, 2, 128), "q", 4, 2, 128, -1),
                 lambda: tg._heads_out(torch.zeros(4, 2, 128, dtype=torch.bfloat16), "q", 5, 2, 128, -1),
                 lambda: tg._flag(torch.zeros(1), -1)):
        with pytest.raises(ValueError):
            call()
