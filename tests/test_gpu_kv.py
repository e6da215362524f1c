"""GPU parity of the attention-side operators: norm and rotation, append to the paged int8 cache,
read-back, attention over it, each against the plain 64-bit forms of kv_util; then a decode layer that
uses them between its linears."""
import numpy as np
import pytest
import torch

import bit_gemv_tern_b200 as tg
from kv_util import BLOCK, FLOOR, Paged, bf16, check_attention, norm_rope

pytestmark = pytest.mark.gpu

H8B, H06B = (32, 8, 128), (16, 8, 128)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def spec_of(heads, seed, norm=True, base=1e6, eps=1e-6):
    r = np.random.default_rng(seed)
    g = [bf16(1 + 0.3 * r.standard_normal(heads[2])) if norm else None for _ in range(2)]
    d = [None if x is None else torch.from_numpy(x).to(torch.bfloat16).cuda() for x in g]
    return tg.QkvSpec(*heads, tg.tern_rope_freqs(heads[2], base), *d, eps), g


def rows_of(rows, heads, seed, dtype, stride=None, per=2):
    """A source tensor [rows, width] (a slice of a wider one where `stride` is given) and its values."""
    r = np.random.default_rng(seed)
    width = (heads[0] + per * heads[1]) * heads[2]
    x = (r.standard_normal((rows, width)) * np.exp(0.5 * r.standard_normal((1, width)))).astype(np.float32)
    full = torch.full((rows, stride or width), float("nan"), dtype=dtype, device="cuda")
    full[:, :width] = torch.from_numpy(x).to(dtype).cuda()
    src = full[:, :width] if stride else full
    return src, src.double().cpu().numpy().reshape(rows, -1, heads[2])


def close_bf16(got, ref, size):
    """One rounding to bf16 (2^-8), after fp32 steps whose angle is off by at most 2^-21 and whose norm and
    products add less than 2^-20 of the pair's size."""
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size).all()


@pytest.mark.parametrize("heads", [H8B, H06B, (3, 1, 64), (10, 2, 64), (7, 7, 128)])
@pytest.mark.parametrize("rows,dtype,norm", [(1, torch.float32, True), (7, torch.bfloat16, True), (33, torch.float32, False)])
def test_qk_norm_rope(heads, rows, dtype, norm):
    spec, g = spec_of(heads, 1, norm)
    src, x = rows_of(rows, heads, rows, dtype, stride=(heads[0] + 2 * heads[1]) * heads[2] + 4 if rows == 7 else None)
    pos = np.random.default_rng(2).integers(0, 2_000_000, rows).astype(np.int32)
    pos[0] = 0 if rows > 1 else 1_999_999
    q = torch.zeros(rows, heads[0], heads[2], dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(rows, heads[1], heads[2], dtype=torch.bfloat16, device="cuda")
    tg.tern_qk_norm_rope(spec, src, dev(pos), q, k)
    f = host(spec.freq)
    close_bf16(host(q), *norm_rope(x[:, :heads[0]], g[0], pos, f, 1e-6))
    close_bf16(host(k), *norm_rope(x[:, heads[0]:heads[0] + heads[1]], g[1], pos, f, 1e-6))


def test_qk_norm_rope_many_rows_and_a_zero_row():
    heads, rows = H06B, 2049
    spec, g = spec_of(heads, 3)
    src, x = rows_of(rows, heads, 4, torch.float32, per=1)
    src[5] = 0
    x[5] = 0
    pos = np.arange(rows, dtype=np.int32)[::-1].copy()
    q = torch.zeros(rows, heads[0], heads[2], dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(rows, heads[1], heads[2], dtype=torch.bfloat16, device="cuda")
    tg.tern_qk_norm_rope(spec, src, dev(pos), q, k)
    f = host(spec.freq)
    close_bf16(host(q), *norm_rope(x[:, :heads[0]], g[0], pos, f, 1e-6))
    close_bf16(host(k), *norm_rope(x[:, heads[0]:], g[1], pos, f, 1e-6))


def check_append(P, spec, g, x, before, after, eps=1e-6):
    """Every appended block: its scale, the earlier codes (exactly what the scale makes of them), the new codes (half
    a step, plus the fp32 steps before it: 2^-18 of the pair's size and 2^-17 of the value's 127 steps);
    and nothing else has changed."""
    f = spec.freq.cpu().numpy()
    touched = np.zeros(before[2].shape, bool)
    kept = {w: np.ones(before[i].shape, bool) for i, w in enumerate("kv")}
    for b, (n, kv) in enumerate(P.lens):
        if not n:
            continue
        s0, p0 = P.row_start[b], kv - n
        xb = x[s0:s0 + n]
        new = {"v": (xb[:, P.q_heads + P.kv_heads:], 0 * xb[:, :P.kv_heads]),
               "k": norm_rope(xb[:, P.q_heads:P.q_heads + P.kv_heads], g[1], np.arange(p0, kv), f, eps)}
        for t0 in range(p0 // BLOCK * BLOCK, kv, BLOCK):
            lo, hi = max(t0, p0), min(kv, t0 + BLOCK)
            pg, bl, pl = P.table[b, t0 // P.page], t0 % P.page // BLOCK, t0 % P.page
            touched[pg, :, bl] = True
            for i, w in enumerate("kv"):
                y, size = (a[lo - p0:hi - p0] for a in new[w])
                s, old = after[2 + i][pg, :, bl], before[2 + i][pg, :, bl]
                top = np.abs(y).max((0, 2)) / 127
                want = np.maximum(np.maximum(top, FLOOR), old.astype(np.float64) if lo > t0 else 0.0)
                assert (np.abs(s - want) <= 2.0 ** -17 * want + 2.0 ** -18 * size.max((0, 2)) / 127).all()
                now = after[i][pg, :, pl:pl + BLOCK]
                if lo > t0:
                    c = before[i][pg, :, pl:pl + lo - t0].astype(np.float32)
                    r = np.where(s != old, old / s, np.float32(1)).astype(np.float32)
                    assert (now[:, :lo - t0] == np.rint(c * r[:, None, None])).all()
                got = now[:, lo - t0:hi - t0].astype(np.float64).transpose(1, 0, 2)
                sd = s.astype(np.float64)[None, :, None]
                assert (np.abs(got * sd - y) <= sd * (0.5 + 127 * 2.0 ** -17) + 2.0 ** -18 * size).all()
                assert np.abs(now).max() <= 127
                kept[w][pg, :, pl:pl + hi - t0] = False
    for i, w in enumerate("kv"):
        assert (before[i][kept[w]] == after[i][kept[w]]).all()
        assert (before[2 + i][~touched].view(np.uint32) == after[2 + i][~touched].view(np.uint32)).all()


def run_append(P, spec, g, dtype, seed, stride=None):
    src, x = rows_of(P.rows, (P.q_heads, P.kv_heads, P.D), seed, dtype, stride)
    cache, batch = P.device(tg)
    before = [host(t).copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    q = torch.full((P.rows, P.q_heads, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg.tern_kv_append(spec, src, cache, batch, q, flag)
    after = [host(t).copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    assert tg.tern_read_flag(flag) == tg.TERN_OK
    end = P.row_start[-1]
    pos = np.concatenate([np.arange(kv - n, kv) for n, kv in P.lens]) if end else np.zeros(0)
    if end:
        close_bf16(host(q)[:end], *norm_rope(x[:end, :P.q_heads], g[0], pos, spec.freq.cpu().numpy(), spec.eps))
    assert (host(q)[end:] == 7.0).all()
    check_append(P, spec, g, x, before, after)
    tg.tern_kv_append(spec, src, cache, batch, q, flag)               # the same rows at the same place
    again = [host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    assert all((a.view(np.uint8) == b.view(np.uint8)).all() for a, b in zip(after, again))
    return cache, batch, src


@pytest.mark.parametrize("heads,page,lens", [
    (H8B, 16, [(1, 1)]),
    (H8B, 64, [(1, 1000)]),
    (H06B, 48, [(1, 17), (0, 0), (1, 16), (1, 33), (0, 70)]),
    (H8B, 16, [(3, 20), (15, 31), (16, 32), (1, 1)]),
    ((5, 1, 64), 32, [(17, 17), (40, 73), (1, 64)]),
    ((4, 4, 64), 80, [(1, 31), (2, 2), (9, 200)]),
    ((6, 2, 128), 16, [(100, 100), (33, 65), (0, 5), (64, 64)]),
    (H06B, 128, [(257, 300)]),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append(heads, page, lens, dtype):
    P = Paged(11, heads, page, lens, extra_rows=3)
    spec, g = spec_of(heads, 12)
    run_append(P, spec, g, dtype, 13, stride=(heads[0] + 2 * heads[1]) * heads[2] + 12 if len(lens) > 1 else None)


def test_append_without_norm_and_growing_and_zero_blocks():
    """A block filled token by token: louder ones make its scale grow, quiet and zero ones leave it, and a head of
    zeros gets the smallest scale."""
    heads = (2, 1, 128)
    spec, g = spec_of(heads, 5, norm=False)
    P = Paged(6, heads, 16, [(1, 1)])
    cache, _ = P.device(tg)
    r = np.random.default_rng(7)
    tokens = r.standard_normal((16, 1, 4 * 128)).astype(np.float32)
    tokens *= np.array([1, .5, 0, 2, 2.1, .1, 4, 3, 0, 8, 1, 1, 9, .01, 20, 5], np.float32)[:, None, None]
    for t in range(16):
        P.lens = [(1, t + 1)]
        P.kv_len[:] = t + 1
        _, batch = P.device(tg)
        before = [host(a).copy() for a in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        q = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
        tg.tern_kv_append(spec, dev(tokens[t]), cache, batch, q)
        after = [host(a).copy() for a in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        check_append(P, spec, g, tokens[t].astype(np.float64).reshape(1, 4, 128), before, after)
    P.lens, P.kv_len[:] = [(1, 1)], 1
    _, batch = P.device(tg)
    tg.tern_kv_append(spec, torch.zeros(1, 512, device="cuda"), cache, batch, q)
    pg = P.table[0, 0]
    assert float(cache.v_scale[pg, 0, 0]) == FLOOR and int(cache.v[pg, 0, 0].abs().max()) == 0


@pytest.mark.parametrize("heads,page,lens", [
    (H8B, 16, [(1, 1), (40, 41), (0, 9), (17, 300)]),
    ((3, 3, 64), 48, [(5, 5), (100, 130)]),
    (H06B, 128, [(700, 700)]),
])
def test_read(heads, page, lens):
    P = Paged(21, heads, page, lens, extra_rows=2)
    cache, batch = P.device(tg)
    k, v = (torch.full((P.rows, heads[1], heads[2]), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg.tern_kv_read(cache, batch, k, v, flag)
    for w, got in (("k", host(k)), ("v", host(v))):
        for b, (n, kv) in enumerate(lens):
            # code * scale is one fp32 product (24 bits), then bf16: that double rounding as it is
            t = np.arange(kv - n, kv)
            pg, pl = P.table[b, t // page], t % page
            codes, sc = (P.k, P.ks) if w == "k" else (P.v, P.vs)
            want = codes[pg, :, pl].astype(np.float32) * sc[pg, :, pl // BLOCK][..., None]
            assert (got[P.row_start[b]:P.row_start[b + 1]] == bf16(want)).all()
        assert (got[P.row_start[-1]:] == 3.0).all()
    assert tg.tern_read_flag(flag) == tg.TERN_OK


def workspace(heads):
    return torch.zeros(tg.tern_paged_attn_workspace_bytes(*heads), dtype=torch.uint8, device="cuda")


def run_attn(P, seed, max_rows=None, scale=None, ws=None, loud=1.0):
    heads = (P.q_heads, P.kv_heads, P.D)
    cache, batch = P.device(tg)
    q = torch.from_numpy(bf16(loud * np.random.default_rng(seed).standard_normal((P.rows, *heads[::2])))).to(torch.bfloat16)
    out = torch.full((P.rows, heads[0], heads[2]), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((P.rows, heads[0]), 7.0, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = workspace(heads) if ws is None else ws
    scale = heads[2] ** -0.5 if scale is None else scale
    tg.tern_paged_attn(q.cuda(), scale, cache, batch, out, ws, max_rows or max(n for n, _ in P.lens), lse, flag)
    assert tg.tern_read_flag(flag) == tg.TERN_OK
    assert tg.tern_device_status() == tg.TERN_OK
    check_attention(P, q.double().numpy(), scale, host(out), host(lse))
    end = P.row_start[-1]
    assert (host(out)[end:] == 7.0).all() and (host(lse)[end:] == 7.0).all()
    return out, lse, (q.cuda(), scale, cache, batch), ws


@pytest.mark.parametrize("heads,page,lens", [
    (H8B, 16, [(1, 1)]),
    (H8B, 64, [(1, 1000)]),
    (H06B, 16, [(1, kv) for kv in (0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257)]),
    (H8B, 48, [(1, 3000), (1, 0), (0, 50), (1, 7), (1, 700)]),
    ((16, 1, 128), 32, [(1, 500), (1, 31)]),
    ((5, 1, 64), 16, [(1, 333), (1, 2)]),
    ((21, 3, 64), 80, [(1, 100), (1, 1000), (1, 81)]),
    ((64, 1, 128), 64, [(1, 250)]),
    ((4, 4, 128), 128, [(1, 511), (1, 4000)]),
])
def test_attention_of_one_row(heads, page, lens):
    run_attn(Paged(31, heads, page, lens, extra_rows=1), 32)


@pytest.mark.parametrize("heads,page,lens", [
    (H8B, 64, [(8, 1000), (3, 3), (8, 5), (0, 0), (5, 64)]),
    (H06B, 16, [(2, 2), (2, 300), (4, 17)]),
    ((6, 2, 64), 32, [(16, 400), (7, 31), (11, 12)]),
    (H8B, 48, [(16, 2000), (16, 16)]),
    ((3, 1, 128), 16, [(9, 100), (2, 1), (13, 0)]),
])
def test_attention_of_a_few_rows(heads, page, lens):
    run_attn(Paged(41, heads, page, lens, extra_rows=2), 42)


@pytest.mark.parametrize("heads,page,lens", [
    (H8B, 64, [(128, 128)]),
    (H06B, 16, [(129, 129), (60, 500), (1, 700), (0, 3), (33, 33)]),
    ((5, 1, 64), 48, [(200, 200), (77, 333)]),
    ((2, 2, 128), 128, [(300, 1000), (257, 300)]),
    ((12, 4, 64), 32, [(31, 31), (100, 20), (65, 65)]),
    ((24, 1, 128), 16, [(50, 150)]),
    ((7, 1, 128), 16, [(90, 260), (19, 19)]),
])
def test_attention_of_many_rows(heads, page, lens):
    run_attn(Paged(51, heads, page, lens, extra_rows=2), 52)


@pytest.mark.parametrize("batch", [1, 2, 5])
@pytest.mark.parametrize("heads,n", [(H8B, 9), (H8B, 16), ((12, 4, 64), 21), ((8, 1, 128), 5)])
def test_attention_of_33_to_64_rows_of_a_tile(heads, n, batch):
    P = Paged(69, heads, 32, [(n, 20), (n - 1, 700), (n, n), (0, 9), (n, 3000)][-batch:])
    run_attn(P, 70, max_rows=n)


@pytest.mark.parametrize("max_rows", [1, 4, 16, 10_000])
def test_attention_is_right_whatever_max_rows_says(max_rows):
    run_attn(Paged(61, H06B, 16, [(1, 90), (70, 200), (5, 5), (0, 0), (1, 0)], extra_rows=1), 62, max_rows)


def test_attention_with_sharp_and_flat_scores():
    """Large scores (one key takes everything) and a scale of zero and below."""
    P = Paged(63, H06B, 16, [(1, 200), (20, 100)])
    run_attn(P, 64, loud=30.0)
    run_attn(P, 65, scale=0.0)
    run_attn(P, 66, scale=-0.2)


def test_attention_with_blocks_of_very_different_scales():
    """Value blocks of zeros (the smallest scale) and of 2^20 beside ordinary ones, key blocks of zeros."""
    for n in (1, 40):
        P = Paged(67, (8, 2, 128), 32, [(n, 300), (n, 64)])
        for b, (_, kv) in enumerate(P.lens):
            for t in range(0, kv, BLOCK):
                at = (P.table[b, t // 32], slice(None), t % 32 // BLOCK)
                if t // BLOCK % 3 == 1:
                    P.vs[at] = FLOOR
                    P.v[P.table[b, t // 32], :, t % 32:t % 32 + BLOCK] = 0
                if t // BLOCK % 5 == 4:
                    P.vs[at] *= 2.0 ** 20 if b == 0 else 2.0 ** -20
                if t // BLOCK % 4 == 2:
                    P.ks[at] = FLOOR
        run_attn(P, 68)


def test_attention_over_a_long_cache_and_again():
    """Work split along the cache; the workspace serves the next call; the same bits each time."""
    heads = H8B
    P = Paged(71, heads, 64, [(1, 20_000), (3, 5000), (1, 64)])
    out, lse, (q, scale, cache, batch), ws = run_attn(P, 72)
    assert int(ws[:1024].sum()) == 0
    for _ in range(3):
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        tg.tern_paged_attn(q, scale, cache, batch, out2, ws, 3, lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    run_attn(Paged(73, heads, 16, [(1, 3000)]), 74, ws=ws)


@pytest.mark.parametrize("heads,n", [((4, 1, 64), 1), ((4, 1, 64), 4), ((8, 1, 64), 4), ((8, 1, 128), 1), ((8, 1, 128), 4), ((8, 1, 64), 9)])
def test_attention_of_one_tile_over_every_cta(heads, n):
    """One key/value head and one sequence of 292 chunks of 64 tokens: as many CTAs leave a partial result of the one tile."""
    run_attn(Paged(76, heads, 64, [(n, 18_688)]), 77)


@pytest.mark.parametrize("lens,max_rows", [([(1, 30_000), (1, 900)], 1), ([(4, 12_000)], 4), ([(8, 12_000)], 8), ([(200, 6000)], 200)])
def test_attention_gives_the_same_bits_whether_its_cache_is_cold_or_not(lens, max_rows):
    """Stages that arrive late and out of order (pages scattered over memory, the L2 flushed) change nothing."""
    P = Paged(75, H8B, 64, lens)
    cache, batch = P.device(tg)
    q = torch.randn(P.rows, 32, 128, device="cuda").to(torch.bfloat16)
    ws, flush = workspace(H8B), torch.zeros(64 << 20, device="cuda")
    want = None
    for turn in range(24):
        if turn % 2 == 0:
            flush.add_(1.0)
        out, lse = torch.zeros_like(q), torch.zeros(P.rows, 32, device="cuda")
        tg.tern_paged_attn(q, 0.09, cache, batch, out, ws, max_rows, lse)
        if want is None:
            want = (out, lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), turn
    check_attention(P, q.double().cpu().numpy(), 0.09, host(out), host(lse))


def test_bad_device_data_is_reported_and_left_out():
    """Lengths, row ranges and pages that only the device can see: flagged, nothing outside is touched."""
    heads = (4, 2, 128)
    P = Paged(81, heads, 16, [(2, 40), (2, 33), (1, 20), (2, 50)])
    spec, g = spec_of(heads, 82)
    P.kv_len[1] = P.max_pages * 16 + 1                 # past the table
    P.table[2, 1] = P.pages                            # no such page (its last token's)
    cache, batch = P.device(tg)
    src, x = rows_of(P.rows, heads, 83, torch.float32)
    q = torch.full((P.rows, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    before = host(cache.k).copy()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg.tern_kv_append(spec, src, cache, batch, q, flag)
    assert tg.tern_read_flag(flag) == tg.TERN_EBADCODE
    assert (host(q)[2:4] == 7.0).all() and (host(q)[:2] != 7.0).any() and (host(q)[5:] != 7.0).any()
    changed = np.argwhere((host(cache.k) != before).any((1, 2, 3)))[:, 0]
    assert set(changed) <= {P.table[0, 2], P.table[3, 3]}
    k, v = (torch.full((P.rows, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    flag.zero_()
    tg.tern_kv_read(cache, batch, k, v, flag)
    assert tg.tern_read_flag(flag) == tg.TERN_EBADCODE
    assert (host(k)[2:5] == 3.0).all() and (host(k)[5:] != 3.0).any()
    for max_rows in (2, 500):
        out = torch.full((P.rows, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        flag.zero_()
        tg.tern_paged_attn(torch.ones_like(out), 0.1, cache, batch, out, workspace(heads), max_rows, None, flag)
        assert tg.tern_read_flag(flag) == tg.TERN_EBADCODE
        assert (host(out)[2:4] == 7.0).all() and (host(out)[5:] != 7.0).any()
        # the sequence with the lost page: its 16 present tokens are seen, the others are not
        P2 = Paged(81, heads, 16, [(1, 16)])
        P2.table, P2.k, P2.v, P2.ks, P2.vs = P.table[2:3], host(cache.k), host(cache.v), host(cache.k_scale), host(cache.v_scale)
        check_attention(P2, np.ones((1, 4, 128)), 0.1, host(out)[4:5], None)
    P.row_start[2] = 1                                 # decreasing
    _, batch = P.device(tg)
    flag.zero_()
    tg.tern_kv_read(cache, batch, k, v, flag)
    assert tg.tern_read_flag(flag) == tg.TERN_EBADCODE


def test_captured_calls_follow_the_lengths():
    """Append and attention in one graph on a side stream: replays with other lengths, rows and pages."""
    heads = H06B
    spec, g = spec_of(heads, 91)
    P = Paged(92, heads, 16, [(1, 80)] * 3)            # five pages each
    P.lens = [(1, 15), (0, 0), (1, 64)]
    P.kv_len, P.row_start = np.array([15, 0, 64], np.int32), np.array([0, 1, 1, 2], np.int32)
    cache, batch = P.device(tg)
    ws = workspace(heads)
    src, _ = rows_of(3, heads, 93, torch.float32)
    q, out = (torch.zeros(3, heads[0], 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step(flags):
        tg.tern_kv_append(spec, src, cache, batch, q, flags=flags)
        tg.tern_paged_attn(q, 128 ** -0.5, cache, batch, out, ws, 2, flags=flags)

    with torch.cuda.stream(st):
        step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(tg.TERN_FLAG_PDL)
    for lens in ([(1, 16), (0, 0), (1, 65)], [(0, 16), (2, 2), (1, 66)], [(1, 17), (1, 3), (0, 66)]):
        src.copy_(rows_of(3, heads, 94 + lens[0][1], torch.float32)[0])
        P.lens = lens
        batch.row_start.copy_(dev(np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)))
        batch.kv_len.copy_(dev(np.array([kv for _, kv in lens], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        P.k, P.v, P.ks, P.vs = (host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
        P.row_start = host(batch.row_start)
        check_attention(P, host(q).astype(np.float64), 128 ** -0.5, host(out), None)


def test_decode_layer_between_its_linears():
    """The operators where they are used: q|k|v linear, append, attention, o linear, over a few tokens of a
    batch, in one graph, against the same layer in 64 bits."""
    import oracle
    import synth
    from gpu_util import make_matrix
    heads, d, B = H06B, 1024, 3
    Hq, Hkv, D = heads
    Wqkv, tq, sq = make_matrix(101, 1, (Hq + 2 * Hkv) * D, d)
    Wo, to, so = make_matrix(101, 2, d, Hq * D)
    spec, g = spec_of(heads, 102)
    P = Paged(103, heads, 16, [(1, 30), (1, 1), (1, 200)], spare=0)
    cache, batch = P.device(tg)
    x = torch.zeros(B, d, dtype=torch.int16, device="cuda")
    qkv, y = torch.zeros(B, Wqkv.N, device="cuda"), torch.zeros(B, d, device="cuda")
    q, att = (torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = workspace(heads)
    lin = [tg.GemvBatch([(Wqkv, x, None, qkv)], tg.TERN_ACT_BF16, M=B), tg.GemvBatch([(Wo, att, None, y)], tg.TERN_ACT_BF16, M=B)]

    def step():
        lin[0](tg.TERN_FLAG_PDL)
        tg.tern_kv_append(spec, qkv, cache, batch, q, flags=tg.TERN_FLAG_PDL)
        tg.tern_paged_attn(q, D ** -0.5, cache, batch, att, ws, 1, flags=tg.TERN_FLAG_PDL)
        lin[1](tg.TERN_FLAG_PDL)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for token in range(2):
        bits = synth.activations(104, token, B, d)
        x.copy_(dev(bits.view(np.int16)))
        batch.kv_len.copy_(dev(np.array([30, 1, 200], np.int32) + (token and -1) * np.array([1, 0, 1], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle.gemm_bf16(oracle.pack(tq), sq, d, bits)
        assert np.linalg.norm(host(qkv) - ref) <= 1e-5 * np.linalg.norm(ref)
        kv = host(batch.kv_len)
        P.lens = [(1, int(k)) for k in kv]
        close_bf16(host(q), *norm_rope(host(qkv).astype(np.float64).reshape(B, -1, D)[:, :Hq], g[0], kv - 1, host(spec.freq), 1e-6))
        P.k, P.v, P.ks, P.vs = (host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
        check_attention(P, host(q).astype(np.float64), D ** -0.5, host(att), None)
        a = att.view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, -1)
        ref = oracle.gemm_bf16(oracle.pack(to), so, Hq * D, a)
        assert np.linalg.norm(host(y) - ref) <= 1e-5 * np.linalg.norm(ref)


def test_two_streams_at_once():
    """Two calls with workspaces of their own on two streams."""
    heads = H8B
    Ps = [Paged(111 + i, heads, 64, [(1, 3000 + i), (1, 100)]) for i in range(2)]
    made = [p.device(tg) for p in Ps]
    qs = [torch.from_numpy(bf16(np.random.default_rng(i).standard_normal((2, 32, 128)))).to(torch.bfloat16).cuda() for i in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    wss = [workspace(heads) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            tg.tern_paged_attn(qs[i], 0.09, *made[i], outs[i], wss[i], 1, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_attention(Ps[i], qs[i].double().cpu().numpy(), 0.09, host(outs[i]), None)
