"""GPU parity of the attention-side operators where they can go wrong: scales of zero, a long flat tail beside one
strong token, batches above a block of the plan, far positions, large pages, queries that are not finite, calls
without rows; each against the plain 64-bit forms of kv_util."""
import numpy as np
import pytest
import torch

import bit_gemv_tern_b200 as tg
from kv_util import BLOCK, Paged, attention, bf16, check_attention, norm_rope
from test_gpu_kv import H06B, H8B, check_append, close_bf16, dev, host, rows_of, run_append, run_attn, spec_of, workspace

pytestmark = pytest.mark.gpu


# (1 .. 8, 9 .. 16, 17 .. 32 rows of a tile, and the tile kernel)
FEW_AND_MANY = [([(1, 300), (1, 40)], 1), ([(3, 300), (4, 65)], 4), ([(8, 300), (5, 30)], 8), ([(100, 300), (40, 40)], 100)]


@pytest.mark.parametrize("lens,max_rows", FEW_AND_MANY)
def test_attention_over_blocks_with_a_scale_of_zero(lens, max_rows):
    """Blocks of zeros by their scale, as another quantiser may leave them, beside ordinary ones: their tokens keep
    their weight. Every row sees the ordinary block 0, beside whose values 127 * 2^-60 does not count."""
    P = Paged(121, (8, 2, 128), 32, lens)
    for b, (_, kv) in enumerate(lens):
        for t in range(0, kv, BLOCK):
            at = (P.table[b, t // 32], slice(None), t % 32 // BLOCK)
            if t // BLOCK % 3 == 1:
                P.vs[at] = 0.0
            if t // BLOCK % 4 == 2:
                P.ks[at] = 0.0
            if t // BLOCK % 5 == 4:
                P.vs[at] = 2.0 ** -70                      # counts as 2^-60
    run_attn(P, 122, max_rows)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("lens,max_rows", FEW_AND_MANY)
def test_attention_over_a_cache_of_zeros(lens, max_rows, codes):
    """A cache filled with zeros (codes too, or scales alone) weighs all tokens alike: the outputs are zero (a code of a
    block without a scale may stand for up to 127 * 2^-60), the log of the sum is that of the tokens seen."""
    P = Paged(123, (8, 2, 128), 16, lens)
    P.ks[:], P.vs[:] = 0.0, 0.0
    if codes:
        P.k[:], P.v[:] = 0, 0
    cache, batch = P.device(tg)
    q = torch.randn(P.rows, 8, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((P.rows, 8), 7.0, device="cuda")
    tg.tern_paged_attn(q, 0.1, cache, batch, out, workspace((8, 2, 128)), max_rows, lse)
    assert (np.abs(host(out)) <= (0.0 if codes else 127 * 2.0 ** -60 * (1 + 2.0 ** -8))).all()
    seen = np.concatenate([kv - n + 1 + np.arange(n) for n, kv in lens])[:, None]
    # The sum of equal terms in fp32 (2^-24 of it each); it holds the terms times 2^60, so that its logarithm of base 2
    # is below 60 + log2(300) < 69 and off by an ulp there, 2^-17; the largest exponent, of a size below 61, is off by
    # half of one, 2^-19. Their sum is exact to 2^-24 of it, and ln 2 * (2^-17 + 2^-19) < 2^-17.
    assert (np.abs(host(lse) - np.log(seen)) <= 2.0 ** -17 + 2.0 ** -22 * np.log(seen) + 2.0 ** -24 * seen).all()


def test_captured_rotations_follow_frequencies_written_just_before():
    """The frequencies rewritten by the kernel in front of a rotation and of an append with programmatic dependent launch."""
    heads, rows = H06B, 40
    spec, g = spec_of(heads, 131)
    src, x = rows_of(rows, heads, 132, torch.float32)
    P = Paged(133, heads, 16, [(rows, 100)])
    cache, batch = P.device(tg)
    pos = np.arange(60, 100, dtype=np.int32)
    pos_dev, new = dev(pos), spec.freq.clone()
    q, qa = (torch.zeros(rows, heads[0], 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.zeros(rows, heads[1], 128, dtype=torch.bfloat16, device="cuda")

    def step():
        spec.freq.copy_(new)
        tg.tern_qk_norm_rope(spec, src, pos_dev, q, k, flags=tg.TERN_FLAG_PDL)
        spec.freq.mul_(2.0)
        tg.tern_kv_append(spec, src, cache, batch, qa, flags=tg.TERN_FLAG_PDL)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for base in (1e4, 1e6, 5e2):
        new.copy_(tg.tern_rope_freqs(128, base))
        graph.replay()
        torch.cuda.synchronize()
        f = host(new)
        close_bf16(host(q), *norm_rope(x[:, :heads[0]], g[0], pos, f, spec.eps))
        close_bf16(host(k), *norm_rope(x[:, heads[0]:heads[0] + heads[1]], g[1], pos, f, spec.eps))
        close_bf16(host(qa), *norm_rope(x[:, :heads[0]], g[0], pos, 2 * f, spec.eps))


@pytest.mark.parametrize("heads,lens", [
    (H8B, [(1, 3000)] * 64),
    (H8B, [(4, 3000)] * 32),
    (H8B, [(8, 3000)] * 16),
    (H06B, [(100, 3000), (64, 1500)]),
])
def test_attention_keeps_a_long_flat_tail_beside_one_strong_token(heads, lens):
    """The first token holds nearly all of the probability and a value of zero, every other one 2^-26.5 of its share: the
    output is the tail's sum. The second product takes a probability times its block's scale in fp16, the largest of a
    row at 2^7 or above, so that one below 2^-24 there, 2^-31 of the largest, is off by 2^-25 there at most, 2^-32
    of the largest; fp32 sums over the tokens and the other terms as in kv_util.check_attention."""
    P = Paged(141, heads, 64, lens)
    P.k[:], P.vs[:] = 0, 0.02
    P.v[:] = np.abs(P.v.astype(np.int16)).clip(1, 127).astype(np.int8)
    for b in range(len(lens)):
        page = P.table[b, 0]
        P.k[page, :, 0, 0], P.v[page, :, 0], P.ks[page, :, 0] = 127, 0, 0.01
    q = np.random.default_rng(142).standard_normal((P.rows, heads[0], heads[2]))
    q[:, :, 0] = 13.0
    q = bf16(q)
    scale = 26.5 * np.log(2.0) / (13.0 * 127 * np.float32(0.01))
    cache, batch = P.device(tg)
    out = torch.zeros(P.rows, heads[0], heads[2], dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(P.rows, heads[0], device="cuda")
    tg.tern_paged_attn(torch.from_numpy(q).to(torch.bfloat16).cuda(), scale, cache, batch, out, workspace(heads), max(n for n, _ in lens), lse)
    ref, rl, mag, size, small = attention(P, q, np.float64(np.float32(scale)))
    got, ds = host(out).astype(np.float64), 2.0 ** -20 * size[..., None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14 + 2 * ds) * mag * (1 + 2.0 ** -8) + 2.0 ** -32 * small
    assert (tol[:, :, 0].min(1) < 0.2 * ref[:, :, 0].min(1)).all()           # the tail is well above what may be lost
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)
    assert (np.abs(host(lse) - rl) <= ds[..., 0] + 2.0 ** -20 * (1 + np.abs(rl)) + 2.0 ** -24 * 3000).all()


def test_calls_without_rows_leave_everything_alone():
    """Tensors of zero rows have no address: such calls are fine and launch nothing."""
    heads = H06B
    P = Paged(151, heads, 16, [(0, 20), (0, 0)])
    cache, batch = P.device(tg)
    spec, _ = spec_of(heads, 152)
    before = [host(t).copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    none = lambda *s, t=torch.bfloat16: torch.zeros(0, *s, dtype=t, device="cuda")  # noqa: E731
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    src, q, k = none(32 * 128, t=torch.float32), none(16, 128), none(8, 128)
    tg.tern_qk_norm_rope(spec, src, none(t=torch.int32), q, k)
    tg.tern_kv_append(spec, src, cache, batch, q, flag)
    tg.tern_kv_read(cache, batch, k, none(8, 128), flag)
    tg.tern_paged_attn(q, 0.1, cache, batch, none(16, 128), workspace(heads), 1, none(16, t=torch.float32), flag)
    assert tg.tern_read_flag(flag) == tg.TERN_OK
    for a, t in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert (a.view(np.uint8) == host(t).view(np.uint8)).all()


def far_rope(x, gain, pos, freq):
    """norm_rope of kv_util with the angles in extended precision."""
    D = x.shape[-1]
    z = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * gain
    a = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)
    a = a - np.rint(a / (2 * np.longdouble(np.pi))) * (2 * np.longdouble("3.14159265358979323846264338327950288"))
    c, s = np.cos(a).astype(np.float64)[:, None], np.sin(a).astype(np.float64)[:, None]
    lo, hi = z[..., :D // 2], z[..., D // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1), np.tile(np.abs(lo) + np.abs(hi), 2)


def test_qk_norm_rope_at_the_last_positions():
    """Up to 2^31 - 1: the angle is a product in fp64 of at most 2^31 / (2 pi) turns, off by 6.2e-8 of a turn (3 * 2^-53
    of it at most, 2^-20 in radians), within close_bf16's 2^-18 together with the sine's 2^-21."""
    heads, rows = H8B, 130
    spec, g = spec_of(heads, 161)
    src, x = rows_of(rows, heads, 162, torch.float32)
    pos = np.concatenate([2 ** 31 - 1 - np.arange(65), np.random.default_rng(163).integers(2 ** 30, 2 ** 31, 65)]).astype(np.int32)
    q = torch.zeros(rows, heads[0], 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(rows, heads[1], 128, dtype=torch.bfloat16, device="cuda")
    tg.tern_qk_norm_rope(spec, src, dev(pos), q, k)
    f = host(spec.freq)
    close_bf16(host(q), *far_rope(x[:, :heads[0]], g[0], pos, f))
    close_bf16(host(k), *far_rope(x[:, heads[0]:heads[0] + heads[1]], g[1], pos, f))


def test_append_and_read_at_the_end_of_the_longest_table():
    """Rows whose tokens are the last of 32766 pages of 65536, all the same page of memory but the last two."""
    heads, page, pages = (2, 1, 64), 65536, 32766
    spec, g = spec_of(heads, 165)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    table[0, -2], table[0, -1] = 2, 1
    kv, n = (pages - 1) * page + 20, 50                # 30 tokens in the last but one page, 20 in the last
    codes = [torch.zeros(3, 1, page, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(3, 1, page // BLOCK, device="cuda") for _ in range(2)]
    cache = tg.KvCache(*codes, *scales)
    batch = tg.KvBatch(dev(np.array([0, n], np.int32)), dev(np.array([kv], np.int32)), table, n)
    src, x = rows_of(n, heads, 166, torch.float32)
    q = torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg.tern_kv_append(spec, src, cache, batch, q, flag)
    tg.tern_kv_read(cache, batch, k, v, flag)
    assert tg.tern_read_flag(flag) == tg.TERN_OK
    f, pos = host(spec.freq), np.arange(kv - n, kv)
    close_bf16(host(q), *far_rope(x[:, :2], g[0], pos, f))
    want, size = far_rope(x[:, 2:3], g[1], pos, f)
    for got, y, sz in ((host(k), want, size), (host(v), x[:, 3:], 0 * size)):
        # half a step of the block's 127 (the largest of its appended rows: none came before), then bf16
        blocks = pos // BLOCK
        top = np.array([np.abs(y[blocks == b]).max() for b in blocks])[:, None, None]
        assert (np.abs(got - y) <= top / 127 * (0.5 + 2.0 ** -9) + 2.0 ** -8 * np.abs(y) + 2.0 ** -17 * (sz + top)).all()
    assert not codes[0][0].any() and not codes[1][0].any()
    assert codes[0][2, 0, -30:].any(1).all() and codes[0][1, 0, :20].any(1).all() and not codes[0][1, 0, 20:].any()


@pytest.mark.parametrize("lens,max_rows", [([(1, 20_000)] * 2, 1), ([(4, 9000)] * 3, 4), ([(8, 9000)] * 3, 8), ([(200, 6000), (130, 900)], 200)])
def test_attention_leaves_every_counter_of_its_workspace_zero(lens, max_rows):
    """Tiles that many CTAs share: their counters (the workspace's first 8192 bytes) serve the next call."""
    _, _, _, ws = run_attn(Paged(171, H8B, 64, lens), 172, max_rows)
    assert not ws[:8192].any()
    assert ws[8192:].any()                              # there were partial results


def many(count, n_most, empty, seed):
    """Lengths of many short sequences, among them some without rows, without tokens, and (`empty`) rows that see nothing."""
    r = np.random.default_rng(seed)
    lens = []
    for b in range(count):
        n = int(r.integers(0, n_most + 1))
        kv = int(r.integers(0, 40)) + (0 if empty else n)
        lens.append((n, 0 if empty and b % 17 == 3 else kv))
    lens[-1] = (n_most, n_most + 33)
    return lens


@pytest.mark.parametrize("count", [192, 193, 256, 257, 512, 513, 1200])
@pytest.mark.parametrize("heads,n_most,max_rows", [((4, 2, 64), 1, 1), ((8, 2, 128), 3, 3), ((8, 2, 128), 6, 6), ((4, 1, 64), 5, 500)])
def test_attention_of_batches_above_a_block_of_the_plan(count, heads, n_most, max_rows):
    run_attn(Paged(181, heads, 16, many(count, n_most, True, count), extra_rows=2), 182, max_rows)


@pytest.mark.parametrize("count", [256, 257, 700])
@pytest.mark.parametrize("n_most", [1, 3, 40])
def test_append_to_batches_above_a_block(count, n_most):
    heads = (2, 1, 64)
    P = Paged(183, heads, 32, many(count, n_most, False, count + 1), extra_rows=1)
    spec, g = spec_of(heads, 184)
    cache, batch, _ = run_append(P, spec, g, torch.float32, 185)
    k, v = (torch.full((P.rows, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tg.tern_kv_read(cache, batch, k, v)
    P.k, P.v, P.ks, P.vs = (host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    for w, got in (("k", host(k)), ("v", host(v))):
        for b, (n, kv) in enumerate(P.lens):
            if n:                                       # an exact product of 8 and 24 bits, to fp32 and to bf16
                want = P.values(b, w)[kv - n:].astype(np.float32)
                assert (got[P.row_start[b]:P.row_start[b + 1]] == bf16(want)).all()
        assert (got[P.row_start[-1]:] == 3.0).all()


@pytest.mark.parametrize("page", [192, 256, 1040, 65536])
def test_large_pages(page):
    heads = (4, 2, 64)
    P = Paged(191, heads, page, [(1, 2500), (70, 1300), (6, 6)], spare=0)
    spec, g = spec_of(heads, 192)
    run_append(P, spec, g, torch.float32, 193)
    for max_rows in (1, 8, 500):
        run_attn(Paged(194, heads, page, [(1, 2500), (70, 1300), (6, 6)], spare=0), 195, max_rows)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,max_rows", [([(1, 300), (1, 40)], 1), ([(3, 300), (4, 65)], 4), ([(8, 300), (5, 30)], 8), ([(100, 300), (40, 40)], 100)])
def test_a_query_that_is_not_finite_spoils_its_own_row_and_head_only(lens, max_rows, bad):
    P = Paged(201, (8, 2, 128), 32, lens)
    P.k[..., 5][P.k[..., 5] == 0] = 1                   # +-infinity or nan scores, and both signs of infinity in every block
    P.k[:, :, ::2, 5], P.k[:, :, 1::2, 5] = np.abs(P.k[:, :, ::2, 5].astype(np.int16)).astype(np.int8), -np.abs(P.k[:, :, 1::2, 5].astype(np.int16)).astype(np.int8)
    cache, batch = P.device(tg)
    q = torch.from_numpy(bf16(np.random.default_rng(202).standard_normal((P.rows, 8, 128)))).to(torch.bfloat16)
    row, head = int(P.row_start[1]) - 1, 3
    dirty = q.clone()
    dirty[row, head, 5] = bad
    ws, got = workspace((8, 2, 128)), []
    for x in (q, dirty):
        out, lse = torch.full((P.rows, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((P.rows, 8), 7.0, device="cuda")
        tg.tern_paged_attn(x.cuda(), 0.09, cache, batch, out, ws, max_rows, lse)
        got.append((host(out), host(lse)))
    (out, lse), (out2, lse2) = got
    assert np.isnan(out2[row, head]).all() and np.isnan(lse2[row, head])
    out2[row, head], lse2[row, head] = out[row, head], lse[row, head]
    check_attention(P, q.double().numpy(), 0.09, out2, lse2)
