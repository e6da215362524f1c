"""Plain 64-bit forms of the attention-side operators (include/tern.h: norm and rotation, paged int8
cache, attention) and small builders for their tests. Nothing here uses the library."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 16
FLOOR = 2.0 ** -60


def bf16(a: np.ndarray) -> np.ndarray:
    """Nearest bf16 values, as float64."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.float32).to(torch.bfloat16).double().numpy()


def norm_rope(x, gain, pos, freq, eps):
    """x [rows, heads, D] fp64; gain [D] or None; pos [rows]; freq [D/2]."""
    z = np.asarray(x, np.float64)
    D = z.shape[-1]
    if gain is not None:
        z = z / np.sqrt((z ** 2).mean(-1, keepdims=True) + eps) * gain
    a = np.asarray(pos, np.float64)[:, None, None] * freq
    c, s = np.cos(a), np.sin(a)
    lo, hi = z[..., :D // 2], z[..., D // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1), np.tile(np.abs(lo) + np.abs(hi), 2)


class Paged:
    """A cache of random pages and the sequences (n rows, kv tokens) of a call, on the host."""

    def __init__(self, seed, heads, page, lens, spare=2, extra_rows=0, codes=True):
        self.q_heads, self.kv_heads, self.D = heads
        self.page, self.lens = page, list(lens)
        r = np.random.default_rng(seed)
        self.r = r
        need = [-(-kv // page) for _, kv in lens]
        self.pages, self.max_pages = sum(need) + spare, max(max(need), 1)
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.zeros((len(lens), self.max_pages), np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        shape = (self.pages, self.kv_heads, page, self.D)
        self.k = r.integers(-127, 128, shape).astype(np.int8)
        self.v = r.integers(-127, 128, shape).astype(np.int8)
        bl = (self.pages, self.kv_heads, page // BLOCK)
        self.ks = (0.01 * np.exp(0.7 * r.standard_normal(bl))).astype(np.float32)
        self.vs = (0.02 * np.exp(0.7 * r.standard_normal(bl))).astype(np.float32)
        used = np.zeros(bl, bool)                     # blocks of tokens that exist
        for b, (_, kv) in enumerate(lens):
            for t in range(0, kv, BLOCK):
                used[self.table[b, t // page], :, t % page // BLOCK] = True
        self.ks[~used], self.vs[~used] = np.nan, np.inf
        self.row_start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([kv for _, kv in lens], np.int32)
        self.rows = int(self.row_start[-1]) + extra_rows

    def values(self, b, which, upto=None):
        """[kv, kv_heads, D] fp64 values of sequence b's tokens."""
        kv = self.lens[b][1] if upto is None else upto
        codes, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        t = np.arange(kv)
        pg, pl = self.table[b, t // self.page], t % self.page
        return codes[pg, :, pl].astype(np.float64) * scale[pg, :, pl // BLOCK].astype(np.float64)[..., None]

    def device(self, tg):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        cache = tg.KvCache(d(self.k), d(self.v), d(self.ks), d(self.vs))
        return cache, tg.KvBatch(d(self.row_start), d(self.kv_len), d(self.table), self.rows)


def attention(P: Paged, q, scale):
    """(out [rows, Hq, D], lse [rows, Hq], sum p|v| [rows, Hq, D], max |s| bound [rows, Hq], sum |code| times the
    largest p * block scale [rows, Hq, D]) in fp64; q [rows, Hq, D]. Rows of nobody are nan."""
    G = P.q_heads // P.kv_heads
    out = np.full((P.rows, P.q_heads, P.D), np.nan)
    mag, lse = out.copy(), np.full((P.rows, P.q_heads), np.nan)
    size, small = np.zeros((P.rows, P.q_heads)), np.zeros(out.shape)
    for b, (n, kv) in enumerate(P.lens):
        if not n:
            continue
        rows = slice(P.row_start[b], P.row_start[b] + n)
        qb = q[rows]
        out[rows], mag[rows], lse[rows] = 0.0, 0.0, -np.inf
        if not kv:
            continue
        k, v = P.values(b, "k"), P.values(b, "v")
        t = np.arange(kv)
        pg, pl = P.table[b, t // P.page], t % P.page
        codes, vs = np.abs(P.v[pg, :, pl].astype(np.float64)), P.vs[pg, :, pl // BLOCK].astype(np.float64)
        seen = np.arange(kv)[None] <= (kv - n + np.arange(n))[:, None]
        for h in range(P.q_heads):
            s = scale * (qb[:, h] @ k[:, h // G].T)
            size[rows, h] = abs(scale) * (np.abs(qb[:, h]) @ np.abs(k[:, h // G]).T).max(-1)
            s = np.where(seen, s, -np.inf)
            top = np.where(seen.any(1), s.max(1), 0.0)
            e = np.exp(s - top[:, None])
            l = e.sum(1)
            some = l > 0
            p = e / np.where(some, l, 1.0)[:, None]
            out[rows, h] = p @ v[:, h // G]
            mag[rows, h] = p @ np.abs(v[:, h // G])
            small[rows, h] = (p * vs[:, h // G]).max(1)[:, None] * (seen @ codes[:, h // G])
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.where(some, top + np.log(l), -np.inf)
    return out, lse, mag, size, small


def check_attention(P, q, scale, out, lse):
    """Against fp64. The scores carry fp32 sums of D exact products (an error of at most 2^-20 of the sum
    of their magnitudes, the scaling included), which moves every probability by that much twice
    over (itself and the sum); a probability times its block's scale is rounded to fp16 (2^-11); fp32
    sums over the tokens add less than 2^-14 for the lengths tested; one rounding to bf16 (2^-8).
    Below fp16's normal range that rounding is absolute, half of 2^-24 where the largest probability
    times scale of the row is held as 1 (and fp32 holds none below 2^-149): every token may be off by
    2^-25 of that largest one times its code's size."""
    ref, rl, mag, size, small = attention(P, q, scale)
    own = ~np.isnan(rl[:, 0])
    ds = 2.0 ** -20 * size[own]
    got = out[own].astype(np.float64)
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref[own]) + (2.0 ** -11 + 2.0 ** -14 + 2 * ds[..., None]) * mag[own] * (1 + 2.0 ** -8)
    tol += 2.0 ** -25 * small[own]
    bad = np.abs(got - ref[own]) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref[own]) / np.maximum(tol, 1e-300)):.3g} tolerances"
    if lse is not None:
        gl, rl = lse[own].astype(np.float64), rl[own]
        empty = np.isneginf(rl)
        assert (np.isneginf(gl) == empty).all()
        assert (got[empty] == 0).all()
        # a running fp32 sum of N positive terms is off by at most N * 2^-24 of itself
        seen = np.concatenate([np.full(n, kv) for n, kv in P.lens])[:, None]
        tl = ds + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl))) + 2.0 ** -24 * seen
        assert (np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl)) <= tl).all()
