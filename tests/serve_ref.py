"""What stands around a cache's attention, in numpy and 64 bits: 4-bit caches,
norms and rotation of queries and keys, pages taken and given back.  Written
from the definitions in include/qmv.h with none of the library's code.

Bounds of a rotation's output (U = 2^-24): the squares are summed in f32, at most
HD / lanes + log2(lanes) <= 13 roundings of positive terms, so the root's inverse
is off by 7 U, and 5 roundings (mean, root, division, two products) follow: 12 U
relative of a normed value, 0 without a norm.  Cosine and sine: the angle's whole
turns go in 64 bits (t 2^-52, and the product t itself is the same rounded f64 in
both), the rest, below 0.8, is rounded to f32 twice (2 U), the series and its
rounding are below 2 U.  Each output is two products and a sum: 3 U.  In all
(20 U + 2^-51 |t|) (|a| + |b|), of the normed a and b.
"""
from __future__ import annotations

import numpy as np

from tests import attn_ref as ref

U = 2.0 ** -24


def f16_bits(x):
    return np.asarray(x, np.float16).view(np.uint16)


def encode4(x):
    """Blocks of 32 f32 values [..., 32]: codes + 8 (uint8) and f16 scales [...]."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        hi, lo = x.max(-1), x.min(-1)          # (NaN where a value is)
        v = np.where(hi >= -lo, hi, lo).astype(np.float32) * np.float32(-0.125)
        nan = np.isnan(x).any(-1)
        d = ref.from_bf16(ref.round_bf16(np.where(nan, 0, np.clip(v, -1e30, 1e30)).astype(np.float32)))
        d = np.clip(d, -2720, 2720).astype(np.float16)
        f = d.astype(np.float32)[..., None]
        code = np.where(f == 0, 0, np.rint((x / np.where(f == 0, 1, f)).astype(np.float32)))
        code = np.where(np.isnan(code), -8, np.clip(code, -8, 7))   # (a NaN among finite ones: any code)
        d = np.where(nan, np.float16(np.nan), d)
        code = np.where(nan[..., None], 0, code)
    return (code + 8).astype(np.uint8), d


PLACE = np.array([p & ~3 | (p & 1) << 1 | p >> 1 & 1 for p in range(16)])


class Cache4(ref.Cache):
    """A pool of 4-bit pages in host memory."""

    def __init__(self, kv, hd, page, n_pages, table, seq_len, fill=None):
        self.t, self.kv, self.hd, self.page, self.n_pages = "q4", kv, hd, page, n_pages
        self.table, self.seq_len = np.asarray(table, np.int32), np.asarray(seq_len, np.int32)
        self.hb = page * hd * 9 // 8
        self.pool = np.zeros((n_pages, kv, self.hb), np.uint8)
        if fill is not None:
            self.pool[:] = fill
        self.cap = self.table.shape[1] * page

    def parts4(self, page, h):
        """Codes of K [page][hd/2] and V [page/16][hd/2][16], scales of K [page][hd/32] and V [hd/32][page]."""
        raw, half, sc = self.pool[page, h], self.page * self.hd // 2, self.page * self.hd // 16
        return (raw[:half].reshape(self.page, self.hd // 2), raw[half:2 * half].reshape(-1, self.hd // 2, 16),
                raw[2 * half:2 * half + sc].view(np.float16).reshape(self.page, -1),
                raw[2 * half + sc:].view(np.float16).reshape(-1, self.page))

    def write(self, s, pos, h, krow, vrow):
        pg, slot = self.where(s, pos)
        if pg is None:
            return
        k, v, ks, vs = self.parts4(pg, h)
        (uk, dk), (uv, dv) = encode4(krow.reshape(-1, 32)), encode4(vrow.reshape(-1, 32))
        k[slot] = (uk[:, :16] | uk[:, 16:] << 4).reshape(-1)
        v[slot // 16, :, PLACE[slot % 16]] = (uv[:, :16] | uv[:, 16:] << 4).reshape(-1)
        ks[slot], vs[:, slot] = dk, dv

    def page_values(self, pg, h):
        k, v, ks, vs = self.parts4(pg, h)
        v = v[:, :, PLACE].transpose(0, 2, 1).reshape(self.page, -1)
        out = []
        with np.errstate(all="ignore"):
            for codes, d in ((k, ks), (v, vs.T)):
                b = codes.reshape(self.page, -1, 16)
                u = np.concatenate([b & 15, b >> 4], -1).astype(np.float64) - 8
                out.append((u * d.astype(np.float64)[..., None]).reshape(self.page, self.hd))
        return out

    def rows(self, s, h, length):
        K, V = np.zeros((length, self.hd)), np.zeros((length, self.hd))
        there = np.zeros(length, bool)
        for p0 in range(0, length, self.page):
            pg, _ = self.where(s, p0)
            if pg is None:
                continue
            m = min(self.page, length - p0)
            k, v = self.page_values(pg, h)
            K[p0:p0 + m], V[p0:p0 + m], there[p0:p0 + m] = k[:m], v[:m], True
        return K, V, there

    def fill_pages(self, rng, kscale=(0.1, 0.35), vscale=(0.05, 0.2)):
        """Random codes and scales (8 bits of significand, both signs) in every slot of the live pages."""
        for pg in {int(p) for p in self.table.reshape(-1) if 0 <= p < self.n_pages}:
            for h in range(self.kv):
                k, v, ks, vs = self.parts4(pg, h)
                k[:] = rng.integers(0, 256, k.shape)
                v[:] = rng.integers(0, 256, v.shape)
                for d, (lo, hi) in ((ks, kscale), (vs, vscale)):
                    x = rng.uniform(lo, hi, d.shape) * rng.choice([-1.0, 1.0], d.shape)
                    d[:] = ref.from_bf16(ref.round_bf16(x.astype(np.float32)))


def copy_row4(c, src, dst, h):
    """One position's row of head h from (page, slot) to (page, slot); page None: zeros."""
    k1, v1, ks1, vs1 = c.parts4(dst[0], h)
    if src[0] is None:
        k1[dst[1]], v1[dst[1] // 16, :, PLACE[dst[1] % 16]], ks1[dst[1]], vs1[:, dst[1]] = 0, 0, 0, 0
        return
    k0, v0, ks0, vs0 = c.parts4(src[0], h)
    k1[dst[1]], ks1[dst[1]], vs1[:, dst[1]] = k0[src[1]], ks0[src[1]], vs0[:, src[1]]
    v1[dst[1] // 16, :, PLACE[dst[1] % 16]] = v0[src[1] // 16, :, PLACE[src[1] % 16]]


def rope(x, weight, pos, freq, rot, pairs, eps):
    """x f32 [rows][heads][hd] normed and turned in f64, and the bound of each value."""
    x = x.astype(np.float64)
    rel = 0.0
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight.astype(np.float64)
        rel = 12 * U
    out, tol = x.copy(), np.abs(x) * rel + 1e-38
    if rot:
        i = np.arange(rot // 2)
        a, b = (i, i + rot // 2) if pairs == "halves" else (2 * i, 2 * i + 1)
        t = (pos.astype(np.float64)[:, None] * freq)[:, None, :]
        c, s = np.cos(t), np.sin(t)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
        tol[..., a] = tol[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * (20 * U + 2.0 ** -51 * np.abs(t)) + 1e-38
    return out, tol


class Pages:
    """Table, lengths and free stack on the host, a page at a time."""

    def __init__(self, table, seq_len, free, count, page, n_pages):
        self.table, self.seq_len = np.array(table, np.int32), np.array(seq_len, np.int32)
        self.free, self.count = np.array(free, np.int32), int(count)
        self.page, self.n_pages = page, n_pages

    def _pages(self, length):
        return -(-length // self.page)

    def release(self, new_len):
        cap = self.table.shape[1] * self.page
        self.count = min(max(self.count, 0), self.n_pages)
        for s in reversed(range(len(self.seq_len))):
            length, to = min(max(int(self.seq_len[s]), 0), cap), int(new_len[s])
            if to < 0 or to >= length:
                continue
            for j in reversed(range(self._pages(to), self._pages(length))):
                pg = int(self.table[s, j])
                if 0 <= pg < self.n_pages and self.count < self.n_pages:
                    self.free[self.count] = pg
                    self.count += 1
                self.table[s, j] = -1
            self.seq_len[s] = to

    def reserve(self, add, n):
        cap = self.table.shape[1] * self.page
        self.count = min(max(self.count, 0), self.n_pages)
        left = self.count
        need_all = rows_all = 0
        granted, start, pos, slot = [], [0], [], []
        for s in range(len(self.seq_len)):
            length, a = int(self.seq_len[s]), int(add[s])
            got = 0
            if a > 0 and length >= 0 and length + a <= cap:
                need = self._pages(length + a) - self._pages(length)
                need_all += need
                rows_all += a
                if rows_all <= n and (need == 0 or need_all <= left):
                    got = a
            for p in range(length, length + got):
                if p % self.page == 0:
                    self.count -= 1
                    self.table[s, p // self.page] = self.free[self.count]
                pg = int(self.table[s, p // self.page])
                pos.append(p)
                slot.append(pg * self.page + p % self.page if 0 <= pg < self.n_pages else -1)
            self.seq_len[s] += got
            granted.append(got)
            start.append(start[-1] + got)
        rest = [-1] * (n - len(pos))
        return (np.array(granted, np.int32), np.array(start, np.int32), np.array(pos + rest, np.int32),
                np.array(slot + rest, np.int64))
