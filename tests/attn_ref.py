"""The paged key-value cache and its attention in numpy and 64 bits: the plain
implementation the GPU tests compare with.  Written from the definitions in
include/qmv.h, byte by byte, with none of the library's code.

Bounds of an attention output (U = 2^-24, per element):
  Products: a query is a sum of two f16 pieces (off by at most 2^-22 of its
  value) or three bf16 pieces (exact), cached values are exact, and the 2 or 3
  times head_dim products are added in f32, in some order: a logit is off by at
  most D = (2^-22 + (3 head_dim + 8) U) A with A = scale * max_t sum_d |q_d K_td|
  (the factors scale, log2 e and an 8-bit row scale: the 8 U, since A is at
  least the logit).
  Weights: 2^x is off by 2 U relative plus the rounding of its argument (x and
  the maximum it is taken against: 4 U A); a weight over the sum thus by 2 D +
  8 U A + 4 U, and its split into pieces by 2^-22.
  Sums: the weights and the weighted values are added chunk by chunk; with at
  most one rounding per position, and those of the joins, (L + 64) U.  Both
  the numerator and the sum carry these.
  All of these are relative to sum_t w_t |V_t|.  With f16 pieces (f16 and
  8-bit caches) there is a floor besides: a weight enters as 2^11 w / w_run,
  w_run at most the row's largest weight w_max, and f16 has a smallest step of
  2^-24, so a small weight is off by up to 2^-25 / 2^11 w_max = 2^-36 w_max.  An
  8-bit row's scale is multiplied in first, brought to at most 1 by a power of
  two, that is by at least half the largest scale: 2^-35 w_max max|V| then covers
  a position, and the number of visible positions times that a row.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
TYPES = {"f16": 1, "bf16": 30, "i8": 24}
SIZE = {"f16": 2, "bf16": 2, "i8": 1}


def head_bytes(t, hd, page):
    return 2 * page * hd * SIZE[t] + (8 * page if t == "i8" else 0)


def round_bf16(x):
    """f32 bits of x rounded to bfloat16, to nearest even (finite x)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16(h):
    return (h.astype(np.uint32) << 16).view(np.float32)


def encode_row(t, x):
    """A row (f32 [hd]) as stored: (array of values' codes, scale or None)."""
    x = np.asarray(x, np.float32)
    if t == "f16":
        return x.astype(np.float16), None
    if t == "bf16":
        return round_bf16(x), None
    d = np.float32(np.max(np.abs(x)) / np.float32(127))
    if d == 0:
        return np.zeros(x.shape, np.int8), d
    return np.clip(np.rint(x / d), -127, 127).astype(np.int8), d


class Cache:
    """A pool of pages in host memory, as include/qmv.h lays it out."""

    def __init__(self, t, kv, hd, page, n_pages, table, seq_len, fill=None):
        self.t, self.kv, self.hd, self.page, self.n_pages = t, kv, hd, page, n_pages
        self.table = np.asarray(table, np.int32)
        self.seq_len = np.asarray(seq_len, np.int32)
        self.hb = head_bytes(t, hd, page)
        self.pool = np.zeros((n_pages, kv, self.hb), np.uint8)
        if fill is not None:
            self.pool[:] = fill
        self.cap = self.table.shape[1] * page

    def _dtype(self):
        return {"f16": np.float16, "bf16": np.uint16, "i8": np.int8}[self.t]

    def parts(self, page, h):
        """Writable views of one head's part of a page: K, V, scales."""
        raw = self.pool[page, h]
        part = self.page * self.hd * SIZE[self.t]
        k = raw[:part].view(self._dtype()).reshape(self.page, self.hd)
        v = raw[part:2 * part].view(self._dtype()).reshape(self.page // 16, self.hd, 16)
        sc = raw[2 * part:].view(np.float32).reshape(2, self.page) if self.t == "i8" else None
        return k, v, sc

    def where(self, s, pos):
        """(page, slot) of a position; page None in a hole or outside the table."""
        if pos < 0 or pos >= self.cap:
            return None, 0
        pg = int(self.table[s, pos // self.page])
        return (pg if 0 <= pg < self.n_pages else None), pos % self.page

    def write(self, s, pos, h, krow, vrow):
        pg, slot = self.where(s, pos)
        if pg is None:
            return
        k, v, sc = self.parts(pg, h)
        k[slot], dk = encode_row(self.t, krow)
        v[slot // 16, :, slot % 16], dv = encode_row(self.t, vrow)
        if sc is not None:
            sc[0, slot], sc[1, slot] = dk, dv

    def append(self, start, k, v):
        """k, v f32 [n][kv][hd]; start as the call takes it."""
        for s in range(len(self.seq_len)):
            m = int(start[s + 1]) - int(start[s])
            for j in range(m):
                r = int(start[s]) + j
                if r < 0 or r >= len(k):
                    continue
                for h in range(self.kv):
                    self.write(s, int(self.seq_len[s]) - m + j, h, k[r, h], v[r, h])

    def rows(self, s, h, length):
        """K, V f64 [length][hd] and whether each position is there (not in a hole)."""
        K, V = np.zeros((length, self.hd)), np.zeros((length, self.hd))
        there = np.zeros(length, bool)
        for p0 in range(0, length, self.page):
            pg, _ = self.where(s, p0)
            if pg is None:
                continue
            m = min(self.page, length - p0)
            k, v, sc = self.parts(pg, h)
            v = v.transpose(0, 2, 1).reshape(self.page, self.hd)
            if self.t == "bf16":
                k, v = from_bf16(np.ascontiguousarray(k)), from_bf16(np.ascontiguousarray(v))
            with np.errstate(all="ignore"):
                kk, vv = k.astype(np.float64), v.astype(np.float64)
                if sc is not None:
                    kk, vv = kk * sc[0][:, None].astype(np.float64), vv * sc[1][:, None].astype(np.float64)
            K[p0:p0 + m], V[p0:p0 + m] = kk[:m], vv[:m]
            there[p0:p0 + m] = True
        return K, V, there

    def length(self, s, max_len):
        return int(min(max(self.seq_len[s], 0), min(max_len, self.cap)))


def attention(cache, start, q, scale, max_len, window=0, sinks=0, acc=None):
    """Outputs f64 [n][heads][hd], their bounds, and acc with the weights added
    (and acc's bounds).  Rows of no sequence are NaN in the outputs."""
    n, heads, hd = q.shape
    g = heads // cache.kv
    out = np.full((n, heads, hd), np.nan)
    tol = np.zeros((n, heads, hd))
    acc = None if acc is None else acc.astype(np.float64).copy()
    acc_tol = None if acc is None else np.zeros(acc.shape)
    for s in range(len(cache.seq_len)):
        m = int(start[s + 1]) - int(start[s])
        length = cache.length(s, max_len)
        lo, hi = max(0, int(start[s])), min(n, int(start[s + 1]))
        if hi <= lo:
            continue
        pos = length - m + (np.arange(lo, hi) - int(start[s]))
        t = np.arange(length)
        see = t[None, :] <= pos[:, None]
        if window > 0:
            see &= (t[None, :] > pos[:, None] - window) | (t[None, :] < sinks)
        for h in range(cache.kv):
            K, V, there = cache.rows(s, h, length)
            K[~there], V[~there] = 0, 0
            ok = see & there[None, :]
            for i in range(h * g, (h + 1) * g):
                qi = q[lo:hi, i].astype(np.float64)
                if length == 0:
                    out[lo:hi, i] = 0
                    continue
                x = qi @ K.T * scale
                A = (np.abs(qi) @ np.abs(K).T * abs(scale))
                A = np.where(ok, A, 0).max(1)
                x[~ok] = -np.inf
                mx = x.max(1)
                mx = np.where(np.isfinite(mx), mx, 0)
                w = np.exp(x - mx[:, None])
                l = w.sum(1)
                w /= np.where(l > 0, l, 1)[:, None]
                out[lo:hi, i] = w @ V
                D = (2.0 ** -22 + (3 * hd + 8) * U) * A
                rel = 2 * D + 8 * U * A + 4 * U + 2.0 ** -22
                tol[lo:hi, i] = (rel + 2 * (length + 64) * U)[:, None] * (w @ np.abs(V)) + 1e-37
                if cache.t != "bf16":
                    big = np.where(ok, np.abs(V).max(1)[None, :], 0).max(1)
                    tol[lo:hi, i] += (2.0 ** -35 * w.max(1) * big * ok.sum(1))[:, None]
                if acc is not None:
                    acc[s, h, :length] += w.sum(0)
                    acc_tol[s, h, :length] += ((rel + (length + 64) * U)[:, None] * w).sum(0)
    if acc is not None:
        acc_tol += (heads // cache.kv * max(1, n // len(cache.seq_len)) + 2) * U * np.abs(acc) + 1e-37
    return out, tol, acc, acc_tol


def evict(cache, dst, keep, first, recent, acc):
    """Writes the kept rows into the pages of dst; returns kept, acc_out, len_out."""
    n_seq = len(cache.seq_len)
    kept = np.full((n_seq, cache.kv, keep), -1, np.int32)
    acc_out = np.zeros((n_seq, cache.kv, keep), np.float32)
    len_out = np.zeros(n_seq, np.int32)
    old = cache.pool.copy()
    src = Cache(cache.t, cache.kv, cache.hd, cache.page, cache.n_pages, cache.table, cache.seq_len)
    src.pool = old
    to = Cache(cache.t, cache.kv, cache.hd, cache.page, cache.n_pages, dst, cache.seq_len)
    to.pool = cache.pool
    for s in range(n_seq):
        length = cache.length(s, acc.shape[2])
        len_out[s] = min(length, keep)
        for h in range(cache.kv):
            if length <= keep:
                chosen = list(range(length))
            else:
                mid = range(first, length - recent)
                rank = sorted(mid, key=lambda p: (-np.inf if np.isnan(acc[s, h, p]) else 0, -float(acc[s, h, p]), p))
                chosen = sorted(list(range(first)) + rank[:keep - first - recent] + list(range(length - recent, length)))
            for i, p in enumerate(chosen):
                kept[s, h, i], acc_out[s, h, i] = p, acc[s, h, p]
                dpg, dslot = to.where(s, i)
                if dpg is None:
                    continue
                k, v, sc = to.parts(dpg, h)
                pg, slot = src.where(s, p)
                if pg is None:
                    k[dslot], v[dslot // 16, :, dslot % 16] = 0, 0
                    if sc is not None:
                        sc[:, dslot] = 0
                    continue
                k0, v0, sc0 = src.parts(pg, h)
                k[dslot], v[dslot // 16, :, dslot % 16] = k0[slot], v0[slot // 16, :, slot % 16]
                if sc is not None:
                    sc[:, dslot] = sc0[:, slot]
    return kept, acc_out, len_out
