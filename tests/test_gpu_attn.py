"""GPU parity of the paged key-value cache calls (append, decode and prompt
attention, eviction) with the 64-bit implementation in attn_ref.py, whose
docstring derives the bounds.  Cached bytes and kept positions have to be equal."""
import numpy as np
import pytest

import synth
from tests import attn_ref as ref
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gguf_dequant_matvec_amd as q  # noqa: E402

NAN_FILL = {"f16": 0xFF, "bf16": 0xFF, "i8": 0xFF}   # 0xFFFF is a NaN in f16, bf16 and f32


def make_cache(t, kv, hd, page, lens, seed, extra_pages=3, cap_pages=None, spare=0):
    """A host cache with the pages scattered over the pool, every slot NaN, then
    positions 0 .. len - 1 of every sequence written with random rows."""
    rng = synth.rng(seed, synth.T_X)
    per = cap_pages or max(1, -(-max(max(lens), 1) // page))
    n_pages = len(lens) * per + extra_pages + spare
    ids = rng.permutation(n_pages - spare)[:len(lens) * per]
    c = ref.Cache(t, kv, hd, page, n_pages, ids.reshape(len(lens), per), lens, fill=NAN_FILL[t])
    for s, length in enumerate(lens):
        if length <= 0:
            continue
        k = rng.standard_normal((length, kv, hd), dtype=np.float32)
        v = rng.standard_normal((length, kv, hd), dtype=np.float32) * np.float32(0.5)
        _fill(c, s, k, v)
    return c, rng


def _fill(c, s, k, v):
    """Rows 0 .. of sequence s, page by page (the row-by-row append is slow in numpy)."""
    length = len(k)
    for p0 in range(0, length, c.page):
        pg, _ = c.where(s, p0)
        m = min(c.page, length - p0)
        for h in range(c.kv):
            kk, vv, sc = c.parts(pg, h)
            for x, put in ((k, 0), (v, 1)):
                rows = x[p0:p0 + m, h]
                if c.t == "i8":
                    d = (np.abs(rows).max(1) / np.float32(127)).astype(np.float32)
                    code = np.clip(np.rint(rows / np.where(d == 0, 1, d)[:, None]), -127, 127).astype(np.int8)
                    sc[put, :m] = d
                else:
                    code = rows.astype(np.float16) if c.t == "f16" else ref.round_bf16(rows)
                if put == 0:
                    kk[:m] = code
                else:
                    slots = np.arange(m)
                    vv[slots // 16, :, slots % 16] = code


class Dev:
    """A host cache's copy on the device."""

    def __init__(self, c):
        self.c = c
        self.pages, self.table, self.lens = dev(c.pool.reshape(-1)), dev(c.table), dev(c.seq_len)
        self.h = q.KvCache(c.t, c.kv, c.hd, c.page, self.pages, self.table, self.lens)
        assert self.h.n_pages == c.n_pages

    def pool(self):
        return host(self.pages).reshape(self.c.pool.shape)


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


def close(got, want, tol, what):
    got = got.astype(np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off; first {np.argwhere(bad)[:3].tolist()}, "
                           f"worst {np.nanmax(np.abs(got - want) / tol):.3g} of the bound, NaN {np.isnan(got).sum()}")


def run_decode(c, n, heads, window=0, sinks=0, max_len=None, with_acc=False, seed=5, qstd=1.5, ld_extra=0, d=None):
    d = d or Dev(c)
    n_seq = len(c.seq_len)
    max_len = max_len or c.cap
    scale = c.hd ** -0.5
    width = heads * c.hd
    qh = synth.normal(seed, synth.T_X, (n_seq * n, width + ld_extra), qstd)
    qd = dev(qh)[:, ld_extra // 2:ld_extra // 2 + width] if ld_extra else dev(qh)
    qh = qh[:, ld_extra // 2:ld_extra // 2 + width].reshape(n_seq * n, heads, c.hd)
    out = torch.full((n_seq * n * heads * c.hd,), float("nan"), device="cuda")
    acc0 = np.abs(synth.normal(seed + 1, synth.T_X, (n_seq, c.kv, max_len), 1.0)) if with_acc else None
    acc = dev(acc0) if with_acc else None
    ws = workspace(q.qmv_attn_decode_workspace(d.h, n, heads, max_len, window, sinks, with_acc))
    q.qmv_attn_decode(d.h, n, heads, qd, scale, out, max_len, window=window, sinks=sinks, acc=acc, workspace=ws)
    start = np.arange(n_seq + 1) * n
    want, tol, acc1, acc_tol = ref.attention(c, start, qh, scale, max_len, window, sinks, acc0)
    what = f"decode {c.t} hd{c.hd} page{c.page} lens{list(c.seq_len)[:4]} n{n} w{window}+{sinks}"
    close(host(out).reshape(want.shape), want, tol, what)
    if with_acc:
        close(host(acc), acc1, acc_tol, what + " acc")
        t = np.arange(max_len)
        for s in range(n_seq):                      # positions that do not exist keep their bits
            keep = t >= c.length(s, max_len)
            assert np.array_equal(host(acc)[s][:, keep], acc0[s][:, keep])
    return host(out)


def run_prefill(c, news, heads, window=0, sinks=0, max_len=None, before=0, after=0, seed=7, use_start=True, qstd=1.5):
    d = Dev(c)
    max_len = max_len or c.cap
    scale = c.hd ** -0.5
    start = before + np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n = int(start[-1]) + after
    qh = synth.normal(seed, synth.T_X, (n, heads, c.hd), qstd)
    out = torch.full((n, heads, c.hd), -77.0, device="cuda")
    ws = workspace(q.qmv_attn_prefill_workspace(d.h, n, heads, max_len, window, sinks))
    q.qmv_attn_prefill(d.h, n, heads, dev(qh), scale, out, max_len, start=dev(start) if use_start else None,
                       window=window, sinks=sinks, workspace=ws)
    want, tol, _, _ = ref.attention(c, start, qh, scale, max_len, window, sinks)
    got = host(out)
    none = np.isnan(want)
    assert np.all(got[none] == -77.0), "rows of no sequence were written"
    what = f"prefill {c.t} hd{c.hd} page{c.page} lens{list(c.seq_len)[:4]} new{list(news)[:4]} w{window}+{sinks}"
    close(np.where(none, 0, got), np.where(none, 0, want), np.where(none, 1, tol), what)
    return got, ws


# ---- append -----------------------------------------------------------------

@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,kv,page", [(64, 3, 16), (96, 1, 32), (128, 2, 64), (256, 1, 16)])
def test_append(t, hd, kv, page):
    lens = [1, 0, 40, 23, 100]
    news = [1, 0, 17, 40, 3]          # the fourth has more rows than positions: its first 17 have no place
    c, rng = make_cache(t, kv, hd, page, lens, 11)
    if page < 64:
        c.table[4, 98 // page] = -1   # the fifth's last rows but one fall into a hole
    d = Dev(c)
    before, after = 2, 5
    start = (before + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + after
    w = kv * hd
    k = rng.standard_normal((n, w + 8), dtype=np.float32) * 3
    v = rng.standard_normal((n, 2 * w), dtype=np.float32)
    k[before, :w] = 0                 # a zero row
    kd, vd = dev(k)[:, :w], dev(v)[:, w:]
    q.qmv_kv_append(d.h, n, kd, vd, start=dev(start))
    c.append(start, np.ascontiguousarray(k[:, :w]).reshape(n, kv, hd), np.ascontiguousarray(v[:, w:]).reshape(n, kv, hd))
    assert np.array_equal(d.pool(), c.pool)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_append_even_rows(t):
    """start = None: n / n_seq rows each; positions that wrap from page to page."""
    kv, hd, page, lens, m = 2, 64, 16, [64, 33, 16, 200], 15
    c, rng = make_cache(t, kv, hd, page, lens, 12)
    d = Dev(c)
    n = m * len(lens)
    k, v = (rng.standard_normal((n, kv, hd), dtype=np.float32) for _ in range(2))
    q.qmv_kv_append(d.h, n, dev(k), dev(v))
    c.append(np.arange(len(lens) + 1) * m, k, v)
    assert np.array_equal(d.pool(), c.pool)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,kv,page", [(64, 8, 64), (96, 9, 16), (128, 8, 32)])
def test_append_many_rows(t, hd, kv, page):
    """Long prompts: runs of 8 positions, cut by the sequences' and the workgroups' borders."""
    lens = [2000, 5, 1203, 64, 1000]
    news = [1997, 1, 1203, 0, 997]
    c, rng = make_cache(t, kv, hd, page, lens, 13)
    c.table[2, 300 // page] = -1
    d = Dev(c)
    start = (1 + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + 2
    k, v = (rng.standard_normal((n, kv, hd), dtype=np.float32) for _ in range(2))
    q.qmv_kv_append(d.h, n, dev(k), dev(v), start=dev(start))
    c.append(start, k, v)
    assert np.array_equal(d.pool(), c.pool)


# ---- decode -----------------------------------------------------------------

@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,heads,kv,page", [(64, 9, 3, 16), (96, 4, 2, 32), (128, 8, 2, 64), (256, 5, 1, 16),
                                              (64, 17, 1, 128), (128, 2, 2, 16), (96, 20, 1, 64), (128, 18, 1, 32)])
def test_decode_lengths(t, hd, heads, kv, page):
    """From an empty sequence to several chunks, ends inside pages and chunks."""
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 257]
    c, _ = make_cache(t, kv, hd, page, lens, 21)
    run_decode(c, 1, heads)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("n,heads,kv,hd", [(2, 4, 2, 64), (5, 6, 2, 128), (8, 8, 2, 64), (16, 3, 1, 96), (16, 8, 1, 256),
                                           (3, 32, 1, 64), (8, 8, 1, 128), (1, 4, 1, 128), (1, 2, 1, 256), (2, 3, 1, 96)])
def test_decode_several_tokens(t, n, heads, kv, hd):
    """n > 1, some sequences shorter than n: tokens without a position give zeros."""
    c, _ = make_cache(t, kv, hd, 32, [0, 1, n - 1, n, 40, 129, 300], 22)
    run_decode(c, n, heads, with_acc=True, ld_extra=12)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (100, 70), (5000, 3), (64, 1000)])
@pytest.mark.parametrize("n", [1, 7])
def test_decode_window(t, window, sinks, n):
    c, _ = make_cache(t, 2, 64, 16, [1, 20, 150, 333, 600], 23)
    run_decode(c, n, 6, window=window, sinks=sinks, with_acc=n == 7)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_decode_split(t, window, sinks):
    """One long sequence: many pieces and their join; max_len beyond the length."""
    c, _ = make_cache(t, 2, 128, 64, [5003], 24, cap_pages=100)
    if window == 0:                   # a window may leave too little to split
        assert q.qmv_attn_decode_workspace(Dev(c).h, 1, 8, c.cap) > 0
    run_decode(c, 1, 8, window=window, sinks=sinks)
    run_decode(c, 4, 8, window=window, sinks=sinks, with_acc=True)


RAGGED = [2700, 0, 1, 64, 700, 31, 5200, 0, 0, 33] + [(37 * i) % 90 for i in range(30)]


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,heads,n,window,sinks", [(64, 16, 1, 0, 0), (64, 16, 5, 5000, 9), (64, 16, 16, 0, 0),
                                                     (96, 8, 1, 5100, 0), (128, 8, 3, 0, 0), (64, 64, 11, 4900, 70)])
def test_decode_ragged(t, hd, heads, n, window, sinks):
    """Long sequences among short and empty ones: workgroups that take parts of
    several sequences, tiles that see different chunks."""
    c, _ = make_cache(t, 8, hd, 64, RAGGED, 71)
    run_decode(c, n, heads, window=window, sinks=sinks, with_acc=n in (3, 5))


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,n,window,sinks", [(64, 11, 5000, 70), (64, 9, 0, 0), (128, 16, 5100, 3), (256, 5, 5000, 40)])
def test_decode_ragged_tiles(t, hd, n, window, sinks):
    """Several row tiles, whose rows see different chunks, of two key-value heads."""
    c, _ = make_cache(t, 2, hd, 64, RAGGED, 75)
    run_decode(c, n, 2 * (48 // n), window=window, sinks=sinks, with_acc=n == 9)


@pytest.mark.parametrize("t", ["f16", "i8"])
def test_decode_ragged_256_columns(t):
    c, _ = make_cache(t, 8, 256, 64, RAGGED, 72)
    run_decode(c, 2, 16, with_acc=True)


@pytest.mark.parametrize("t", ["bf16", "i8"])
@pytest.mark.parametrize("n", [1, 16])
def test_decode_hundreds_ragged(t, n):
    """More sequences than a wave has at a time, the long ones behind them; one key-value head."""
    lens = [(61 * i) % 120 for i in range(600)]
    lens[5], lens[257], lens[300], lens[599] = 1900, 0, 1300, 1700
    c, _ = make_cache(t, 1, 64, 16, lens, 73)
    run_decode(c, n, 3, with_acc=n == 1)
    c.seq_len[:] = np.minimum(c.seq_len, 3)     # far fewer chunks than workgroups
    run_decode(c, n, 3)


@pytest.mark.parametrize("t,longest", [("f16", 90000), ("i8", 170000)])
def test_decode_one_sequence_takes_all(t, longest):
    """One key-value head: every workgroup of the launch is the long sequence's."""
    c, _ = make_cache(t, 1, 64, 256, [longest, 10, 0], 76)
    run_decode(c, 1, 2)


def test_decode_ragged_follows_lengths():
    """The same call captured once: each replay cuts by the lengths it finds."""
    c, rng = make_cache("f16", 8, 64, 64, RAGGED, 74)
    d = Dev(c)
    x = dev(synth.normal(2, synth.T_X, (len(RAGGED), 16 * 64)))
    out = torch.zeros(len(RAGGED), 16 * 64, device="cuda")
    ws = workspace(q.qmv_attn_decode_workspace(d.h, 1, 16, c.cap))

    def fn():
        q.qmv_attn_decode(d.h, 1, 16, x, 0.125, out, c.cap, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    full = np.array(RAGGED, np.int32)
    for rep in range(4):
        lens = np.minimum(full, [5200, 40, 2600, 0][rep]).astype(np.int32)
        d.lens.copy_(dev(lens))
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        got = host(out).copy()
        ws.fill_(0xFF)
        out.fill_(7)
        fn()
        torch.cuda.synchronize()
        assert np.array_equal(got, host(out)), rep
        c.seq_len[:] = lens
        want, tol, _, _ = ref.attention(c, np.arange(len(RAGGED) + 1), host(x).reshape(-1, 16, 64), 0.125, c.cap)
        close(got.reshape(want.shape), want, tol, f"replay {rep}")


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_decode_holes(t):
    """Positions in holes are not seen: released pages of a window, a row whose
    every page is a hole."""
    c, _ = make_cache(t, 1, 64, 16, [300, 300, 40], 25)
    c.table[0, 2:14] = -1
    c.table[1, 5] = c.n_pages
    c.table[1, 18] = 2 ** 31 - 1
    c.table[2, :] = -5
    run_decode(c, 1, 4, with_acc=True)
    run_decode(c, 3, 4, window=70, sinks=20)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_decode_large_logits(t):
    """Logits that grow along the sequence: the running maximum moves often."""
    c, _ = make_cache(t, 1, 64, 64, [700, 64], 26)
    run_decode(c, 2, 4, qstd=40.0, with_acc=True)


@pytest.mark.parametrize("t", ["f16", "i8"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e9, 1e30])
def test_decode_query_range(t, size):
    """Queries far outside f16's range (the f16 pieces are taken of scaled rows)."""
    c, _ = make_cache(t, 1, 64, 64, [90], 27)
    d = Dev(c)
    qh = synth.normal(3, synth.T_X, (1, 4, 64), 1.0) * np.float32(size)
    out = torch.empty(4 * 64, device="cuda")
    scale = 0.2 / size
    q.qmv_attn_decode(d.h, 1, 4, dev(qh.reshape(1, -1)), scale, out, 128)
    want, tol, _, _ = ref.attention(c, [0, 1], qh, float(np.float32(scale)), 128)
    close(host(out).reshape(want.shape), want, tol, f"query size {size}")


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-38])
def test_scale_sign(t, scale):
    """Any scale: negative, none, vanishing; in both calls."""
    c, _ = make_cache(t, 1, 64, 16, [70], 30)
    d = Dev(c)
    qh = synth.normal(3, synth.T_X, (20, 2, 64), 1.0)
    want, tol, _, _ = ref.attention(c, [0, 20], qh, float(np.float32(scale)), 80)
    out = torch.empty(20, 128, device="cuda")
    q.qmv_attn_prefill(d.h, 20, 2, dev(qh.reshape(20, -1)), scale, out, 80)
    close(host(out).reshape(want.shape), want, tol, f"prefill scale {scale}")
    out = torch.empty(16, 128, device="cuda")
    q.qmv_attn_decode(d.h, 16, 2, dev(qh[4:].reshape(16, -1)), scale, out, 80)
    close(host(out).reshape(16, 2, 64), want[4:], tol[4:], f"decode scale {scale}")


@pytest.mark.parametrize("size", [1e-20, 1e-7, 3e4, 1e20])
def test_decode_i8_value_range(size):
    """8-bit V rows of any scale, and of very different scales in one sequence."""
    c, rng = make_cache("i8", 1, 64, 16, [150], 28)
    for p in range(150):
        pg, slot = c.where(0, p)
        c.parts(pg, 0)[2][1, slot] *= np.float32(size * 10.0 ** (p % 5 - 4))
    run_decode(c, 1, 4)


def test_decode_far_pages():
    """Pages beyond 4 GiB of the pool."""
    t, kv, hd, page = "f16", 2, 128, 64
    c, _ = make_cache(t, kv, hd, page, [500], 29)
    pb = q.qmv_kv_page_bytes(t, kv, hd, page)
    n_pages = (9 << 30) // (2 * pb)                 # 4.5 GiB
    pool = torch.zeros(n_pages * pb, dtype=torch.uint8, device="cuda")
    far = np.array([[n_pages - 1 - 3 * i for i in range(c.table.shape[1])]], np.int32)
    view = pool.view(n_pages, pb)
    for i, pg in enumerate(c.table[0]):
        view[int(far[0, i])] = dev(c.pool[pg].reshape(-1))
    cache = q.KvCache(t, kv, hd, page, pool, dev(far), dev(c.seq_len))
    qh = synth.normal(4, synth.T_X, (20, 8, hd), 1.0)
    want, tol, _, _ = ref.attention(c, [0, 1], qh[:1], hd ** -0.5, 512)
    out = torch.empty(20, 8, hd, device="cuda")
    q.qmv_attn_decode(cache, 1, 8, dev(qh[:1].reshape(1, -1)), hd ** -0.5, out[:1], 512,
                      workspace=workspace(q.qmv_attn_decode_workspace(cache, 1, 8, 512)))
    close(host(out[:1]), want, tol, "far pages, decode")
    want, tol, _, _ = ref.attention(c, [0, 20], qh, hd ** -0.5, 512)
    q.qmv_attn_prefill(cache, 20, 8, dev(qh.reshape(20, -1)), hd ** -0.5, out, 512,
                       workspace=workspace(q.qmv_attn_prefill_workspace(cache, 20, 8, 512)))
    close(host(out), want, tol, "far pages, prefill")
    k, v = (synth.normal(i, synth.T_X, (3, kv, hd)) for i in (5, 6))
    q.qmv_kv_append(cache, 3, dev(k), dev(v))
    c.append([0, 3], k, v)
    for i, pg in enumerate(c.table[0]):
        assert np.array_equal(host(view[int(far[0, i])]), c.pool[pg].reshape(-1))


# ---- prefill ----------------------------------------------------------------

@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,heads,kv,page", [(64, 9, 3, 16), (96, 4, 2, 32), (128, 8, 2, 64), (256, 5, 1, 16),
                                              (64, 17, 1, 128)])
def test_prefill_ragged(t, hd, heads, kv, page):
    """Whole prompts and later parts, empty sequences, rows of no sequence."""
    lens = [0, 1, 33, 64, 130, 200]
    news = [0, 1, 33, 20, 130, 97]
    c, _ = make_cache(t, kv, hd, page, lens, 31)
    run_prefill(c, news, heads, before=3, after=4)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("n,length", [(1, 1), (16, 16), (17, 40), (150, 150), (64, 300)])
def test_prefill_even(t, n, length):
    c, _ = make_cache(t, 2, 64, 32, [length, max(0, length - 9), length], 32)
    run_prefill(c, [n] * 3, 6, use_start=False)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (17, 4), (64, 0), (100, 70), (250, 1000)])
def test_prefill_window(t, window, sinks):
    c, _ = make_cache(t, 1, 64, 16, [400, 90, 300], 33)
    run_prefill(c, [400, 90, 40], 4, window=window, sinks=sinks)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 5)])
def test_prefill_split(t, hd, window, sinks):
    """Few new rows after a long context: pieces and their join."""
    c, _ = make_cache(t, 1, hd, 64, [3000, 2100], 34)
    _, ws = run_prefill(c, [40, 19], 3, window=window, sinks=sinks, before=1, after=2)
    assert ws is not None or window > 0


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_prefill_holes_and_large_logits(t):
    c, _ = make_cache(t, 1, 64, 16, [300, 40], 35)
    c.table[0, 2:14] = -1
    c.table[0, 17] = c.n_pages
    c.table[1, :] = -5
    run_prefill(c, [60, 40], 4)
    run_prefill(c, [60, 40], 4, window=90, sinks=20, qstd=40.0)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 3)])
def test_hidden_values_do_not_matter(t, hd, window, sinks):
    """NaN and infinities in K or V of existing positions: rows that do not see
    the position are as without them, rows that do are not finite (V: in that
    column, or for the 8-bit scales in all)."""
    n, length, heads, page = 16, 333, 4, 16
    spots = [(332, "v", np.nan, 5), (330, "v", np.inf, 7), (325, "k", np.nan, 3), (299, "v", -np.inf, 0),
             (290, "k", np.inf, 9), (1, "v", np.nan, 11), (length - 60, "v", np.nan, 2)]
    base, _ = make_cache(t, 1, hd, page, [length], 37)
    scale = hd ** -0.5
    qh = synth.normal(8, synth.T_X, (n + 44, heads, hd), 1.0)
    for what, m in (("decode", 1), ("decode", n), ("prefill", n + 44)):
        q0 = qh[-m:]
        clean, tol, _, _ = ref.attention(base, [0, m], q0, scale, base.cap, window, sinks)
        for p, part, bad, col in spots:
            c = ref.Cache(t, 1, hd, page, base.n_pages, base.table, base.seq_len)
            c.pool = base.pool.copy()
            pg, slot = c.where(0, p)
            k, v, sc = c.parts(pg, 0)
            if t == "i8":
                sc[0 if part == "k" else 1, slot] = bad
            else:
                code = np.float16(bad) if t == "f16" else ref.round_bf16(np.float32(bad) if np.isinf(bad) else 0)
                if t == "bf16" and np.isnan(bad):
                    code = np.uint16(0x7FC0)
                if part == "k":
                    k[slot, col] = code
                else:
                    v[slot // 16, col, slot % 16] = code
            d = Dev(c)
            out = torch.empty(m * heads * hd, device="cuda")
            if what == "decode":
                ws = workspace(q.qmv_attn_decode_workspace(d.h, m, heads, c.cap, window, sinks))
                q.qmv_attn_decode(d.h, m, heads, dev(q0.reshape(m, -1)), scale, out, c.cap, window=window, sinks=sinks,
                                  workspace=ws)
            else:
                ws = workspace(q.qmv_attn_prefill_workspace(d.h, m, heads, c.cap, window, sinks))
                q.qmv_attn_prefill(d.h, m, heads, dev(q0.reshape(m, -1)), scale, out, c.cap, window=window, sinks=sinks,
                                   workspace=ws)
            got = host(out).reshape(m, heads, hd)
            pos = length - m + np.arange(m)
            sees = p <= pos
            if window:
                sees &= (p > pos - window) | (p < sinks)
            name = f"{what} {t} m{m} {part}[{p}]={bad}"
            close(got[~sees], clean[~sees], tol[~sees], name)
            if not sees.any():
                continue
            if part == "v" and t != "i8":
                assert not np.isfinite(got[sees][:, :, col]).any(), name
                other = np.arange(hd) != col
                close(got[sees][:, :, other], clean[sees][:, :, other], tol[sees][:, :, other], name)
            elif part == "v" or np.isnan(bad):
                assert not np.isfinite(got[sees]).any(), name


def test_prefill_matches_decode():
    """Both calls compute the same rows (n <= 16), each within its bound."""
    c, _ = make_cache("f16", 2, 128, 64, [700, 16, 31], 36)
    a = run_decode(c, 16, 8, seed=9).reshape(48, 8, 128)
    b, _ = run_prefill(c, [16] * 3, 8, seed=9, use_start=False)
    assert np.max(np.abs(a - b)) < 1e-4


# ---- eviction ----------------------------------------------------------------

def run_evict(c, keep, first, recent, acc, dst=None):
    n_seq = len(c.seq_len)
    per = -(-keep // c.page)
    if dst is None:
        dst = np.arange(c.n_pages - n_seq * per, c.n_pages, dtype=np.int32)[::-1].reshape(n_seq, per)
    d = Dev(c)
    kept = torch.full((n_seq, c.kv, keep), -9, dtype=torch.int32, device="cuda")
    out = torch.full((n_seq, c.kv, keep + 5), -9.0, device="cuda")
    lens = torch.full((n_seq,), -9, dtype=torch.int32, device="cuda")
    q.qmv_kv_evict(d.h, dev(dst), keep, first, recent, dev(acc), kept, out, lens)
    k, a, n = ref.evict(c, dst, keep, first, recent, acc)
    assert np.array_equal(host(kept), k)
    assert np.array_equal(host(out)[..., :keep].view(np.uint32), a.view(np.uint32))
    assert np.all(host(out)[..., keep:] == -9.0)
    assert np.array_equal(host(lens), n)
    assert np.array_equal(d.pool(), c.pool)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("hd,kv,page", [(64, 3, 16), (96, 1, 32), (128, 2, 64), (256, 1, 16)])
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (33, 4, 20), (64, 0, 64), (100, 4, 17), (100, 100, 0)])
def test_evict(t, hd, kv, page, keep, first, recent):
    lens = [0, 1, 63, 100, 101, 300]
    c, rng = make_cache(t, kv, hd, page, lens, 41, spare=len(lens) * -(-keep // page))
    run_evict(c, keep, first, recent, rng.random((len(lens), kv, 310), dtype=np.float32) ** 2)


@pytest.mark.parametrize("case", ["equal", "two", "signs", "special", "tiny"])
def test_evict_scores(case):
    """Equal scores, few distinct ones, negative ones and zeros of both signs,
    infinities and NaN, differences in the last bit."""
    n, kv = 2500, 2
    c, rng = make_cache("f16", kv, 64, 64, [n], 42, spare=20)
    x = {"equal": np.ones((1, kv, n)), "two": rng.integers(0, 2, (1, kv, n)),
         "signs": rng.integers(-2, 3, (1, kv, n)) * rng.choice([1.0, 0.0, -0.0], (1, kv, n)),
         "special": rng.choice([np.inf, -np.inf, np.nan, 0.5, 1e-40], (1, kv, n)),
         "tiny": np.float32(1) + rng.integers(0, 40, (1, kv, n)).astype(np.float32) * np.float32(2.0 ** -23)}[case]
    run_evict(c, 1203, 4, 100, x.astype(np.float32))


@pytest.mark.parametrize("n,keep", [(8192, 8000), (8193, 300), (20011, 15000)])
def test_evict_long(n, keep):
    """More positions than a workgroup ranks at a time."""
    c, rng = make_cache("bf16", 1, 64, 64, [n, 100], 44, spare=2 * -(-keep // 64))
    x = np.round(rng.random((2, 1, n + 3), dtype=np.float32) * 500)      # many equal scores
    run_evict(c, keep, 4, 128, x)


def test_evict_holes():
    """A destination hole drops its rows, a source hole gives zeros."""
    c, rng = make_cache("i8", 2, 64, 16, [200, 90], 43, spare=20)
    c.table[0, 3] = -1
    c.table[1, 0] = c.n_pages + 7
    per = 5
    dst = np.arange(c.n_pages - 2 * per, c.n_pages, dtype=np.int32).reshape(2, per)
    dst[0, 2] = -1
    dst[1, 4] = c.n_pages
    run_evict(c, 70, 4, 10, rng.random((2, 2, 200), dtype=np.float32), dst)


@pytest.mark.parametrize("t", ["f16", "i8"])
def test_evict_lengths_in_place(t):
    """len_out may be the cache's own seq_len: every head still cuts from the old length."""
    keep, lens = 100, [1500, 0, 99, 100, 101, 1030]
    c, rng = make_cache(t, 16, 64, 16, lens, 45, spare=len(lens) * -(-keep // 16))
    per = -(-keep // 16)
    dst = np.arange(c.n_pages - len(lens) * per, c.n_pages, dtype=np.int32).reshape(len(lens), per)
    acc = rng.random((len(lens), 16, 1500), dtype=np.float32)
    d = Dev(c)
    kept = torch.full((len(lens), 16, keep), -9, dtype=torch.int32, device="cuda")
    out = torch.full((len(lens), 16, keep), -9.0, device="cuda")
    q.qmv_kv_evict(d.h, dev(dst), keep, 4, 20, dev(acc), kept, out, d.lens)
    k, a, n = ref.evict(c, dst, keep, 4, 20, acc)
    assert np.array_equal(host(kept), k)
    assert np.array_equal(host(out).view(np.uint32), a.view(np.uint32))
    assert np.array_equal(host(d.lens), n)
    assert np.array_equal(d.pool(), c.pool)


# ---- together -----------------------------------------------------------------

@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_prompt_decode_evict_decode(t):
    """As a program uses them: prompts appended and attended, tokens decoded one
    by one with their weights collected, drafted tokens checked, the cache cut,
    decoding again from the cut cache."""
    kv, heads, hd, page, prompts = 2, 6, 64, 16, [50, 7, 33]
    n_seq, per, keep = 3, 8, 40
    rng = synth.rng(51, synth.T_X)
    n_pages = 2 * n_seq * per
    ids = rng.permutation(n_pages).astype(np.int32)
    c = ref.Cache(t, kv, hd, page, n_pages, ids[:n_seq * per].reshape(n_seq, per), prompts, fill=0xFF)
    d = Dev(c)
    acc_ref = np.zeros((n_seq, kv, c.cap), np.float32)
    acc = dev(acc_ref)
    scale, max_len = hd ** -0.5, c.cap
    ws = workspace(max(q.qmv_attn_decode_workspace(d.h, n, heads, max_len, 0, 0, True) for n in (1, 4)))

    def qkv(n):
        x = rng.standard_normal((n, (heads + 2 * kv) * hd), dtype=np.float32)
        xd = dev(x)
        a, b = heads * hd, (heads + kv) * hd
        return (x[:, :a].reshape(n, heads, hd), x[:, a:b].reshape(n, kv, hd), x[:, b:].reshape(n, kv, hd),
                xd[:, :a], xd[:, a:b], xd[:, b:])

    # prompts
    start = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    n = int(start[-1])
    qh, kh, vh, qd, kd, vd = qkv(n)
    sd = dev(start)
    q.qmv_kv_append(d.h, n, kd, vd, start=sd)
    c.append(start, kh, vh)
    out = torch.empty(n, heads * hd, device="cuda")
    assert q.qmv_attn_prefill_workspace(d.h, n, heads, max_len) == 0
    q.qmv_attn_prefill(d.h, n, heads, qd, scale, out, max_len, start=sd)
    want, tol, _, _ = ref.attention(c, start, qh, scale, max_len)
    close(host(out).reshape(want.shape), want, tol, "prompt")

    def step(n, what):
        nonlocal acc_ref
        c.seq_len += n
        d.lens.add_(n)
        rows = n_seq * n
        qh, kh, vh, qd, kd, vd = qkv(rows)
        q.qmv_kv_append(d.h, rows, kd, vd)
        st = np.arange(n_seq + 1) * n
        c.append(st, kh, vh)
        out = torch.empty(rows, heads * hd, device="cuda")
        q.qmv_attn_decode(d.h, n, heads, qd, scale, out, max_len, acc=acc, workspace=ws)
        want, tol, a1, at = ref.attention(c, st, qh, scale, max_len, acc=acc_ref)
        close(host(out).reshape(want.shape), want, tol, what)
        close(host(acc), a1, at, what + " acc")
        acc_ref = host(acc).copy()

    for i in range(5):
        step(1, f"step {i}")
    step(4, "draft")
    assert np.array_equal(d.pool(), c.pool)

    # cut to `keep` positions and go on
    dst = np.full((n_seq, per), -1, np.int32)
    dst[:] = ids[n_seq * per:].reshape(n_seq, per)
    kept = torch.empty(n_seq, kv, keep, dtype=torch.int32, device="cuda")
    acc2 = torch.zeros(n_seq, kv, max_len, device="cuda")
    lens2 = torch.empty(n_seq, dtype=torch.int32, device="cuda")
    q.qmv_kv_evict(d.h, dev(dst), keep, 4, 16, acc, kept, acc2, lens2)
    k, a, n2 = ref.evict(c, dst, keep, 4, 16, acc_ref)
    assert np.array_equal(host(kept), k) and np.array_equal(host(lens2), n2)
    d.table.copy_(dev(dst))
    d.lens.copy_(lens2)
    acc.copy_(acc2)
    c.table, c.seq_len = dst, n2
    acc_ref = np.zeros_like(acc_ref)
    acc_ref[..., :keep] = a
    for i in range(3):
        step(1, f"step {i} after the cut")
    assert np.array_equal(d.pool(), c.pool)


@pytest.mark.parametrize("window", [0, 90])
def test_graph_replay_follows_lengths(window):
    """Append and decode captured once; every replay follows the lengths and the
    inputs in place, with eager work between replays, and equals the eager call
    bit for bit."""
    kv, heads, hd, page = 2, 8, 128, 64
    c, rng = make_cache("f16", kv, hd, page, [900, 130], 61, cap_pages=20)
    d = Dev(c)
    max_len = c.cap
    acc = torch.zeros(2, kv, max_len, device="cuda")
    qd, kd, vd = (torch.zeros(2, w, device="cuda") for w in (heads * hd, kv * hd, kv * hd))
    out = torch.empty(2, heads * hd, device="cuda")
    ws = workspace(q.qmv_attn_decode_workspace(d.h, 1, heads, max_len, window, 4, True))

    def fn():
        q.qmv_kv_append(d.h, 2, kd, vd)
        q.qmv_attn_decode(d.h, 1, heads, qd, hd ** -0.5, out, max_len, window=window, sinks=4, acc=acc, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    for rep in range(4):
        for x, w in ((qd, 1.5), (kd, 1.0), (vd, 1.0)):
            x.copy_(dev(rng.standard_normal(x.shape, dtype=np.float32) * np.float32(w)))
        d.lens.add_(1)
        acc.zero_()
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got, got_acc, pool = host(out).copy(), host(acc).copy(), d.pool().copy()
        acc.zero_()
        fn()                                         # the same again, eagerly
        torch.cuda.synchronize()
        assert np.array_equal(got, host(out)) and np.array_equal(got_acc, host(acc)), rep
        assert np.array_equal(pool, d.pool())
        assert np.isfinite(got).all()


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
def test_lengths_out_of_range(t):
    """Lengths below 0, past max_len and past what a table row addresses are cut to the range."""
    # (304: all that a table row addresses holds finite values)
    c, rng = make_cache(t, 2, 64, 16, [304, 304, 304, 304, 40], 64)
    c.seq_len = np.array([300, -3, 10 ** 9, 2 ** 31 - 1, -2 ** 31], np.int32)
    run_decode(c, 2, 4, with_acc=True)
    run_decode(c, 2, 4, max_len=200, window=64, sinks=2)
    run_prefill(c, [20, 3, 200, 0, 5], 4)
    run_prefill(c, [20, 3, 200, 0, 5], 4, max_len=100)
    k, v = (rng.standard_normal((10, 2, 64), dtype=np.float32) for _ in range(2))
    d = Dev(c)
    q.qmv_kv_append(d.h, 10, dev(k), dev(v))
    c.append(np.arange(6) * 2, k, v)
    assert np.array_equal(d.pool(), c.pool)
    c2, rng = make_cache(t, 2, 64, 16, [300, 300, 300], 65, spare=30)
    c2.seq_len = np.array([10 ** 9, -1, 299], np.int32)
    run_evict(c2, 150, 3, 10, rng.random((3, 2, 280), dtype=np.float32))      # scores for 280 positions only


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("page", [256, 4096])
def test_large_pages(t, page):
    lens = [700, 5, 256]
    c, rng = make_cache(t, 2, 64, page, lens, 66, spare=12)
    run_decode(c, 1, 4, with_acc=True)
    run_prefill(c, [100, 5, 256], 4, window=70, sinks=3)
    k, v = (rng.standard_normal((9, 2, 64), dtype=np.float32) for _ in range(2))
    d = Dev(c)
    q.qmv_kv_append(d.h, 9, dev(k), dev(v))
    c.append(np.arange(4) * 3, k, v)
    assert np.array_equal(d.pool(), c.pool)
    run_evict(c, 300, 4, 60, rng.random((3, 2, 700), dtype=np.float32))


@pytest.mark.parametrize("t", ["f16", "i8"])
def test_many_sequences(t):
    """More sequences than a wave has lanes, many of them without new rows."""
    n = 300
    lens = [(7 * i) % 41 for i in range(n)]
    news = [0 if i % 3 else min(lens[i], (5 * i) % 23) for i in range(n)]
    c, _ = make_cache(t, 1, 64, 16, lens, 67)
    run_prefill(c, news, 2, before=2, after=1)
    run_decode(c, 1, 2)


def test_outputs_at_any_float():
    """q, out and acc may start at any float of a tensor."""
    c, _ = make_cache("f16", 1, 64, 16, [90, 41], 68)
    d = Dev(c)
    qh = synth.normal(2, synth.T_X, (2, 3 * 64 + 1), 1.0)
    qd = dev(qh)[:, 1:]
    for off in (1, 3):
        buf = torch.full((2 * 3 * 64 + 8,), -5.0, device="cuda")
        out = buf[off:off + 2 * 3 * 64]
        q.qmv_attn_decode(d.h, 1, 3, qd, 0.125, out, 96)
        want, tol, _, _ = ref.attention(c, [0, 1, 2], np.ascontiguousarray(qh[:, 1:]).reshape(2, 3, 64), 0.125, 96)
        close(host(out).reshape(want.shape), want, tol, f"decode, out + {off}")
        out.fill_(-5.0)
        q.qmv_attn_prefill(d.h, 2, 3, qd, 0.125, out, 96)
        close(host(out).reshape(want.shape), want, tol, f"prefill, out + {off}")
        assert torch.all(buf[:off] == -5.0) and torch.all(buf[off + 2 * 3 * 64:] == -5.0)


@pytest.mark.parametrize("exp", [-20, -22, 3])
def test_f16_values_near_the_ends(exp):
    """Cached f16 values among the subnormals keep their relative precision."""
    c, _ = make_cache("f16", 1, 64, 16, [150], 69)
    for p in range(c.n_pages):
        k, v, _ = c.parts(p, 0)
        with np.errstate(all="ignore"):
            k[:] = (k.astype(np.float32) * np.float32(2.0 ** exp)).astype(np.float16)
            v[:] = (v.astype(np.float32) * np.float32(2.0 ** exp)).astype(np.float16)
    d = Dev(c)
    qh = synth.normal(2, synth.T_X, (1, 2, 64), 1.0)
    scale = float(np.float32(0.2 * 2.0 ** -exp))
    want, tol, _, _ = ref.attention(c, [0, 1], qh, scale, 150)
    out = torch.empty(128, device="cuda")
    q.qmv_attn_decode(d.h, 1, 2, dev(qh.reshape(1, -1)), scale, out, 150)
    close(host(out).reshape(want.shape), want, tol, f"decode 2^{exp}")
    q.qmv_attn_prefill(d.h, 1, 2, dev(qh.reshape(1, -1)), scale, out, 150)
    close(host(out).reshape(want.shape), want, tol, f"prefill 2^{exp}")


def test_graph_replay_prefill_and_evict():
    """A split prompt call and an eviction captured once; each replay, with new
    inputs in place and eager work between, equals the eager calls bit for bit."""
    kv, heads, hd, page, keep = 1, 4, 128, 64, 700
    c, rng = make_cache("bf16", kv, hd, page, [3000, 900], 70, spare=2 * -(-keep // 64))
    d = Dev(c)
    start = dev(np.array([0, 30, 41], np.int32))
    qd, out = torch.zeros(41, heads * hd, device="cuda"), torch.zeros(41, heads * hd, device="cuda")
    ws = workspace(q.qmv_attn_prefill_workspace(d.h, 41, heads, c.cap))
    assert ws is not None
    per = -(-keep // page)
    dst = dev(np.arange(c.n_pages - 2 * per, c.n_pages, dtype=np.int32).reshape(2, per))
    acc = torch.zeros(2, kv, 3000, device="cuda")
    kept = torch.zeros(2, kv, keep, dtype=torch.int32, device="cuda")
    acc_out, len_out = torch.zeros(2, kv, keep, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")

    def fn():
        q.qmv_attn_prefill(d.h, 41, heads, qd, hd ** -0.5, out, c.cap, start=start, workspace=ws)
        q.qmv_kv_evict(d.h, dst, keep, 4, 64, acc, kept, acc_out, len_out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    outs = (out, kept, acc_out, len_out, d.pages)
    for rep in range(4):
        qd.copy_(dev(rng.standard_normal(qd.shape, dtype=np.float32)))
        acc.copy_(dev(rng.random(acc.shape, dtype=np.float32)))
        for x in outs[:4]:
            x.fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        got = [host(x).copy() for x in outs]
        for x in outs[:4]:
            x.fill_(-3)
        fn()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert np.array_equal(a, host(b)), rep


def test_other_stream():
    """On a stream of its own, ordered by the caller; two streams at once with a
    workspace each."""
    c, _ = make_cache("f16", 2, 64, 64, [2000], 62)
    d = Dev(c)
    qd = dev(synth.normal(1, synth.T_X, (1, 8 * 64)))
    need = q.qmv_attn_decode_workspace(d.h, 1, 8, c.cap)
    base = torch.empty(1, 8 * 64, device="cuda")
    q.qmv_attn_decode(d.h, 1, 8, qd, 0.125, base, c.cap, workspace=workspace(need))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(1, 8 * 64, device="cuda") for _ in streams]
    wss = [workspace(need) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, outs, wss):
            q.qmv_attn_decode(d.h, 1, 8, qd, 0.125, o, c.cap, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, base)


def test_results_repeat():
    """The same call twice gives the same bits (no order-dependent sums)."""
    c, _ = make_cache("bf16", 2, 64, 32, [3000, 411], 63)
    a = run_decode(c, 5, 8, with_acc=True)
    assert np.array_equal(a, run_decode(c, 5, 8, with_acc=True))


def test_tensors_of_the_host_are_refused():
    """A kernel cannot tell a host address: the binding refuses it before the launch."""
    c, _ = make_cache("f16", 1, 64, 16, [40], 64)
    d = Dev(c)
    x, out = torch.zeros(1, 128, device="cuda"), torch.zeros(1, 128, device="cuda")
    with pytest.raises(ValueError):
        q.KvCache("f16", 1, 64, 16, d.pages, d.table.cpu(), d.lens)
    with pytest.raises(ValueError):
        q.KvCache("f16", 1, 64, 16, d.pages, d.table, d.lens.cpu())
    with pytest.raises(ValueError):
        q.qmv_kv_append(d.h, 1, x[:, :64], x[:, 64:].cpu())
    with pytest.raises(ValueError):
        q.qmv_attn_decode(d.h, 1, 2, x.cpu(), 0.125, out, 64)
    with pytest.raises(ValueError):
        q.qmv_attn_prefill(d.h, 1, 2, x, 0.125, out.cpu(), 64)
    torch.cuda.synchronize()
    assert not host(out).any()


# ---- ends of the ranges ----------------------------------------------------------

def _one_cache(t, hd, page, length, kv=1, seed=80, extra=0):
    """A cache of one sequence and its rows, to be filled by the test."""
    c, rng = make_cache(t, kv, hd, page, [length], seed, cap_pages=-(-(length + extra) // page))
    return c, rng


def _both(c, qh, scale, window=0, sinks=0, n_decode=(1,), max_len=None):
    """Outputs of the last rows of qh by qmv_attn_decode, and of all by qmv_attn_prefill."""
    d = Dev(c)
    heads, max_len = qh.shape[1], max_len or c.cap
    for m in (*n_decode, 0):
        rows = qh[len(qh) - m:] if m else qh
        m0 = len(rows)
        out = torch.full((m0, heads * c.hd), -7.0, device="cuda")
        if m:
            ws = workspace(q.qmv_attn_decode_workspace(d.h, m, heads, max_len, window, sinks))
            q.qmv_attn_decode(d.h, m, heads, dev(rows.reshape(m0, -1)), scale, out, max_len, window=window, sinks=sinks,
                              workspace=ws)
        else:
            ws = workspace(q.qmv_attn_prefill_workspace(d.h, m0, heads, max_len, window, sinks))
            q.qmv_attn_prefill(d.h, m0, heads, dev(rows.reshape(m0, -1)), scale, out, max_len, window=window, sinks=sinks,
                               workspace=ws)
        yield (f"decode n{m}" if m else f"prefill {m0}"), rows, host(out).reshape(m0, heads, c.hd)


@pytest.mark.parametrize("hd,length,n", [(64, 1, 1), (64, 3, 3), (128, 300, 40), (64, 3000, 20), (256, 700, 20)])
@pytest.mark.parametrize("exp", [-100, 100, 116, 125])
def test_bf16_value_range(hd, length, n, exp):
    """bf16 values up to the type's largest: sums of weighted values stay finite."""
    c, rng = _one_cache("bf16", hd, 64, length)
    k = rng.standard_normal((length, 1, hd), dtype=np.float32)
    v = np.clip(rng.standard_normal((length, 1, hd), dtype=np.float32), -3, 3) * np.float32(2.0 ** exp)
    _fill(c, 0, k, v)
    qh = synth.normal(3, synth.T_X, (n, 4, hd), 1.5)
    scale = float(np.float32(hd ** -0.5))
    for what, rows, got in _both(c, qh, scale, n_decode=(1, min(n, 16))):
        want, tol, _, _ = ref.attention(c, [0, len(rows)], rows, scale, c.cap)
        close(got, want, tol, f"{what} 2^{exp}")


@pytest.mark.parametrize("length", [1, 70, 5000])
def test_bf16_largest_values(length):
    """Every value the largest bf16: so is the mean, to rounding."""
    c, rng = _one_cache("bf16", 64, 64, length)
    top = np.array([0x7F7F], np.uint16).view(np.uint16)
    _fill(c, 0, rng.standard_normal((length, 1, 64), dtype=np.float32), np.zeros((length, 1, 64), np.float32))
    for pg in c.table[0]:
        c.parts(pg, 0)[1][:] = top
    qh = synth.normal(3, synth.T_X, (min(length, 20), 4, 64), 1.5)
    scale = 0.125
    for what, rows, got in _both(c, qh, scale, n_decode=(1, min(length, 16))):
        want, tol, _, _ = ref.attention(c, [0, len(rows)], rows, scale, c.cap)
        close(got, want, tol, f"{what} largest")


@pytest.mark.parametrize("length,n", [(1, 1), (64, 20), (2500, 20), (20000, 20)])
@pytest.mark.parametrize("exp", [-100, 100])
@pytest.mark.parametrize("flat", [True, False])
def test_i8_scales_at_the_ends(length, n, exp, flat):
    """8-bit V row scales at both ends of what the header names, every code the
    largest; every position the same weight, or any."""
    c, rng = _one_cache("i8", 64, 64, length)
    k = rng.standard_normal((length, 1, 64), dtype=np.float32) * np.float32(not flat)
    _fill(c, 0, k, np.full((length, 1, 64), 127.0, np.float32))
    for pg in c.table[0]:
        sc = c.parts(pg, 0)[2]
        sc[1] = np.where(np.isnan(sc[1]), sc[1], np.float32(2.0 ** exp))
    qh = synth.normal(3, synth.T_X, (n, 4, 64), 1.5)
    for what, rows, got in _both(c, qh, 0.125, n_decode=(1, min(n, 16))):
        want, tol, _, _ = ref.attention(c, [0, len(rows)], rows, 0.125, c.cap)
        close(got, want, tol, f"{what} 2^{exp}")


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("size", [1e5, 1e8, 1e12, 1e30, 1e36])
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_logits(t, size, sign):
    """Logits far beyond the exponent's range, of either sign: each row takes the
    value of its largest one.

    K holds sign * (1 + i / 128) in one column, so neighbouring logits differ by
    size / 128 * log2 e, over 1000, and the other weights are zero.  The output is
    then V of one position, off by the split of its weight (2^-22) and at most 16
    roundings (2^-20): 1.25 * 2^-20 of |V|."""
    length, n = 120, 50
    c, rng = _one_cache(t, 64, 16, length)
    order = rng.permutation(128)[:length]
    k = np.zeros((length, 1, 64), np.float32)
    k[:, 0, 0] = sign * (1 + order / 128.0)
    v = rng.standard_normal((length, 1, 64), dtype=np.float32)
    _fill(c, 0, k, v)
    _, V, _ = c.rows(0, 0, length)
    qh = np.zeros((n, 2, 64), np.float32)
    qh[:, :, 0] = size
    for what, rows, got in _both(c, qh, 1.0, n_decode=(1, 16)):
        m = len(rows)
        best = [int(np.argmax(k[:length - m + j + 1, 0, 0])) for j in range(m)]
        want = V[best][:, None, :]
        close(got, np.broadcast_to(want, got.shape), np.broadcast_to(np.abs(want) * 1.25 * 2.0 ** -20 + 1e-37, got.shape),
              f"{what} {t} {sign * size}")
    # the weights: one for each row's position
    d = Dev(c)
    out, acc = torch.empty(16, 128, device="cuda"), torch.zeros(1, 1, c.cap, device="cuda")
    ws = workspace(q.qmv_attn_decode_workspace(d.h, 16, 2, c.cap, 0, 0, True))
    q.qmv_attn_decode(d.h, 16, 2, dev(qh[-16:].reshape(16, -1)), 1.0, out, c.cap, acc=acc, workspace=ws)
    want = np.zeros(c.cap)
    for j in range(16):
        want[int(np.argmax(k[:length - 16 + j + 1, 0, 0]))] += 2
    close(host(acc).reshape(-1), want, want * 2.0 ** -20 + 1e-37, f"weights {t} {sign * size}")


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("bad", [1e12, 1e25, 1e30])
@pytest.mark.parametrize("window,sinks,length,n", [(37, 3, 333, 9), (100, 0, 150, 1), (64, 5, 200, 60)])
def test_i8_hidden_scales(hd, bad, window, sinks, length, n):
    """A large finite V row scale at a position that no row of the call sees,
    before the window, behind the sinks, or behind the last position."""
    c, _ = make_cache("i8", 1, hd, 16, [length], 81, cap_pages=-(-length // 16) + 1)
    qh = synth.normal(8, synth.T_X, (n, 4, hd), 1.0)
    scale = float(np.float32(hd ** -0.5))
    first = length - n - window + 1                # the first position in some row's window
    for p in (first - 1, first - 2, first - 17, sinks, length):
        pool = c.pool.copy()
        pg, slot = c.where(0, p)
        c.parts(pg, 0)[2][1, slot] = bad
        for what, rows, got in _both(c, qh, scale, window, sinks, n_decode=(n,) if n <= 16 else ()):
            want, tol, _, _ = _without(c, pool, rows, scale, window, sinks)
            close(got, want, tol, f"{what} hd{hd} scale[{p}] = {bad}")
        c.pool[:] = pool


def _without(c, pool, rows, scale, window, sinks):
    clean = ref.Cache(c.t, c.kv, c.hd, c.page, c.n_pages, c.table, c.seq_len)
    clean.pool = pool
    return ref.attention(clean, [0, len(rows)], rows, scale, c.cap, window, sinks)


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("spot", [3, 40, 70, 119])
@pytest.mark.parametrize("top", [10, 50, 100])
@pytest.mark.parametrize("window", [0, 200])
def test_seen_values_without_weight(t, bad, spot, top, window):
    """A value that is not finite reaches every row that sees it, also where its
    weight underflows to zero."""
    length, n, hd = 120, 20, 64
    c, rng = _one_cache(t, hd, 16, length, extra=100)
    k = np.zeros((length, 1, hd), np.float32)
    k[:, 0, 0] = np.where(np.arange(length) == top, 8.0, -8.0)      # all weight on one position
    _fill(c, 0, k, rng.standard_normal((length, 1, hd), dtype=np.float32))
    pg, slot = c.where(0, spot)
    _, v, sc = c.parts(pg, 0)
    if t == "i8":
        sc[1, slot] = bad
    else:
        v[slot // 16, 5, slot % 16] = np.float16(bad) if t == "f16" else 0x7FC0 if np.isnan(bad) else 0x7F80
    qh = np.zeros((n, 2, hd), np.float32)
    qh[:, :, 0] = 100.0
    for what, rows, got in _both(c, qh, 1.0, window, 0, n_decode=(1, 16)):
        m = len(rows)
        sees = spot <= length - m + np.arange(m)
        cols = slice(None) if t == "i8" else slice(5, 6)
        assert not np.isfinite(got[sees][:, :, cols]).any(), f"{what} {t} {bad} at {spot}, weight at {top}"
        assert np.isfinite(got[~sees]).all(), f"{what} {t} {bad} at {spot}, weight at {top}"


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("exp", [-100, 100])
@pytest.mark.parametrize("flat", [True, False])
def test_value_range_in_the_longest_call(t, exp, flat):
    """Values at the ends of the range in calls whose max_len is the largest: the
    range goes by the sequences' own lengths.  (f16: its own range.)"""
    length, hd, page, n = 700, 64, 4096, 20
    c, rng = make_cache(t, 1, hd, page, [length, 0], 82)
    exp = exp if t != "f16" else exp // 10
    k, v = (rng.standard_normal((length, 1, hd), dtype=np.float32) for _ in range(2))
    _fill(c, 0, k * np.float32(not flat), v * np.float32(2.0 ** exp))
    table = np.full((2, (1 << 30) // page), -1, np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table, c.cap = table, 1 << 30
    qh = synth.normal(3, synth.T_X, (2 * n, 4, hd), 1.5)
    d = Dev(c)
    for m, what in ((1, "decode"), (16, "decode"), (n, "prefill")):
        rows = np.ascontiguousarray(qh[:2 * m])
        out = torch.full((2 * m, 4 * hd), -7.0, device="cuda")
        if what == "decode":
            ws = workspace(q.qmv_attn_decode_workspace(d.h, m, 4, c.cap))
            q.qmv_attn_decode(d.h, m, 4, dev(rows.reshape(2 * m, -1)), 0.125, out, c.cap, workspace=ws)
        else:
            ws = workspace(q.qmv_attn_prefill_workspace(d.h, 2 * m, 4, c.cap))
            q.qmv_attn_prefill(d.h, 2 * m, 4, dev(rows.reshape(2 * m, -1)), 0.125, out, c.cap, workspace=ws)
        want, tol, _, _ = ref.attention(c, [0, m, 2 * m], rows, 0.125, length)
        close(host(out).reshape(want.shape), want, tol, f"{what} {t} m{m} 2^{exp}")


@pytest.mark.parametrize("t", ["f16", "bf16", "i8"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("hd", [64, 128])
def test_other_rows_of_a_bad_query(t, bad, hd):
    """A query that is not finite leaves its own row unspecified and no other."""
    length, n = 200, 40
    c, rng = make_cache(t, 1, hd, 16, [length], 83)
    qh = synth.normal(3, synth.T_X, (n, 3, hd), 1.5)
    scale = float(np.float32(hd ** -0.5))
    want, tol, _, _ = ref.attention(c, [0, n], qh, scale, c.cap)
    for i, j, col in ((n - 1, 0, 3), (n - 2, 2, 0), (n - 13, 1, hd - 1)):
        x = qh.copy()
        x[i, j, col] = bad
        for what, rows, got in _both(c, x, scale, n_decode=(16,)):
            m = len(rows)
            rest = np.ones((m, 3), bool)
            rest[i - (n - m), j] = False
            close(got[rest], want[n - m:][rest], tol[n - m:][rest], f"{what} {t} query {i} {bad}")
