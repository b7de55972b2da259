"""GPU parity of what stands around a cache's attention with the 64-bit
implementations in serve_ref.py and attn_ref.py, whose docstrings derive the
bounds: 4-bit caches (written, read, attended over, evicted from), norms and
rotation of queries and keys, pages taken and given back, and a run of them
together.  Cached bytes, pages and positions have to be equal."""
import numpy as np
import pytest

import synth
from tests import attn_ref as ref
from tests import serve_ref as sref
from tests.gpu_util import dev, host
from tests.serve_ref import PLACE, U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gguf_dequant_matvec_amd as q  # noqa: E402


def make4(kv, hd, page, lens, seed, extra=3, cap_pages=None, **scales):
    """A 4-bit cache with scattered pages; slots behind a length hold NaN scales."""
    rng = np.random.default_rng(seed)
    per = cap_pages or max(1, -(-max(max(lens), 1) // page))
    n_pages = len(lens) * per + extra
    table = rng.permutation(n_pages)[:len(lens) * per].reshape(len(lens), per)
    c = sref.Cache4(kv, hd, page, n_pages, table, lens, fill=0xFF)
    c.fill_pages(rng, **scales)
    for s, length in enumerate(lens):
        for p0 in range(0, per * page, page):
            pg, _ = c.where(s, p0)
            for h in range(kv):
                _, _, ks, vs = c.parts4(pg, h)
                ks[max(0, length - p0):] = np.nan
                vs[:, max(0, length - p0):] = np.nan
    return c, rng


class Dev:
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


def decode(c, n, heads, window=0, sinks=0, max_len=None, with_acc=False, seed=5, qstd=1.5):
    d = Dev(c)
    n_seq, max_len, scale = len(c.seq_len), max_len or c.cap, c.hd ** -0.5
    qh = synth.normal(seed, synth.T_X, (n_seq * n, heads, c.hd), qstd)
    out = torch.full((n_seq * n, heads, c.hd), float("nan"), device="cuda")
    acc0 = np.abs(synth.normal(seed + 1, synth.T_X, (n_seq, c.kv, max_len), 1.0)) if with_acc else None
    acc = dev(acc0) if with_acc else None
    ws = workspace(q.qmv_attn_decode_workspace(d.h, n, heads, max_len, window, sinks, with_acc))
    q.qmv_attn_decode(d.h, n, heads, dev(qh.reshape(n_seq * n, -1)), scale, out, max_len, window=window, sinks=sinks,
                      acc=acc, workspace=ws)
    want, tol, acc1, acc_tol = ref.attention(c, np.arange(n_seq + 1) * n, qh, scale, max_len, window, sinks, acc0)
    what = f"decode q4 hd{c.hd} page{c.page} lens{list(c.seq_len)[:4]} n{n} w{window}+{sinks}"
    close(host(out), want, tol, what)
    if with_acc:
        close(host(acc), acc1, acc_tol, what + " acc")


def prefill(c, news, heads, window=0, sinks=0, before=0, after=0, use_start=True, qstd=1.5):
    d = Dev(c)
    scale = c.hd ** -0.5
    start = (before + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + after
    qh = synth.normal(7, synth.T_X, (n, heads, c.hd), qstd)
    out = torch.full((n, heads, c.hd), -77.0, device="cuda")
    ws = workspace(q.qmv_attn_prefill_workspace(d.h, n, heads, c.cap, window, sinks))
    q.qmv_attn_prefill(d.h, n, heads, dev(qh.reshape(n, -1)), scale, out, c.cap, start=dev(start) if use_start else None,
                       window=window, sinks=sinks, workspace=ws)
    want, tol, _, _ = ref.attention(c, start, qh, scale, c.cap, window, sinks)
    got, none = host(out), np.isnan(want)
    assert np.all(got[none] == -77.0), "rows of no sequence were written"
    close(np.where(none, 0, got), np.where(none, 0, want), np.where(none, 1, tol),
          f"prefill q4 hd{c.hd} page{c.page} new{list(news)[:4]} w{window}+{sinks}")


# ---- a 4-bit cache written and read --------------------------------------------

def corner_rows(rng, n, kv, hd):
    """Rows whose blocks hold what rounding stumbles over."""
    x = rng.standard_normal((n, kv, hd), dtype=np.float32) * 2
    b = x.reshape(n, -1, 32)
    for r in range(n):
        i = r % 10
        if i == 0:
            b[r, 0] = 0
        elif i == 1:
            b[r, 0, 5], b[r, 0, 9] = 7.0, -7.0                       # both signs of the largest
        elif i == 2:
            b[r, -1] *= np.float32(1e-7)                             # subnormal scales
        elif i == 3:
            b[r, 0, 31] = np.inf
        elif i == 4:
            b[r, -1, 16] = -np.inf
        elif i == 5:
            b[r, 0, 3] = 3e38
        elif i == 6:
            b[r, 0] = np.arange(-16, 16, dtype=np.float32) * 0.5     # ties between codes
        elif i == 7:
            b[r, 0] = np.float32(1e-30)
        elif i == 8:
            b[r, -1] = -0.0
    return x


@pytest.mark.parametrize("hd,kv,page", [(64, 3, 16), (96, 1, 32), (128, 2, 64), (256, 1, 16)])
def test_append_q4(hd, kv, page):
    lens = [1, 0, 40, 23, 100]
    news = [1, 0, 17, 40, 3]          # the fourth has more rows than positions
    c, rng = make4(kv, hd, page, lens, 11)
    if page < 64:
        c.table[4, 98 // page] = -1
    d = Dev(c)
    start = (2 + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + 5
    k, v = corner_rows(rng, n, kv, hd), corner_rows(rng, n, kv, hd)[::-1].copy()
    both = dev(np.concatenate([k.reshape(n, -1), v.reshape(n, -1), k.reshape(n, -1)[:, :3]], 1))   # odd row stride
    w = kv * hd
    q.qmv_kv_append(d.h, n, both[:, :w], both[:, w:2 * w], start=dev(start))
    c.append(start, k, v)
    assert np.array_equal(d.pool(), c.pool)


def test_append_q4_nan():
    """A NaN makes its block NaN, in K and V, and no other."""
    c, rng = make4(1, 64, 16, [4], 12)
    d = Dev(c)
    k, v = (rng.standard_normal((4, 1, 64), dtype=np.float32) for _ in range(2))
    k[1, 0, 40], v[2, 0, 3] = np.nan, np.nan
    q.qmv_kv_append(d.h, 4, dev(k.reshape(4, -1)), dev(v.reshape(4, -1)))
    ko, vo = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda")
    q.qmv_kv_read(d.h, 4, ko, vo)
    ko, vo = host(ko), host(vo)
    assert np.all(np.isnan(ko[1, 32:])) and np.isnan(ko).sum() == 32
    assert np.all(np.isnan(vo[2, :32])) and np.isnan(vo).sum() == 32


@pytest.mark.parametrize("hd,kv,page", [(64, 8, 64), (96, 9, 16), (128, 8, 32)])
def test_append_q4_many_rows(hd, kv, page):
    """Long prompts: runs of 8 positions, cut by the sequences' and the workgroups' borders."""
    lens, news = [700, 5, 1203, 64, 500], [697, 1, 1203, 0, 497]
    c, rng = make4(kv, hd, page, lens, 13)
    c.table[2, 300 // page] = -1
    d = Dev(c)
    start = (1 + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + 2
    k, v = (rng.standard_normal((n, kv, hd), dtype=np.float32) for _ in range(2))
    q.qmv_kv_append(d.h, n, dev(k), dev(v), start=dev(start))
    c.append(start, k, v)
    assert np.array_equal(d.pool(), c.pool)


def test_append_q4_one_by_one_and_at_once():
    """Rows appended one at a time leave the bytes that appending all at once does: a byte of V
    holds two columns of one position, so none is shared between rows."""
    kv, hd, page, m = 2, 128, 16, 21
    c, rng = make4(kv, hd, page, [0, 0], 14, cap_pages=2)
    k, v = (rng.standard_normal((2, m, kv, hd), dtype=np.float32) for _ in range(2))
    c.seq_len[:] = m
    d = Dev(c)
    q.qmv_kv_append(d.h, 2 * m, dev(k.reshape(2 * m, -1)), dev(v.reshape(2 * m, -1)))
    e = Dev(c)
    for j in range(m):
        e.lens.fill_(j + 1)
        q.qmv_kv_append(e.h, 2, dev(k[:, j].reshape(2, -1)), dev(v[:, j].reshape(2, -1)))
    assert np.array_equal(d.pool(), e.pool())


@pytest.mark.parametrize("t", ["f16", "bf16", "i8", "q4"])
@pytest.mark.parametrize("hd,kv,page", [(64, 3, 16), (96, 2, 32), (128, 2, 64), (256, 1, 16)])
def test_read(t, hd, kv, page):
    """What append wrote comes back as the values it stands for; holes as zeros, other rows untouched."""
    rng = np.random.default_rng(15)
    lens, news = [30, 0, 100, 17], [30, 0, 40, 20]
    n_pages, per = 4 * 7, 7
    c = (sref.Cache4(kv, hd, page, n_pages, rng.permutation(n_pages).reshape(4, per), lens, fill=0x11) if t == "q4" else
         ref.Cache(t, kv, hd, page, n_pages, rng.permutation(n_pages).reshape(4, per), lens, fill=0x11))
    c.table[2, 80 // page] = -1
    start = (3 + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + 2
    k, v = (rng.standard_normal((n, kv, hd), dtype=np.float32) for _ in range(2))
    c.append(start, k, v)
    d = Dev(c)
    w = kv * hd
    ko, vo = torch.full((n, w + 4), -7.0, device="cuda"), torch.full((n, w), -7.0, device="cuda")
    q.qmv_kv_read(d.h, n, ko[:, 3:3 + w], vo, start=dev(start))
    want = np.full((2, n, kv, hd), -7.0)
    for s in range(4):
        for h in range(kv):
            K, V, there = c.rows(s, h, lens[s])
            K[~there], V[~there] = 0, 0
            for j in range(news[s]):
                p = lens[s] - news[s] + j
                if p >= 0:
                    want[0, start[s] + j, h], want[1, start[s] + j, h] = K[p], V[p]
    got = host(ko)
    assert np.all(got[:, :3] == -7) and np.all(got[:, 3 + w:] == -7)
    # (an 8-bit value is an f32 product of a scale and a code)
    assert np.array_equal(got[:, 3:3 + w].reshape(n, kv, hd), want[0].astype(np.float32))
    assert np.array_equal(host(vo).reshape(n, kv, hd), want[1].astype(np.float32))
    assert np.array_equal(d.pool(), c.pool)


# ---- attention over a 4-bit cache -----------------------------------------------

@pytest.mark.parametrize("hd,heads,kv,page", [(64, 9, 3, 16), (96, 4, 2, 32), (128, 8, 2, 64), (256, 5, 1, 16),
                                              (64, 17, 1, 128), (128, 2, 2, 16), (96, 20, 1, 64), (128, 18, 1, 32)])
def test_decode_q4_lengths(hd, heads, kv, page):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 257]
    c, _ = make4(kv, hd, page, lens, 21)
    decode(c, 1, heads)


@pytest.mark.parametrize("n,heads,kv,hd", [(2, 4, 2, 64), (5, 6, 2, 128), (8, 8, 2, 64), (16, 3, 1, 96), (16, 8, 1, 256),
                                           (3, 32, 1, 64), (8, 8, 1, 128), (1, 4, 1, 128), (1, 2, 1, 256), (2, 3, 1, 96)])
def test_decode_q4_several_tokens(n, heads, kv, hd):
    c, _ = make4(kv, hd, 32, [0, 1, n - 1, n, 40, 129, 300], 22)
    decode(c, n, heads, with_acc=True)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (100, 70), (5000, 3), (64, 1000)])
@pytest.mark.parametrize("n", [1, 7])
def test_decode_q4_window(window, sinks, n):
    c, _ = make4(2, 64, 16, [1, 20, 150, 333, 600], 23)
    decode(c, n, 6, window=window, sinks=sinks, with_acc=n == 7)


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_decode_q4_split(hd, window, sinks):
    c, _ = make4(2, hd, 64, [5003], 24, cap_pages=100)
    if window == 0:
        assert q.qmv_attn_decode_workspace(Dev(c).h, 1, 8, c.cap) > 0
    decode(c, 1, 8, window=window, sinks=sinks)
    decode(c, 4, 8, window=window, sinks=sinks, with_acc=True)


RAGGED = [2700, 0, 1, 64, 700, 31, 5200, 0, 0, 33] + [(37 * i) % 90 for i in range(30)]


@pytest.mark.parametrize("hd,kv,heads,n,window,sinks", [(64, 8, 16, 1, 0, 0), (64, 8, 16, 5, 5000, 9), (96, 8, 8, 1, 5100, 0),
                                                        (128, 8, 8, 3, 0, 0), (64, 2, 8, 11, 5000, 70), (128, 2, 6, 16, 5100, 3),
                                                        (256, 2, 18, 5, 5000, 40)])
def test_decode_q4_ragged(hd, kv, heads, n, window, sinks):
    """Even ranges over sequences of all lengths; several row tiles."""
    c, _ = make4(kv, hd, 64, RAGGED, 71)
    decode(c, n, heads, window=window, sinks=sinks, with_acc=n in (3, 5))


EVERY = [200, 0, 5200, 33, 64, 700] + [(53 * i) % 130 for i in range(34)]


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [3, 4, 5, 8, 9, 16, 20])
@pytest.mark.parametrize("shape", ["short", "split", "ranges"])
def test_decode_q4_every_kernel(hd, rows, shape):
    """Each way a call is cut (eight waves, pieces of one sequence, even ranges) with each packing of rows
    into the operand's columns, with and without weights."""
    n, group = (rows, 1) if rows <= 16 else (10, 2)
    lens, kv, cap = {"short": ([70, 300], 2, 5), "split": ([4100], 1, 70), "ranges": (EVERY, 8, 82)}[shape]
    c, _ = make4(kv, hd, 64, lens, 81, cap_pages=cap)
    for with_acc in (False, True):
        decode(c, n, kv * group, with_acc=with_acc)


def test_decode_q4_holes():
    c, _ = make4(1, 64, 16, [300, 300, 40], 25)
    c.table[0, 2:14] = -1
    c.table[1, 5] = c.n_pages
    c.table[1, 18] = 2 ** 31 - 1
    c.table[2, :] = -5
    decode(c, 1, 4, with_acc=True)
    decode(c, 3, 4, window=70, sinks=20)
    prefill(c, [20, 300, 7], 4)


@pytest.mark.parametrize("scales", [dict(kscale=(1e-6, 1e-4)), dict(kscale=(3, 9)), dict(vscale=(6e-8, 1e-6)),
                                    dict(vscale=(1000, 2720)), dict(kscale=(50, 2720))])
def test_q4_scale_range(scales):
    """Scales down to f16's smallest step and up to the largest that the writer gives; logits of thousands."""
    c, _ = make4(1, 128, 64, [700, 64], 26, **scales)
    decode(c, 2, 4, with_acc=True)
    prefill(c, [130, 64], 4)


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("what", ["k", "v"])
def test_q4_hidden_nan(hd, what):
    """Blocks whose scale is NaN or infinite reach the rows that see them and no others: those of V
    only their own columns."""
    n, length, group, bad = 12, 150, 2, 143           # the rows at 138 .. 142 do not see position 143
    c, _ = make4(1, hd, 16, [length], 27)
    clean, _, _, _ = ref.attention(c, [0, n], synth.normal(5, synth.T_X, (n, group, hd), 1.5), hd ** -0.5, 160)
    pg, slot = c.where(0, bad)
    _, _, ks, vs = c.parts4(pg, 0)
    if what == "k":
        ks[slot, 1] = np.nan
    else:
        vs[1, slot] = np.inf
    qh = synth.normal(5, synth.T_X, (n, group, hd), 1.5)
    _, tol, _, _ = ref.attention(make4(1, hd, 16, [length], 27)[0], [0, n], qh, hd ** -0.5, 160)
    for call in ("decode", "prefill"):
        d = Dev(c)
        out = torch.empty(n, group, hd, device="cuda")
        if call == "decode":
            ws = workspace(q.qmv_attn_decode_workspace(d.h, n, group, 160))
            q.qmv_attn_decode(d.h, n, group, dev(qh.reshape(n, -1)), hd ** -0.5, out, 160, workspace=ws)
        else:
            q.qmv_attn_prefill(d.h, n, group, dev(qh.reshape(n, -1)), hd ** -0.5, out, 160,
                               workspace=workspace(q.qmv_attn_prefill_workspace(d.h, n, group, 160)))
        got = host(out)
        blind = bad - (length - n)
        close(got[:blind], clean[:blind], tol[:blind], f"{call} rows that do not see it")
        if what == "v":
            assert not np.isfinite(got[blind:, :, 32:64]).any()
            rest = np.r_[0:32, 64:hd]
            close(got[blind:][..., rest], clean[blind:][..., rest], tol[blind:][..., rest], f"{call} other columns")


# the f16 scales whose 24-fold is infinite, of which the readers make infinite or NaN values
LARGE = np.arange(0x6955, 0x7C00, dtype=np.uint16)


def leave_scales(c, rng, hidden=lambda s, p: False):
    """Any codes and finite scales past what the writer gives in every slot that no row sees: behind the
    lengths, in pages of no sequence (page 0 among them, which is read in place of a hole) and where
    hidden(s, positions) says so."""
    old = np.flatnonzero(c.table.reshape(-1) == 0)
    if old.size:                                  # page 0 into no sequence's table
        spare = next(p for p in range(c.n_pages) if p not in set(c.table.reshape(-1).tolist()))
        c.pool[[0, spare]] = c.pool[[spare, 0]]
        c.table.reshape(-1)[old] = spare
    owner = {int(c.table[s, j]): (s, j) for s in range(c.table.shape[0]) for j in range(c.table.shape[1])}
    for pg in range(c.n_pages):
        s, j = owner.get(pg, (None, 0))
        at = np.arange(c.page)
        if s is not None:
            at = at[(j * c.page + at >= c.seq_len[s]) | hidden(s, j * c.page + at)]
        for h in range(c.kv):
            k, v, ks, vs = c.parts4(pg, h)
            k[at] = rng.integers(0, 256, (len(at), c.hd // 2))
            if s is None:
                v[:] = rng.integers(0, 256, v.shape)
            for d in (ks.view(np.uint16).T, vs.view(np.uint16)):
                d[:, at] = rng.choice(LARGE, (c.hd // 32, len(at))) | rng.choice([0, 0x8000], (c.hd // 32, len(at))).astype(np.uint16)
    assert not (c.table == 0).any()


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [1, 4, 6, 9, 20])
@pytest.mark.parametrize("shape", ["short", "split", "ranges"])
def test_decode_q4_leftover_scales(hd, rows, shape):
    """What slots that no row sees hold does not matter: scales that are finite but too large for attention."""
    n, group = {1: (1, 1), 4: (2, 2), 6: (6, 1), 9: (3, 3), 20: (10, 2)}[rows]
    lens, kv, cap = {"short": ([70, 301, 0, 1], 2, 5), "split": ([4133], 1, 70), "ranges": (EVERY, 8, 82)}[shape]
    c, rng = make4(kv, hd, 64, lens, 82, cap_pages=cap)
    leave_scales(c, rng)
    for with_acc in (False, True):
        decode(c, n, kv * group, with_acc=with_acc)


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
@pytest.mark.parametrize("window,sinks", [(33, 0), (100, 21)])
def test_q4_leftover_scales_outside_windows(hd, window, sinks):
    """... in holes, and in positions between the sinks and every row's window."""
    lens, news = [600, 333, 41], [1, 1, 1]
    for n in (1, 5):
        c, rng = make4(2, hd, 16, lens, 83)
        leave_scales(c, rng, lambda s, p: (p >= sinks) & (p <= c.seq_len[s] - n - window))
        c.table[0, 35] = -1                       # a hole inside the window, another behind it
        c.table[1, 3] = c.n_pages
        decode(c, n, 6, window=window, sinks=sinks, with_acc=True)
        prefill(c, [n] * 3, 6, window=window, sinks=sinks)


@pytest.mark.parametrize("hd,heads,kv,page", [(64, 9, 3, 16), (96, 4, 2, 32), (128, 8, 2, 64), (256, 5, 1, 16)])
def test_prefill_q4_leftover_scales(hd, heads, kv, page):
    c, rng = make4(kv, hd, page, [0, 1, 33, 64, 130, 203], 84)
    leave_scales(c, rng)
    c.table[5, 64 // page] = -1
    prefill(c, [0, 1, 33, 20, 130, 97], heads, before=3, after=4)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bits", [0x6954, 0xE954, 0x6955, 0xE955, 0x7BFF, 0xFBFF])
def test_q4_scale_too_large(hd, bits):
    """A V scale past 2728 counts as not finite for the rows that see it, in chunks that all rows see and
    in others, and changes nothing for other rows and columns; one of 2728 is a scale like others."""
    n, length, group = 70, 300, 2
    finite = bits & 0x7FFF < 0x6955
    for bad in (40, 271, 294, 299):              # seen by all rows; by the last 29, 6, 1
        c, _ = make4(1, hd, 16, [length], 85)
        pg, slot = c.where(0, bad)
        _, _, _, vs = c.parts4(pg, 0)
        qh = synth.normal(5, synth.T_X, (n, group, hd), 1.5)
        clean, tol, _, _ = ref.attention(c, [0, n], qh, hd ** -0.5, 304)
        vs.view(np.uint16)[1, slot] = bits
        want, wtol, _, _ = ref.attention(c, [0, n], qh, hd ** -0.5, 304)
        # (24 * 2728 is an f16 value; scale * code, below 2^15 and of more bits than f16 has, is rounded once, to
        # steps of 16: off by 8, times a weight of at most 1)
        wtol = wtol + np.where(np.arange(hd) // 32 == 1, 8.0, 0.0)
        blind = max(0, bad - (length - n))
        for call, m in (("decode", 2), ("decode", 4), ("decode", 12), ("prefill", n)):
            d = Dev(c)
            rows = dev(qh[-m:].reshape(m, -1))
            out = torch.empty(m, group, hd, device="cuda")
            if call == "decode":
                q.qmv_attn_decode(d.h, m, group, rows, hd ** -0.5, out, 304,
                                  workspace=workspace(q.qmv_attn_decode_workspace(d.h, m, group, 304)))
            else:
                q.qmv_attn_prefill(d.h, m, group, rows, hd ** -0.5, out, 304,
                                   workspace=workspace(q.qmv_attn_prefill_workspace(d.h, m, group, 304)))
            got = np.full((n, group, hd), np.nan, np.float32)
            got[n - m:] = host(out)
            what = f"{call} of {m} {bits:#x} at {bad}"
            first = max(blind, n - m)
            if finite:
                close(got[n - m:], want[n - m:], wtol[n - m:], what)
                continue
            if blind > n - m:
                close(got[n - m:blind], clean[n - m:blind], tol[n - m:blind], what + ", rows that do not see it")
            assert not np.isfinite(got[first:, :, 32:64]).any(), what
            rest = np.r_[0:32, 64:hd]
            close(got[first:][..., rest], clean[first:][..., rest], tol[first:][..., rest], what + ", other columns")


@pytest.mark.parametrize("hd,heads,kv,page", [(64, 9, 3, 16), (96, 4, 2, 32), (128, 8, 2, 64), (256, 5, 1, 16), (64, 17, 1, 128)])
def test_prefill_q4_ragged(hd, heads, kv, page):
    c, _ = make4(kv, hd, page, [0, 1, 33, 64, 130, 200], 31)
    prefill(c, [0, 1, 33, 20, 130, 97], heads, before=3, after=4)


@pytest.mark.parametrize("n,length", [(1, 1), (17, 40), (150, 150), (64, 300)])
def test_prefill_q4_even(n, length):
    c, _ = make4(2, 64, 32, [length, max(0, length - 9), length], 32)
    prefill(c, [n] * 3, 6, use_start=False)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (300, 0), (1000, 70)])
def test_prefill_q4_window(hd, window, sinks):
    c, _ = make4(2, hd, 16, [600, 333], 33)
    prefill(c, [600, 200], 6, window=window, sinks=sinks)


def test_prefill_q4_split():
    """Few rows after a long context are cut along the length."""
    c, _ = make4(1, 128, 64, [6000], 34)
    assert q.qmv_attn_prefill_workspace(Dev(c).h, 20, 4, c.cap) > 0
    prefill(c, [20], 4)


def test_q4_far_pages():
    """Pages beyond 4 GiB of the pool, written, read and attended over."""
    kv, hd, page = 8, 256, 64
    c, rng = make4(kv, hd, page, [200], 35)
    pb = q.qmv_kv_page_bytes("q4", kv, hd, page)
    n_pages = (9 << 29) // pb + 7                    # 4.5 GiB
    pool = torch.zeros(n_pages * pb, dtype=torch.uint8, device="cuda")
    far = np.array([[n_pages - 1 - 3 * i for i in range(c.table.shape[1])]], np.int32)
    view = pool.view(n_pages, pb)
    for i, pg in enumerate(c.table[0]):
        view[int(far[0, i])] = dev(c.pool[pg].reshape(-1))
    cache = q.KvCache("q4", kv, hd, page, pool, dev(far), dev(c.seq_len))
    k, v = (rng.standard_normal((3, kv, hd), dtype=np.float32) for _ in range(2))
    q.qmv_kv_append(cache, 3, dev(k), dev(v))
    c.append([0, 3], k, v)
    for i, pg in enumerate(c.table[0]):
        assert np.array_equal(host(view[int(far[0, i])]), c.pool[pg].reshape(-1))
    qh = synth.normal(4, synth.T_X, (20, 8, hd), 1.0)
    want, tol, _, _ = ref.attention(c, [0, 20], qh, hd ** -0.5, 256)
    out = torch.empty(20, 8, hd, device="cuda")
    q.qmv_attn_prefill(cache, 20, 8, dev(qh.reshape(20, -1)), hd ** -0.5, out, 256,
                       workspace=workspace(q.qmv_attn_prefill_workspace(cache, 20, 8, 256)))
    close(host(out), want, tol, "far pages, prefill")
    want, tol, _, _ = ref.attention(c, [0, 1], qh[:1], hd ** -0.5, 256)
    q.qmv_attn_decode(cache, 1, 8, dev(qh[:1].reshape(1, -1)), hd ** -0.5, out[:1], 256,
                      workspace=workspace(q.qmv_attn_decode_workspace(cache, 1, 8, 256)))
    close(host(out[:1]), want, tol, "far pages, decode")


@pytest.mark.parametrize("hd,kv,page", [(64, 3, 16), (96, 1, 32), (128, 2, 64), (256, 1, 16)])
@pytest.mark.parametrize("keep,first,recent", [(70, 4, 16), (97, 0, 0), (33, 10, 23), (300, 4, 4), (1, 1, 0)])
def test_evict_q4(hd, kv, page, keep, first, recent):
    """Kept rows move with their codes and scales; a hole's become zeros."""
    lens = [200, 0, 90, 130]
    c, rng = make4(kv, hd, page, lens, 41, extra=4 * (-(-300 // page)) + 2)
    used = set(c.table.reshape(-1).tolist())
    free = np.array([p for p in range(c.n_pages) if p not in used])
    per = -(-keep // page)
    dst = free[:4 * per].reshape(4, per).astype(np.int32)
    c.table[3, 32 // page] = -1
    if per > 1:
        dst[2, 1] = -1
    acc = rng.random((4, kv, 200), dtype=np.float32)
    d = Dev(c)
    kept = torch.full((4, kv, keep), -9, dtype=torch.int32, device="cuda")
    acc_out, len_out = torch.empty(4, kv, keep, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    q.qmv_kv_evict(d.h, dev(dst), keep, first, recent, dev(acc), kept, acc_out, len_out)
    old = sref.Cache4(c.kv, c.hd, c.page, c.n_pages, c.table, c.seq_len)
    old.pool = c.pool.copy()
    to = sref.Cache4(c.kv, c.hd, c.page, c.n_pages, dst, c.seq_len)
    to.pool = c.pool
    for s, length in enumerate(lens):
        for h in range(kv):
            if length <= keep:
                chosen = list(range(length))
            else:
                rank = sorted(range(first, length - recent), key=lambda p: (-float(acc[s, h, p]), p))
                chosen = sorted(list(range(first)) + rank[:keep - first - recent] + list(range(length - recent, length)))
            assert host(kept)[s, h, :len(chosen)].tolist() == chosen
            for i, p in enumerate(chosen):
                at = to.where(s, i)
                if at[0] is None:
                    continue
                src = old.where(s, p)
                if src[0] is None:
                    sref.copy_row4(to, src, at, h)
                    continue
                k0, v0, ks0, vs0 = old.parts4(src[0], h)
                k1, v1, ks1, vs1 = to.parts4(at[0], h)
                k1[at[1]], ks1[at[1]], vs1[:, at[1]] = k0[src[1]], ks0[src[1]], vs0[:, src[1]]
                v1[at[1] // 16, :, PLACE[at[1] % 16]] = v0[src[1] // 16, :, PLACE[src[1] % 16]]
    assert host(len_out).tolist() == [min(x, keep) for x in lens]
    assert np.array_equal(d.pool(), c.pool)


def test_q4_captured():
    """Append, decode, prompt and read captured once; replays follow lengths and pages changed in place."""
    kv, hd, page, heads = 2, 128, 16, 8
    c, rng = make4(kv, hd, page, [200, 90], 91, cap_pages=16)
    d = Dev(c)
    k, v, x = (torch.zeros(2, w, device="cuda") for w in (kv * hd, kv * hd, heads * hd))
    ko, vo, out = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(x)
    ws = workspace(q.qmv_attn_decode_workspace(d.h, 1, heads, c.cap))
    pout = torch.zeros(2, heads * hd, device="cuda")
    pws = workspace(q.qmv_attn_prefill_workspace(d.h, 2, heads, c.cap))

    def step():
        q.qmv_kv_append(d.h, 2, k, v)
        q.qmv_attn_decode(d.h, 1, heads, x, hd ** -0.5, out, c.cap, workspace=ws)
        q.qmv_attn_prefill(d.h, 2, heads, x, hd ** -0.5, pout, c.cap, workspace=pws)
        q.qmv_kv_read(d.h, 2, ko, vo)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        lens = np.array([[200, 90], [201, 1], [17, 256], [0, 33]][rep], np.int32)
        d.lens.copy_(dev(lens))
        c.seq_len[:] = lens
        kh, vh, xh = (rng.standard_normal(tuple(t.shape), dtype=np.float32) for t in (k, v, x))
        c.pool[:] = d.pool()
        for t, h in ((k, kh), (v, vh), (x, xh)):
            t.copy_(dev(h))
        g.replay()
        torch.cuda.synchronize()
        c.append([0, 1, 2], kh.reshape(2, kv, hd), vh.reshape(2, kv, hd))
        assert np.array_equal(d.pool(), c.pool), rep
        want, tol, _, _ = ref.attention(c, [0, 1, 2], xh.reshape(2, heads, hd), hd ** -0.5, c.cap)
        # (positions behind the first lengths hold NaN scales: a longer one sees them, and is NaN)
        nan = np.isnan(want)
        assert nan.any() == (rep == 2)
        for got, what in ((out, "decode"), (pout, "prompt")):
            got = host(got).reshape(want.shape)
            assert np.isnan(got[nan]).all()
            close(np.where(nan, 0, got), np.where(nan, 0, want), np.where(nan, 1, tol), f"replay {rep}, {what}")
        eager = [t.clone() for t in (out, pout, ko, vo)]
        step()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(a), host(b), equal_nan=True) for a, b in zip(eager, (out, pout, ko, vo)))


# ---- norms and rotation -----------------------------------------------------------

def make_rope(hd, rot, pairs, norm, rng, base=10000.0, eps=1e-5):
    freq = base ** (-2 * np.arange(rot // 2) / max(rot, 1))
    wq, wk = ((1 + 0.3 * rng.standard_normal((2, hd))).astype(np.float32) if norm else (None, None))
    h = q.QkRope(dev(freq) if rot else 0, rot, pairs, dev(wq) if norm else None, dev(wk) if norm else None, eps)
    return h, freq, wq, wk, eps


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("hd,rot", [(64, 64), (64, 24), (96, 96), (96, 64), (96, 8), (128, 128), (128, 32), (256, 256), (256, 80),
                                    (128, 0)])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(hd, rot, pairs, norm):
    """Column ranges of stacked rows in, rows with a gap out; rows at negative positions stay."""
    rng = np.random.default_rng(hd + rot)
    h, freq, wq, wk, eps = make_rope(hd, rot, pairs, norm, rng)
    for n, heads, kv in ((1, 1, 1), (7, 9, 3), (37, 5, 0), (3, 0, 2)):
        pos = rng.integers(0, 5000, n).astype(np.int32)
        if n > 3:
            pos[2], pos[5] = -1, 0
        w = (heads + 2 * kv) * hd
        x = rng.standard_normal((n, w), dtype=np.float32) * rng.uniform(0.01, 30, (n, 1)).astype(np.float32)
        xd = dev(x)
        qo, ko = torch.full((n, heads * hd + 3), -5.0, device="cuda"), torch.full((n, max(kv, 1) * hd), -5.0, device="cuda")
        q.qmv_qk_norm_rope(h, hd, n, dev(pos), heads, xd[:, :heads * hd] if heads else None, qo[:, 1:1 + heads * hd] if heads else None,
                           kv, xd[:, heads * hd:(heads + kv) * hd] if kv else None, ko if kv else None)
        for part, got, weight, m in ((x[:, :heads * hd], host(qo)[:, 1:1 + heads * hd], wq, heads),
                                     (x[:, heads * hd:(heads + kv) * hd], host(ko)[:, :kv * hd], wk, kv)):
            if m == 0:
                continue
            want, tol = sref.rope(part.reshape(n, m, hd), weight, pos, freq, rot, pairs, eps)
            got = got.reshape(n, m, hd)
            assert np.all(got[pos < 0] == -5)
            close(got[pos >= 0], want[pos >= 0], tol[pos >= 0], f"hd{hd} rot{rot} {pairs} norm {norm} n{n}")
        qo = host(qo)
        assert np.all(qo[:, 0] == -5) and np.all(qo[:, 1 + heads * hd:] == -5)
        assert np.array_equal(host(xd), x)


@pytest.mark.parametrize("hd", [64, 96, 128, 256])
def test_norm_rope_many_rows(hd):
    """Enough rows for several heads a lane group; a number of heads that it does not divide."""
    rng = np.random.default_rng(3)
    h, freq, wq, wk, eps = make_rope(hd, hd, "halves", True, rng)
    n, heads, kv = 3001, 9, 3
    pos = rng.integers(-3, 100000, n).astype(np.int32)
    x = rng.standard_normal((n, heads + kv, hd), dtype=np.float32)
    xd = dev(x.reshape(n, -1))
    qo, ko = torch.zeros(n, heads * hd, device="cuda"), torch.zeros(n, kv * hd, device="cuda")
    q.qmv_qk_norm_rope(h, hd, n, dev(pos), heads, xd[:, :heads * hd], qo, kv, xd[:, heads * hd:], ko)
    for part, got, weight in ((x[:, :heads], qo, wq), (x[:, heads:], ko, wk)):
        want, tol = sref.rope(part, weight, pos, freq, hd, "halves", eps)
        want[pos < 0] = 0
        close(host(got).reshape(want.shape), want, tol, f"hd{hd}")
    # in place: the same bits
    q.qmv_qk_norm_rope(h, hd, n, dev(pos), heads, xd[:, :heads * hd], xd[:, :heads * hd], kv, xd[:, heads * hd:], xd[:, heads * hd:])
    got = host(xd).reshape(n, heads + kv, hd)
    live = pos >= 0
    assert np.array_equal(got[live][:, :heads], host(qo).reshape(n, heads, hd)[live])
    assert np.array_equal(got[live][:, heads:], host(ko).reshape(n, kv, hd)[live])
    assert np.array_equal(got[~live], x[~live])


def test_norm_rope_far_positions():
    """Positions up to 2^30 and any frequency: whole turns go in 64 bits."""
    rng = np.random.default_rng(4)
    freq = np.concatenate([rng.uniform(0, 1, 28), [1.0, 0.0, 1e-12, -0.37]])
    h = q.QkRope(dev(freq), 64, "adjacent")
    pos = np.array([0, 1, 4095, 65537, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 29 + 3, 2 ** 30], np.int32)
    x = rng.standard_normal((8, 2, 64), dtype=np.float32)
    out = torch.empty(8, 128, device="cuda")
    q.qmv_qk_norm_rope(h, 64, 8, dev(pos), 2, dev(x.reshape(8, -1)), out)
    want, tol = sref.rope(x, None, pos, freq, 64, "adjacent", 0)
    close(host(out).reshape(8, 2, 64), want, tol, "far positions")


def test_norm_of_zero_and_large_rows():
    """A zero row stays zero, eps 0 or not (0 / 0 is NaN, as the formula says); rows near the ends of the range."""
    rng = np.random.default_rng(5)
    w = dev(np.ones(64, np.float32))
    x = rng.standard_normal((4, 1, 64), dtype=np.float32)
    x[0] = 0
    x[1] *= np.float32(1e17)
    x[2] *= np.float32(1e-15)
    for eps in (1e-6, 0.0):
        h = q.QkRope(0, 0, "halves", w, None, eps)
        out = torch.empty(4, 64, device="cuda")
        q.qmv_qk_norm_rope(h, 64, 4, dev(np.arange(4, dtype=np.int32)), 1, dev(x.reshape(4, -1)), out)
        got = host(out).reshape(4, 1, 64)
        want, tol = sref.rope(x[1:], np.ones(64), np.arange(3), None, 0, "halves", eps)
        close(got[1:], want, tol, f"eps {eps}")
        assert np.isnan(got[0]).all() if eps == 0 else not got[0].any()


@pytest.mark.parametrize("t", ["f16", "bf16", "i8", "q4"])
@pytest.mark.parametrize("hd,kv,heads,page,pairs,rot", [(64, 3, 9, 16, "halves", 64), (96, 2, 4, 32, "adjacent", 96),
                                                        (128, 2, 8, 64, "halves", 48), (256, 1, 5, 16, "adjacent", 256)])
@pytest.mark.parametrize("many", [False, True])
def test_append_rope(t, hd, kv, heads, page, pairs, rot, many):
    """The joined call leaves the bytes that the two calls leave, and the same queries; those are
    held to the reference above."""
    rng = np.random.default_rng(6)
    lens, news = ([900, 8000 // kv, 0, 3000 // kv], [700, 8000 // kv, 0, 2900 // kv]) if many else ([5, 0, 40, 20, 100], [1, 0, 17, 33, 3])
    n_seq, per = len(lens), -(-max(lens) // page)
    n_pages = n_seq * per + 2
    table = rng.permutation(n_pages)[:n_seq * per].reshape(n_seq, per).astype(np.int32)
    table[-1, (lens[-1] - 2) // page] = -1
    pb = q.qmv_kv_page_bytes(t, kv, hd, page)
    pools = [torch.full((n_pages * pb,), 0x3C, dtype=torch.uint8, device="cuda") for _ in range(2)]
    caches = [q.KvCache(t, kv, hd, page, p, dev(table), dev(np.array(lens, np.int32))) for p in pools]
    h, freq, wq, wk, eps = make_rope(hd, rot, pairs, True, rng)
    start = (2 + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
    n = int(start[-1]) + 3
    x = rng.standard_normal((n, (heads + 2 * kv) * hd), dtype=np.float32)
    pos = np.full(n, -1, np.int32)
    for s in range(n_seq):
        pos[start[s]:start[s + 1]] = np.maximum(lens[s] - news[s] + np.arange(news[s]), -1)
    xd = dev(x)
    qd, kd, vd = xd[:, :heads * hd], xd[:, heads * hd:(heads + kv) * hd], xd[:, (heads + kv) * hd:]
    two, k2, one = torch.full((n, heads * hd), -5.0, device="cuda"), torch.zeros(n, kv * hd, device="cuda"), \
        torch.full((n, heads * hd), -5.0, device="cuda")
    q.qmv_qk_norm_rope(h, hd, n, dev(pos), heads, qd, two, kv, kd, k2)
    q.qmv_kv_append(caches[0], n, k2, vd, start=dev(start))
    q.qmv_kv_append_rope(caches[1], h, n, heads, qd, one, kd, vd, start=dev(start))
    assert torch.equal(pools[0], pools[1])
    assert torch.equal(one, two)
    want, tol = sref.rope(x[:, :heads * hd].reshape(n, heads, hd), wq, pos, freq, rot, pairs, eps)
    live = pos >= 0
    close(host(one).reshape(want.shape)[live], want[live], tol[live], "queries")
    # in place, the rows' queries among their keys and values
    pools[1].fill_(0x3C)
    q.qmv_kv_append_rope(caches[1], h, n, heads, qd, qd, kd, vd, start=dev(start))
    assert torch.equal(pools[0], pools[1]) and torch.equal(qd[torch.from_numpy(live).cuda()], one[torch.from_numpy(live).cuda()])
    assert np.array_equal(host(xd)[~live], x[~live]) and np.array_equal(host(xd)[:, heads * hd:], x[:, heads * hd:])


# ---- pages ------------------------------------------------------------------------

class Pool:
    """A page table's state on the device beside the reference's."""

    def __init__(self, table, lens, free, count, page, n_pages):
        self.ref = sref.Pages(table, lens, free, count, page, n_pages)
        self.table, self.lens = dev(self.ref.table), dev(self.ref.seq_len)
        self.free, self.count = dev(self.ref.free), dev(np.array([count], np.int32))
        self.n_seq = len(lens)
        pages = torch.empty(n_pages * q.qmv_kv_page_bytes("q4", 1, 64, page), dtype=torch.uint8, device="cuda")
        self.h = q.KvCache("q4", 1, 64, page, pages, self.table, self.lens)

    def same(self, what):
        assert np.array_equal(host(self.table), self.ref.table), what
        assert np.array_equal(host(self.lens), self.ref.seq_len), what
        assert int(host(self.count)[0]) == self.ref.count, what
        assert np.array_equal(host(self.free), self.ref.free), what

    def reserve(self, add, n, rows=True):
        m = self.n_seq
        granted, start = (torch.full((k,), -3, dtype=torch.int32, device="cuda") for k in (m, m + 1))
        pos = torch.full((n + 3,), -9, dtype=torch.int32, device="cuda") if rows else None
        slot = torch.full((n + 3,), -9, dtype=torch.int64, device="cuda") if rows else None
        q.qmv_kv_reserve(self.h, dev(np.array(add, np.int32)), self.free, self.count, n, granted, start, pos=pos, slot=slot)
        g, st, p, sl = self.ref.reserve(add, n)
        assert np.array_equal(host(granted), g) and np.array_equal(host(start), st)
        if rows:
            assert np.array_equal(host(pos)[:n], p) and np.array_equal(host(slot)[:n], sl)
            assert np.all(host(pos)[n:] == -9) and np.all(host(slot)[n:] == -9)
        self.same("reserve")
        return g

    def release(self, new_len):
        q.qmv_kv_release(self.h, dev(np.array(new_len, np.int32)), self.free, self.count)
        self.ref.release(new_len)
        self.same("release")


def empty_pool(n_seq, per, page, n_pages, seed=1):
    rng = np.random.default_rng(seed)
    return Pool(np.full((n_seq, per), -1), [0] * n_seq, rng.permutation(n_pages), n_pages, page, n_pages), rng


@pytest.mark.parametrize("n_seq,per,page,n_pages,n", [(1, 4, 16, 4, 64), (7, 9, 16, 40, 500), (64, 20, 64, 700, 4096),
                                                      (300, 30, 32, 3000, 9000), (1024, 4, 16, 3000, 4097),
                                                      (1025, 5, 16, 2500, 30000), (2500, 3, 16, 4000, 4000)])
def test_pages_random_steps(n_seq, per, page, n_pages, n):
    """Steps of a serving loop: some sequences end, some give up drafted tokens, all ask for more, more
    than there is now and then."""
    p, rng = empty_pool(n_seq, per, page, n_pages)
    for step in range(6):
        top = [1, per * page, 16, per * page // 2, 3, per * page + 5][step]
        add = rng.integers(-1, top + 1, n_seq)
        if step == 3:
            add[rng.random(n_seq) < 0.5] = 0
        p.reserve(add, n, rows=step != 4)
        lens = p.ref.seq_len
        new = np.where(rng.random(n_seq) < 0.3, rng.integers(0, np.maximum(lens, 1) + 1), -1)
        new[rng.random(n_seq) < 0.2] = 0
        if step == 2:
            new[:] = lens + 1                     # nothing to give back
        p.release(new)


def test_pages_refused_sequences():
    """Exactly enough pages, one too few, a table row too short, a length below 0, rows past n."""
    def fresh(count):
        return Pool(np.full((6, 4), -1), [0, 16, 5, -2, 60, 64], np.arange(10)[::-1].copy(), count, 16, 10)
    p = fresh(4)
    p.ref.table[1, 0] = p.ref.table[2, 0] = 9
    p.table.copy_(dev(p.ref.table))
    g = p.reserve([32, 1, 11, 5, 4, 1], 100)
    assert g.tolist() == [32, 1, 11, 0, 4, 0]     # 2 pages, 1, none wanted; -2; none wanted; the row is full
    p = fresh(2)
    assert p.reserve([32, 1, 11, 5, 4, 1], 100).tolist() == [32, 0, 11, 0, 4, 0]
    p = fresh(1)
    assert p.reserve([32, 1, 11, 5, 4, 1], 100).tolist() == [0, 0, 11, 0, 4, 0]
    p = fresh(10)
    assert p.reserve([32, 1, 11, 5, 4, 1], 43).tolist() == [32, 1, 0, 0, 0, 0]   # what comes behind the 44th row
    p = fresh(10)
    assert p.reserve([2 ** 31 - 1, 1, 2 ** 31 - 1, -2 ** 31, 1, 2 ** 31 - 1], 43).tolist() == [0, 1, 0, 0, 1, 0]
    p = fresh(0)
    assert not p.reserve([0] * 6, 1).any()


def test_pages_any_state():
    """Counts and lengths out of range, holes and foreign numbers in the table and the stack."""
    rng = np.random.default_rng(8)
    for count in (-5, 0, 37, 2 ** 31 - 1):
        table = rng.integers(-3, 45, (40, 6))
        lens = rng.integers(-20, 130, 40)
        lens[3], lens[4] = 2 ** 31 - 1, -2 ** 31
        p = Pool(table, lens, rng.integers(-2, 45, 40), count, 16, 40)
        p.ref.count = min(max(count, 0), 40)
        new = rng.integers(-1, 60, 40)
        q.qmv_kv_release(p.h, dev(new.astype(np.int32)), p.free, p.count)
        p.ref.release(new)
        p.same(f"count {count}")
        p.reserve(np.clip(rng.integers(-5, 30, 40), None, None), 300)


def test_pages_come_back_in_order():
    """What is released and reserved again lies where it lay."""
    p, rng = empty_pool(50, 12, 16, 500)
    p.reserve(rng.integers(1, 150, 50), 10000)
    table, lens = p.ref.table.copy(), p.ref.seq_len.copy()
    p.release(lens // 3)
    p.reserve(lens - lens // 3, 10000)
    assert np.array_equal(host(p.table), table)


# ---- together ---------------------------------------------------------------------

def serve_step(p, pool, h, heads, kv, hd, add, n, x, keep, captured=False):
    """One step of a serving loop on the current stream: drafted tokens of the last step given up, new ones
    reserved, normed, turned and appended, and their attention."""
    q.qmv_kv_release(p["cache"], keep, p["free"], p["count"])
    q.qmv_kv_reserve(p["cache"], add, p["free"], p["count"], n, p["granted"], p["start"], pos=p["pos"])
    xq, xk, xv = x[:, :heads * hd], x[:, heads * hd:(heads + kv) * hd], x[:, (heads + kv) * hd:]
    q.qmv_kv_append_rope(p["cache"], h, n, heads, xq, p["q"], xk, xv, start=p["start"])
    q.qmv_attn_decode(p["cache"], n // p["cache"].n_seq, heads, p["q"], hd ** -0.5, p["out"], p["max"], workspace=p["ws"])


@pytest.mark.parametrize("t", ["q4", "f16"])
def test_serving_steps_in_a_graph(t):
    """Steps of four sequences with three tokens each, captured once and replayed with new rows, lengths and
    pages, against the references step by step; eager calls between the replays."""
    rng = np.random.default_rng(9)
    n_seq, m, heads, kv, hd, page, per = 4, 3, 6, 2, 64, 16, 8
    n, n_pages = n_seq * m, 40
    c = (sref.Cache4(kv, hd, page, n_pages, np.full((n_seq, per), -1), [0] * n_seq, fill=0xFF) if t == "q4" else
         ref.Cache(t, kv, hd, page, n_pages, np.full((n_seq, per), -1), [0] * n_seq, fill=0xFF))
    d = Dev(c)
    state = sref.Pages(c.table, c.seq_len, rng.permutation(n_pages), n_pages, page, n_pages)
    h, freq, wq, wk, eps = make_rope(hd, hd, "halves", True, rng)

    def i32(k):
        return torch.zeros(k, dtype=torch.int32, device="cuda")

    p = dict(cache=d.h, free=dev(state.free), count=dev(np.array([n_pages], np.int32)), granted=i32(n_seq), start=i32(n_seq + 1),
             pos=i32(n), q=torch.zeros(n, heads * hd, device="cuda"), out=torch.zeros(n, heads * hd, device="cuda"), max=per * page)
    p["ws"] = workspace(q.qmv_attn_decode_workspace(d.h, m, heads, per * page))
    add, keep, x = dev(np.full(n_seq, m, np.int32)), i32(n_seq), torch.zeros(n, (heads + 2 * kv) * hd, device="cuda")
    keep.fill_(-1)

    def step():
        serve_step(p, d, h, heads, kv, hd, add, n, x, keep)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                  # a first, eager step on a stream of its own
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    q.qmv_kv_release(d.h, i32(n_seq), p["free"], p["count"])
    d.pages.fill_(0xFF)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens = np.zeros(n_seq, np.int64)
    for rep in range(9):
        cut = np.maximum(lens - rng.integers(0, m + 1, n_seq), 0)
        if rep == 5:
            cut[2] = 0                              # a sequence ends, another takes its place
        if rep == 0:
            cut[:] = -1
        xh = rng.standard_normal(tuple(x.shape), dtype=np.float32)
        keep.copy_(dev(cut.astype(np.int32)))
        x.copy_(dev(xh))
        p["out"].fill_(7)
        if rep % 3 == 2:
            step()
        else:
            g.replay()
        torch.cuda.synchronize()
        state.release(cut)
        granted, start, pos, _ = state.reserve([m] * n_seq, n)
        assert granted.tolist() == [m] * n_seq
        assert np.array_equal(host(d.table), state.table) and np.array_equal(host(d.lens), state.seq_len)
        assert np.array_equal(host(p["pos"]), pos) and int(host(p["count"])[0]) == state.count
        lens = state.seq_len.astype(np.int64)
        c.table[:], c.seq_len[:] = state.table, state.seq_len
        want_q, tol_q = sref.rope(xh[:, :heads * hd].reshape(n, heads, hd), wq, pos, freq, hd, "halves", eps)
        close(host(p["q"]).reshape(want_q.shape), want_q, tol_q, f"step {rep} queries")
        # the cache as the device holds it (its rounding of the turned keys is tested above)
        c.pool[:] = d.pool()
        want, tol, _, _ = ref.attention(c, start, host(p["q"]).reshape(n, heads, hd), hd ** -0.5, per * page)
        close(host(p["out"]).reshape(want.shape), want, tol, f"step {rep}")


@pytest.mark.parametrize("t", ["q4", "f16"])
def test_evicted_and_appended_at_the_callers_positions(t):
    """After an eviction a sequence's lengths are less than its tokens were, and kept keys stay turned by their
    old positions: the next tokens are turned to their own by qmv_qk_norm_rope and appended as they are."""
    rng = np.random.default_rng(12)
    kv, heads, hd, page, n, keep, m = 2, 6, 64, 16, 90, 40, 3
    per = 8
    c = (sref.Cache4(kv, hd, page, 2 * per, np.arange(per)[None], [n], fill=0) if t == "q4" else
         ref.Cache(t, kv, hd, page, 2 * per, np.arange(per)[None], [n], fill=0))
    d = Dev(c)
    h, freq, wq, wk, eps = make_rope(hd, hd, "halves", True, rng)
    x = rng.standard_normal((n, (heads + 2 * kv) * hd), dtype=np.float32)
    xd, w = dev(x), heads * hd
    qo = torch.empty(n, w, device="cuda")
    q.qmv_kv_append_rope(d.h, h, n, heads, xd[:, :w], qo, xd[:, w:w + kv * hd], xd[:, w + kv * hd:])
    acc = dev(rng.random((1, kv, n), dtype=np.float32))
    dst = dev((per + np.arange(per, dtype=np.int32))[None])
    kept, acc_out = torch.empty(1, kv, keep, dtype=torch.int32, device="cuda"), torch.empty(1, kv, keep, device="cuda")
    q.qmv_kv_evict(d.h, dst, keep, 4, 8, acc, kept, acc_out, d.lens)
    assert int(host(d.lens)[0]) == keep
    after = q.KvCache(t, kv, hd, page, d.pages, dst, d.lens)
    d.lens.add_(m)
    # tokens n, n + 1, n + 2 of the sequence at the cache's positions keep, keep + 1, keep + 2
    y = rng.standard_normal((m, (heads + 2 * kv) * hd), dtype=np.float32)
    yd, pos = dev(y), np.arange(n, n + m, dtype=np.int32)
    yq, yk = torch.empty(m, w, device="cuda"), torch.empty(m, kv * hd, device="cuda")
    q.qmv_qk_norm_rope(h, hd, m, dev(pos), heads, yd[:, :w], yq, kv, yd[:, w:w + kv * hd], yk)
    q.qmv_kv_append(after, m, yk, yd[:, w + kv * hd:])
    out = torch.empty(m, heads, hd, device="cuda")
    q.qmv_attn_decode(after, m, heads, yq, hd ** -0.5, out, per * page,
                      workspace=workspace(q.qmv_attn_decode_workspace(after, m, heads, per * page)))
    want_k, tol_k = sref.rope(y[:, w:w + kv * hd].reshape(m, kv, hd), wk, pos, freq, hd, "halves", eps)
    close(host(yk).reshape(want_k.shape), want_k, tol_k, "keys at their positions")
    c.pool[:], c.seq_len[:], c.table[:] = d.pool(), keep + m, host(dst)
    # the kept keys as they were turned, the new ones behind them
    for hh in range(kv):
        K, V, _ = c.rows(0, hh, keep + m)
        old = sref.rope(x[:, w:w + kv * hd].reshape(n, kv, hd), wk, np.arange(n), freq, hd, "halves", eps)[0][:, hh]
        rows = np.concatenate([old[host(kept)[0, hh]], want_k[:, hh]])
        # f16: half a step relative, or of its smallest; 4 bits: a step and 8 2^-8 of one (1% more: f32), of an eighth
        # of the block's largest, which the scale's rounding changes by 2^-8 relative
        bound = (np.abs(rows) * (2.0 ** -11 + 1e-4) + 2.0 ** -25 if t == "f16" else
                 np.repeat(np.abs(rows).reshape(keep + m, -1, 32).max(-1), 32, axis=-1) / 8 * (1 + 2.0 ** -8) * (1 + 8.1 * 2.0 ** -8))
        close(K.astype(np.float32), rows, bound, "kept and new keys")
    want, tol, _, _ = ref.attention(c, [0, m], host(yq).reshape(m, heads, hd), hd ** -0.5, per * page)
    close(host(out), want, tol, "attention after an eviction")


def test_two_streams_at_once():
    """Independent caches on two streams, calls interleaved: each as if alone."""
    rng = np.random.default_rng(10)
    kv, hd, page, heads = 2, 128, 32, 8
    h, *_ = make_rope(hd, hd, "halves", True, rng)
    outs, streams, keepers = [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    sets = []
    for i in range(2):
        c, _ = make4(kv, hd, page, [500 - 100 * i, 77], 50 + i)
        x = dev(rng.standard_normal((2, (heads + 2 * kv) * hd), dtype=np.float32))
        sets.append((c, x))

    def run(c, x):
        d = Dev(c)
        qo, out = torch.empty(2, heads * hd, device="cuda"), torch.empty(2, heads * hd, device="cuda")
        ws = workspace(q.qmv_attn_decode_workspace(d.h, 1, heads, c.cap))
        torch.cuda.synchronize()
        return d, qo, out, ws

    def calls(d, qo, out, ws, x, stream):
        q.qmv_kv_append_rope(d.h, h, 2, heads, x[:, :heads * hd], qo, x[:, heads * hd:(heads + kv) * hd], x[:, (heads + kv) * hd:],
                             stream=stream)
        q.qmv_attn_decode(d.h, 1, heads, qo, hd ** -0.5, out, d.c.cap, workspace=ws, stream=stream)

    both = [run(c, x) for c, x in sets]
    for _ in range(3):
        for (d, qo, out, ws), (c, x), s in zip(both, sets, streams):
            calls(d, qo, out, ws, x, s)
    torch.cuda.synchronize()
    for (d, qo, out, ws), (c, x) in zip(both, sets):
        e, qo1, out1, ws1 = run(c, x)
        calls(e, qo1, out1, ws1, x, None)
        torch.cuda.synchronize()
        assert torch.equal(out, out1) and torch.equal(d.pages, e.pages) and torch.equal(qo, qo1)
