"""CPU checks of the calls around a cache's attention: sizes, refusals (every
status comes from the host, nothing is enqueued), the binding's own checks, and
the 64-bit references that the GPU tests use."""
import os

import numpy as np
import pytest

import gguf_dequant_matvec_amd as q
from tests import attn_ref as ref
from tests import serve_ref as sref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="libqmv.so not built")

A16 = 1 << 20      # fake, 16-byte aligned addresses: never dereferenced
B16 = 2 << 20


def cache(t="q4", kv=2, hd=64, page=16, pages=A16, table=A16, seq_len=A16, n_pages=8, n_seq=2, table_ld=4):
    return q.KvCache(t, kv, hd, page, pages, table, seq_len, n_pages=n_pages, n_seq=n_seq, table_ld=table_ld)


def rope(freq=A16, rot=64, pairs="halves", q_norm=A16, k_norm=A16, eps=1e-5):
    return q.QkRope(freq, rot, pairs, q_norm, k_norm, eps)


def append(c, n=2, k=A16, v=A16, **kw):
    return q.qmv_kv_append(c, n, k, v, stream=0, **kw)


def read(c, n=2, k=A16, v=A16, **kw):
    return q.qmv_kv_read(c, n, k, v, stream=0, **kw)


def append_rope(c, r=None, n=2, heads=4, x=A16, y=B16, k=A16, v=A16, **kw):
    return q.qmv_kv_append_rope(c, r or rope(rot=c.head_dim if c.head_dim in (64, 96, 128, 256) else 64), n, heads, x, y,
                                k, v, stream=0, **kw)


def norm_rope(r=None, hd=64, n=2, pos=A16, heads=4, x=A16, y=B16, kv=2, k=A16, ko=B16, **kw):
    return q.qmv_qk_norm_rope(r or rope(), hd, n, pos, heads, x, y, kv, k, ko, stream=0, **kw)


def reserve(c, add=A16, free=A16, count=A16, n=8, granted=A16, start=A16, pos=A16, slot=A16):
    return q.qmv_kv_reserve(c, add, free, count, n, granted, start, pos, slot, stream=0)


def release(c, new_len=A16, free=A16, count=A16):
    return q.qmv_kv_release(c, new_len, free, count, stream=0)


CALLS = [append, read, append_rope, reserve, release]


def status_of(fn, *args, **kw):
    with pytest.raises(q.QmvError) as e:
        fn(*args, **kw)
    return e.value.status_name


def test_page_bytes():
    assert q.qmv_kv_page_bytes("q4", 8, 128, 64) == 8 * 2 * 64 * (64 + 8)
    assert q.qmv_kv_page_bytes("q4", 3, 96, 16) == 3 * 2 * 16 * (48 + 6)
    for hd in (64, 96, 128, 256):
        for page in (16, 4096):
            assert q.qmv_kv_page_bytes("q4", 1, hd, page) % 16 == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("t", ["f16", "q4"])
def test_cache_refusals(call, t):
    for kw in (dict(kv=0), dict(hd=80), dict(page=8), dict(page=24), dict(n_pages=0), dict(n_pages=1 << 31),
               dict(n_seq=0), dict(n_seq=65536), dict(table_ld=0), dict(table_ld=(1 << 26) + 1)):
        assert status_of(call, cache(t=t, **kw)) == "QMV_ESHAPE", kw
    for bad in (2, 20, 103, 105):
        assert status_of(call, cache(t=bad)) == "QMV_EINVAL"
    for kw in (dict(pages=0), dict(table=0), dict(seq_len=0)):
        assert status_of(call, cache(t=t, **kw)) == "QMV_EINVAL", kw
    for kw in (dict(pages=A16 + 8), dict(table=A16 + 2), dict(seq_len=A16 + 1)):
        assert status_of(call, cache(t=t, **kw)) == "QMV_EALIGN", kw


@pytest.mark.parametrize("call", [read, append_rope])
def test_row_refusals(call):
    c = cache()
    for kw, want in ((dict(n=0), "QMV_ESHAPE"), (dict(n=3), "QMV_ESHAPE"), (dict(n=q.MAX_KV_ROWS + 1, start=A16), "QMV_ESHAPE"),
                     (dict(ldk=127), "QMV_ESHAPE"), (dict(ldv=127), "QMV_ESHAPE"), (dict(ldk=(1 << 40) + 1), "QMV_ESHAPE"),
                     (dict(k=0), "QMV_EINVAL"), (dict(v=0), "QMV_EINVAL"), (dict(k=A16 + 2), "QMV_EALIGN"),
                     (dict(v=A16 + 1), "QMV_EALIGN"), (dict(n=3, start=A16 + 2), "QMV_EALIGN")):
        assert status_of(call, c, **kw) == want, kw


@pytest.mark.parametrize("call", [norm_rope, lambda r=None, **kw: append_rope(cache(), r, **kw)])
def test_rope_refusals(call):
    for kw, want in ((dict(rot=-8), "QMV_ESHAPE"), (dict(rot=72), "QMV_ESHAPE"), (dict(rot=12), "QMV_ESHAPE"),
                     (dict(pairs=2), "QMV_EINVAL"), (dict(pairs=-1), "QMV_EINVAL"), (dict(eps=-1e-9), "QMV_EINVAL"),
                     (dict(eps=float("nan")), "QMV_EINVAL"), (dict(eps=float("inf")), "QMV_EINVAL"),
                     (dict(freq=0), "QMV_EINVAL"), (dict(freq=A16 + 4), "QMV_EALIGN"), (dict(q_norm=A16 + 2), "QMV_EALIGN"),
                     (dict(k_norm=A16 + 1), "QMV_EALIGN")):
        assert status_of(call, rope(**kw)) == want, kw
    for kw, want in ((dict(n=0), "QMV_ESHAPE"), (dict(heads=-1), "QMV_ESHAPE"), (dict(heads=32768), "QMV_ESHAPE"),
                     (dict(ldq=255), "QMV_ESHAPE"), (dict(ldqo=255), "QMV_ESHAPE"), (dict(x=0), "QMV_EINVAL"),
                     (dict(y=0), "QMV_EINVAL"), (dict(x=A16 + 2), "QMV_EALIGN"), (dict(y=B16 + 1), "QMV_EALIGN"),
                     (dict(x=A16, y=A16, ldq=256, ldqo=260), "QMV_EINVAL")):
        assert status_of(call, **kw) == want, kw


def test_norm_rope_refusals():
    assert status_of(norm_rope, hd=80) == "QMV_ESHAPE"
    assert status_of(norm_rope, n=q.MAX_KV_ROWS + 1) == "QMV_ESHAPE"
    assert status_of(norm_rope, heads=0, kv=0) == "QMV_ESHAPE"
    assert status_of(norm_rope, kv=32768) == "QMV_ESHAPE"
    assert status_of(norm_rope, pos=0) == "QMV_EINVAL"
    assert status_of(norm_rope, pos=A16 + 2) == "QMV_EALIGN"
    assert status_of(norm_rope, ko=0) == "QMV_EINVAL"
    assert status_of(norm_rope, ldko=100) == "QMV_ESHAPE"
    assert status_of(append_rope, cache(), heads=0) == "QMV_ESHAPE"
    assert status_of(append_rope, cache(kv=40000), heads=30000, ldk=1 << 30, ldv=1 << 30) == "QMV_ESHAPE"


def test_pages_refusals():
    c = cache()
    for kw, want in ((dict(n=0), "QMV_ESHAPE"), (dict(n=q.MAX_KV_ROWS + 1), "QMV_ESHAPE"), (dict(add=0), "QMV_EINVAL"),
                     (dict(free=0), "QMV_EINVAL"), (dict(count=0), "QMV_EINVAL"), (dict(granted=0), "QMV_EINVAL"),
                     (dict(start=0), "QMV_EINVAL"), (dict(add=A16 + 2), "QMV_EALIGN"), (dict(pos=A16 + 1), "QMV_EALIGN"),
                     (dict(slot=A16 + 4), "QMV_EALIGN"), (dict(start=A16 + 3), "QMV_EALIGN")):
        assert status_of(reserve, c, **kw) == want, kw
    for kw, want in ((dict(new_len=0), "QMV_EINVAL"), (dict(free=0), "QMV_EINVAL"), (dict(count=0), "QMV_EINVAL"),
                     (dict(new_len=A16 + 2), "QMV_EALIGN"), (dict(free=A16 + 1), "QMV_EALIGN")):
        assert status_of(release, c, **kw) == want, kw
    # more table entries than the sums of pages count (n_seq table_ld above 2^30; then the other checks go on)
    assert status_of(release, cache(n_seq=17, table_ld=1 << 26)) == "QMV_ESHAPE"
    assert status_of(release, cache(n_seq=16, table_ld=1 << 26), new_len=0) == "QMV_EINVAL"


def test_binding_checks():
    """Tensors of the wrong type, size or place are refused before the call."""
    c = cache()
    f = torch.zeros
    with pytest.raises(ValueError):
        q.QkRope(f(32), 64)                                          # float32 frequencies
    with pytest.raises(ValueError):
        q.QkRope(f(31, dtype=torch.float64), 64)
    with pytest.raises(ValueError):
        q.QkRope(f(32, dtype=torch.float64), 64)                     # on the host
    with pytest.raises(ValueError):
        q.QkRope(A16, 64, q_norm=f(64, dtype=torch.float16))
    with pytest.raises(KeyError):
        q.QkRope(A16, 64, "thirds")
    with pytest.raises(AttributeError):
        rope().eps = 1.0
    with pytest.raises(ValueError):
        norm_rope(pos=f(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        norm_rope(pos=f(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        norm_rope(x=f(2, 255))
    with pytest.raises(ValueError):
        norm_rope(y=f(1, 256))
    with pytest.raises(ValueError):
        append_rope(c, k=f(2, 128, dtype=torch.float64))
    with pytest.raises(ValueError):
        read(c, k=f(2, 127))
    with pytest.raises(ValueError):
        reserve(c, add=f(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        reserve(c, free=f(7, dtype=torch.int32))
    with pytest.raises(ValueError):
        reserve(c, slot=f(8, dtype=torch.int32))
    with pytest.raises(ValueError):
        reserve(c, start=f(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        release(c, new_len=f(2, dtype=torch.int64))


@pytest.mark.parametrize("r", [q.QkRope(None, 0), q.QkRope(0, 0, "adjacent")])
def test_rows_beside_a_rotation_without_tensors(r):
    """Neither frequencies nor norms: the rows' own tensors say which GPU the call is for, and that they are
    on one (a kernel that got host memory would fault)."""
    f, n = torch.zeros, 2
    rows = dict(pos=f(n, dtype=torch.int32), n_heads=1, q=f(n, 64), q_out=f(n, 64))
    for kw in (rows, dict(rows, pos=A16), dict(rows, pos=A16, q=A16),
               dict(pos=A16, n_kv_heads=1, k=f(n, 64), k_out=B16), dict(pos=A16, n_kv_heads=1, k=A16, k_out=f(n, 64))):
        with pytest.raises(ValueError, match="not on a GPU"):
            q.qmv_qk_norm_rope(r, 64, n, **kw)
    # addresses alone are taken as they are
    assert status_of(q.qmv_qk_norm_rope, r, 64, n, 0, 1, A16, B16, stream=0) == "QMV_EINVAL"


def test_attention_units_are_built_with_the_machine_verifier():
    """The compiler once made an attention kernel that read registers which nothing had written; built with
    its own verifier, such a unit ends the build."""
    from gguf_dequant_matvec_amd import build
    flags = {os.path.basename(src): extra for src, _, extra in build.units()}
    for unit in ("qmv_attn_decode.hip", "qmv_attn_prefill.hip"):
        at = flags[unit].index("-verify-machineinstrs")
        assert flags[unit][at - 1] == "-mllvm"


# ---- the references ---------------------------------------------------------

def test_encode4_is_near():
    """A value is within half a step of what it was, the largest within its scale's rounding (a bf16 half
    step, 2^-8 relative).  At the clamped end |x| <= 8 |d| / (1 - 2^-8) and the code 7 |d|: a step, and 8 2^-8
    of one (and 1% of that)."""
    x = np.random.default_rng(1).standard_normal((500, 32)).astype(np.float32)
    u, d = sref.encode4(x)
    f = d.astype(np.float64)[:, None]
    got = (u.astype(np.float64) - 8) * f
    step = np.abs(f)
    assert np.all(np.abs(got - x) <= step * (1 + 8.1 * 2.0 ** -8))
    clamped = (u == 15) | (u == 0)
    assert np.all(np.abs(got - x)[~clamped] <= (step / 2 * (1 + 1e-6) + 1e-9).repeat(32, 1)[~clamped])
    i = np.abs(x).argmax(1)
    assert np.all(u[np.arange(500), i] == 0)             # the largest has the code -8
    assert np.all(np.abs(got - x)[np.arange(500), i] <= 2.0 ** -8 * np.abs(x).max(1))


def test_encode4_corners():
    z = np.zeros(32, np.float32)
    u, d = sref.encode4(z)
    assert d == 0 and np.all(u == 8)
    x = z.copy()
    x[3], x[7] = 2.0, -2.0                               # both signs: the positive one has -8
    u, d = sref.encode4(x)
    assert d == np.float16(-0.25) and u[3] == 0 and u[7] == 15
    x = z.copy()
    x[0], x[1] = np.inf, 1.0
    u, d = sref.encode4(x)
    assert d == np.float16(-2720) and u[0] == 0 and u[1] == 8
    x[2] = np.nan
    u, d = sref.encode4(x)
    assert np.isnan(d)
    x = z.copy()
    x[0] = 1e-9                                          # below half of f16's smallest step
    u, d = sref.encode4(x)
    assert d == 0 and np.all(u == 8)
    # 24 d and every (u - 8) d are f16 values: what the readers rely on
    for bits in range(1, 0x7C00):
        v = np.uint16(bits).view(np.float16)
        b = ref.from_bf16(ref.round_bf16(np.float32(v)))
        if b != np.float32(v) or v > 2720:
            continue
        m = np.float64(v) * np.arange(1, 9)
        assert np.array_equal(m.astype(np.float16).astype(np.float64), m)
        assert np.float64(np.float16(24 * np.float64(v))) == 24 * np.float64(v)


def test_place_is_its_own_inverse():
    assert np.array_equal(sref.PLACE[sref.PLACE], np.arange(16))


def test_rope_reference_turns():
    """A rotation keeps every pair's length, and two of them add up."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    freq = 10000.0 ** (-2 * np.arange(16) / 32)
    for pairs in ("halves", "adjacent"):
        y, _ = sref.rope(x, None, np.array([0, 5, 999]), freq, 32, pairs, 0)
        assert np.allclose((y ** 2).sum(-1), (x.astype(np.float64) ** 2).sum(-1), rtol=1e-12)
        assert np.array_equal(y[..., 32:], x[..., 32:].astype(np.float64)) and np.array_equal(y[0], x[0].astype(np.float64))
        once, _ = sref.rope(x, None, np.array([7] * 3), freq, 32, pairs, 0)
        both, _ = sref.rope(x, None, np.array([14] * 3), freq, 32, pairs, 0)
        # (the second turn of an f64 row, by the same code)
        i = np.arange(16)
        a, b = (i, i + 16) if pairs == "halves" else (2 * i, 2 * i + 1)
        t = 7 * freq
        assert np.allclose(once[..., a] * np.cos(t) - once[..., b] * np.sin(t), both[..., a], rtol=0, atol=1e-12)


def test_pages_reference_gives_back_what_it_took():
    rng = np.random.default_rng(3)
    table = np.full((5, 8), -1, np.int32)
    p = sref.Pages(table, [0] * 5, rng.permutation(40), 40, 16, 40)
    p.reserve([100, 0, 17, 16, 1], 200)
    taken = p.table.copy()
    lens, free, count = p.seq_len.copy(), p.free.copy(), p.count
    p.release([0] * 5)
    assert p.count == 40 and np.all(p.table == -1) and sorted(p.free) == list(range(40))
    p.reserve(lens, 200)
    assert np.array_equal(p.table, taken) and p.count == count and np.array_equal(p.free[:count], free[:count])
