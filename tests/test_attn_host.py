"""CPU checks of the cache and attention entry points: sizes, workspaces and
refusals (every status comes from the host, nothing is enqueued), the binding's
own checks, and the 64-bit reference the GPU tests use."""
import os

import numpy as np
import pytest

import gguf_dequant_matvec_amd as q
from tests import attn_ref as ref

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="libqmv.so not built")

A16 = 1 << 20      # fake, 16-byte aligned addresses: never dereferenced


def cache(t="f16", kv=2, hd=64, page=16, pages=A16, table=A16, seq_len=A16, n_pages=8, n_seq=2, table_ld=4):
    return q.KvCache(t, kv, hd, page, pages, table, seq_len, n_pages=n_pages, n_seq=n_seq, table_ld=table_ld)


def append(c, n=2, k=A16, v=A16, **kw):
    return q.qmv_kv_append(c, n, k, v, stream=0, **kw)


def decode(c, n=1, heads=4, qp=A16, scale=0.125, out=A16, max_len=64, **kw):
    kw.setdefault("workspace", A16)
    kw.setdefault("ws_bytes", 1 << 40)
    return q.qmv_attn_decode(c, n, heads, qp, scale, out, max_len, stream=0, **kw)


def prefill(c, n=20, heads=4, qp=A16, scale=0.125, out=A16, max_len=64, **kw):
    kw.setdefault("workspace", A16)
    kw.setdefault("ws_bytes", 1 << 40)
    return q.qmv_attn_prefill(c, n, heads, qp, scale, out, max_len, stream=0, **kw)


def evict(c, dst=A16, keep=32, first=4, recent=8, acc=A16, kept=A16, acc_out=A16, len_out=A16, dst_ld=2, ld_acc=64,
          ld_out=32):
    return q.qmv_kv_evict(c, dst, keep, first, recent, acc, kept, acc_out, len_out, dst_ld=dst_ld, ld_acc=ld_acc,
                          ld_out=ld_out, stream=0)


CALLS = [append, decode, prefill, evict]


def status_of(fn, *args, **kw):
    with pytest.raises(q.QmvError) as e:
        fn(*args, **kw)
    return e.value.status_name


def test_page_bytes():
    assert q.qmv_kv_page_bytes("f16", 8, 128, 64) == 8 * 2 * 64 * 128 * 2
    assert q.qmv_kv_page_bytes("bf16", 3, 64, 16) == 3 * 2 * 16 * 64 * 2
    assert q.qmv_kv_page_bytes("i8", 2, 96, 32) == 2 * (2 * 32 * 96 + 8 * 32)
    for bad in [("f16", 0, 64, 16), ("f16", 1, 80, 16), ("f16", 1, 64, 8), ("f16", 1, 64, 48), ("f16", 1, 64, 8192),
                (0, 1, 64, 16), (8, 1, 64, 16), ("f16", 65536, 64, 16)]:
        assert q.qmv_kv_page_bytes(*bad) == 0, bad


@pytest.mark.parametrize("call", CALLS)
def test_cache_refusals(call):
    """Every call checks the cache it is given."""
    shape = [dict(kv=0), dict(hd=80), dict(hd=0), dict(page=8), dict(page=24), dict(n_pages=0), dict(n_pages=1 << 31),
             dict(n_seq=0), dict(n_seq=65536), dict(table_ld=0), dict(table_ld=(1 << 26) + 1)]
    for kw in shape:
        assert status_of(call, cache(**kw)) == "QMV_ESHAPE", kw
    assert status_of(call, cache(t=2)) == "QMV_EINVAL"
    for kw in (dict(pages=0), dict(table=0), dict(seq_len=0)):
        assert status_of(call, cache(**kw)) == "QMV_EINVAL", kw
    for kw in (dict(pages=A16 + 8), dict(table=A16 + 2), dict(seq_len=A16 + 1)):
        assert status_of(call, cache(**kw)) == "QMV_EALIGN", kw


def test_append_refusals():
    c = cache()
    assert status_of(append, c, n=0) == "QMV_ESHAPE"
    assert status_of(append, c, n=3) == "QMV_ESHAPE"           # not a multiple of n_seq
    assert status_of(append, c, n=q.MAX_KV_ROWS + 1, start=A16) == "QMV_ESHAPE"
    assert status_of(append, c, ldk=127) == "QMV_ESHAPE"
    assert status_of(append, c, ldv=127) == "QMV_ESHAPE"
    assert status_of(append, c, k=0) == "QMV_EINVAL"
    assert status_of(append, c, v=0) == "QMV_EINVAL"
    assert status_of(append, c, k=A16 + 2) == "QMV_EALIGN"
    assert status_of(append, c, v=A16 + 1) == "QMV_EALIGN"
    assert status_of(append, c, n=3, start=A16 + 2) == "QMV_EALIGN"


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_refusals(call):
    c = cache()
    assert status_of(call, c, heads=3) == "QMV_ESHAPE"          # not a multiple of n_kv_heads
    assert status_of(call, c, heads=0) == "QMV_ESHAPE"
    assert status_of(call, c, max_len=0) == "QMV_ESHAPE"
    assert status_of(call, c, max_len=65) == "QMV_ESHAPE"       # more than a table row addresses
    assert status_of(call, c, window=-1) == "QMV_ESHAPE"
    assert status_of(call, c, sinks=-1) == "QMV_ESHAPE"
    assert status_of(call, c, ldq=255) == "QMV_ESHAPE"
    assert status_of(call, c, qp=0) == "QMV_EINVAL"
    assert status_of(call, c, out=0) == "QMV_EINVAL"
    assert status_of(call, c, qp=A16 + 2) == "QMV_EALIGN"
    assert status_of(call, c, out=A16 + 2) == "QMV_EALIGN"
    assert status_of(call, c, n=0) == "QMV_ESHAPE"


def test_decode_refusals():
    c = cache()
    assert status_of(decode, c, n=q.MAX_ATTN_N + 1) == "QMV_ESHAPE"
    assert status_of(decode, c, acc=A16, ld_acc=63) == "QMV_ESHAPE"
    assert status_of(decode, c, acc=A16 + 2, ld_acc=64) == "QMV_EALIGN"
    assert status_of(decode, cache(n_seq=65535), n=16, heads=4096) == "QMV_ESHAPE"
    assert status_of(decode, cache(n_seq=65535), n=16, heads=32, acc=A16, ld_acc=64) == "QMV_ESHAPE"
    # the weights need a workspace; so does a long cache, which is split
    need = q.qmv_attn_decode_workspace(c, 1, 4, 64, 0, 0, True)
    assert need > 2 * 4 * 64 * 4                                # the logits, and each row's sums
    assert status_of(decode, c, acc=A16, ld_acc=64, workspace=0, ws_bytes=0) == "QMV_EWORKSPACE"
    assert status_of(decode, c, acc=A16, ld_acc=64, ws_bytes=need - 1) == "QMV_EWORKSPACE"
    assert status_of(decode, c, acc=A16, ld_acc=64, workspace=A16 + 4, ws_bytes=need) == "QMV_EALIGN"
    big = cache(kv=8, hd=128, page=64, n_seq=1, table_ld=2048)
    need = q.qmv_attn_decode_workspace(big, 1, 32, 131072)
    assert need > 0
    assert status_of(decode, big, heads=32, max_len=131072, ws_bytes=need - 1) == "QMV_EWORKSPACE"
    assert q.qmv_attn_decode_workspace(c, 1, 4, 64) == 0         # a short one needs none
    assert q.qmv_attn_decode_workspace(c, 17, 4, 64, 0, 0, True) == 0
    assert q.qmv_attn_decode_workspace(cache(hd=80), 1, 4, 64, 0, 0, True) == 0


def test_prefill_refusals():
    c = cache()
    assert status_of(prefill, c, n=21) == "QMV_ESHAPE"
    assert status_of(prefill, c, n=21, start=A16 + 1) == "QMV_EALIGN"
    assert status_of(prefill, c, n=q.MAX_KV_ROWS + 1, start=A16) == "QMV_ESHAPE"
    assert status_of(prefill, c, n=1 << 23, start=A16) == "QMV_ESHAPE"      # 2^17 row tiles
    big = cache(kv=1, hd=128, page=64, n_seq=1, table_ld=2048)
    need = q.qmv_attn_prefill_workspace(big, 40, 4, 131072)
    assert need > 0                                             # few rows, a long cache: split
    assert status_of(prefill, big, n=40, max_len=131072, ws_bytes=need - 1) == "QMV_EWORKSPACE"
    assert status_of(prefill, big, n=40, max_len=131072, workspace=A16 + 8) == "QMV_EALIGN"
    assert q.qmv_attn_prefill_workspace(cache(kv=8, hd=128, page=64, n_seq=1, table_ld=64), 4096, 32, 4096) == 0
    assert q.qmv_attn_prefill_workspace(big, 0, 4, 131072) == 0


def test_evict_refusals():
    c = cache()
    for kw in (dict(dst=0), dict(acc=0), dict(kept=0), dict(acc_out=0), dict(len_out=0)):
        assert status_of(evict, c, **kw) == "QMV_EINVAL", kw
    for kw in (dict(keep=0), dict(keep=33), dict(dst_ld=0), dict(first=-1), dict(recent=-1), dict(first=20, recent=13),
               dict(ld_acc=0), dict(ld_out=31)):
        assert status_of(evict, c, **kw) == "QMV_ESHAPE", kw
    for kw in (dict(dst=A16 + 2), dict(acc=A16 + 2), dict(kept=A16 + 1), dict(acc_out=A16 + 2), dict(len_out=A16 + 2)):
        assert status_of(evict, c, **kw) == "QMV_EALIGN", kw


def test_evict_largest_keep():
    """The most positions whose workgroups one launch can have."""
    c = cache(table_ld=1 << 26)
    assert status_of(evict, c, keep=(1 << 30) - 63, dst_ld=1 << 26, ld_out=1 << 30) == "QMV_ESHAPE"


def test_binding_refusals():
    """Tensors whose type, shape or strides the C call cannot see."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    pages, table, lens = z(8 * 8192, dtype=torch.uint8), z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    c = q.KvCache("f16", 2, 64, 16, pages, table, lens)
    assert (c.n_pages, c.n_seq, c.table_ld) == (8, 2, 4)
    for bad in (dict(table=table.long()), dict(table=table[:, ::2]), dict(table=table[0]), dict(table=z(2, 8, dtype=torch.int32)[:, :4]),
                dict(seq_len=lens[:1]), dict(seq_len=lens.float()), dict(pages=pages[::2])):
        kw = dict(pages=pages, table=table, seq_len=lens, **{})
        kw.update(bad)
        with pytest.raises(ValueError):
            q.KvCache("f16", 2, 64, 16, kw["pages"], kw["table"], kw["seq_len"])
    with pytest.raises(ValueError):
        q.KvCache("f16", 2, 64, 16, pages, table, lens, n_pages=9)
    k = z(2, 128)
    for bad in (k.half(), z(2, 256)[:, ::2], z(1, 128), z(2, 64), k[0]):
        with pytest.raises(ValueError):
            q.qmv_kv_append(c, 2, bad, k, stream=0)
    with pytest.raises(ValueError):
        q.qmv_kv_append(c, 2, k, k, start=z(2, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError):
        q.qmv_attn_decode(c, 1, 4, z(2, 256), 0.1, z(2, 128), 64, stream=0)
    with pytest.raises(ValueError):
        q.qmv_attn_decode(c, 1, 4, z(2, 256), 0.1, z(2, 256), 64, acc=z(2, 4, 64), stream=0)
    with pytest.raises(ValueError):
        q.qmv_attn_prefill(c, 4, 4, z(4, 256), 0.1, z(4, 256).double(), 64, stream=0)
    with pytest.raises(ValueError):
        q.qmv_kv_evict(c, table, 8, 0, 0, z(2, 2, 64), z(2, 2, 8), z(2, 2, 8), lens, stream=0)


def test_binding_row_widths():
    """Rows that are not exactly as wide as the call takes them: a kernel would
    read past a single short row, and the neighbouring columns of a wider matrix."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    pages, table, lens = z(8 * 8192, dtype=torch.uint8), z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    c = q.KvCache("f16", 2, 64, 16, pages, table, lens)
    c1 = q.KvCache("f16", 2, 64, 16, pages, table, lens, n_seq=1)
    wide = z(4, 512)
    for a in (z(2, 100), z(2, 65), z(2, 127), z(2, 129), z(2, 192), z(2, 1, 100), z(2, 2, 63), z(2, 3, 43), wide[:, :100],
              wide[:, :127], wide[:, :200], z(2, 128, 2)[:, :, 0], z(2, 0), z(2, 0, 128), z(2, 1, 2, 33)):
        for k, v in ((a, z(2, 128)), (z(2, 128), a)):
            with pytest.raises(ValueError, match="rows of"):
                q.qmv_kv_append(c, 2, k, v, stream=0)
    for a in (z(1, 100), z(1, 65), z(1, 129), z(1, 2, 33)):      # one row: the single-user step
        with pytest.raises(ValueError, match="rows of"):
            q.qmv_kv_append(c1, 1, a, z(1, 128), stream=0)
        with pytest.raises(ValueError, match="rows of"):
            q.qmv_attn_decode(c1, 1, 2, a, 0.1, z(1, 128), 64, stream=0)
        with pytest.raises(ValueError, match="rows of"):
            q.qmv_attn_prefill(c1, 1, 2, a, 0.1, z(1, 128), 64, stream=0)
    # what is a row: any shape of the right size, in any wider matrix
    for a in (z(2, 128), z(2, 2, 64), z(2, 1, 128), z(2, 2, 1, 64), wide[:, 100:228], wide[1:, :128], z(2, 2, 2, 32)):
        with pytest.raises(ValueError, match="not on a GPU"):
            q.qmv_kv_append(c, 2, a, a, stream=0)


def test_binding_workspaces():
    """A workspace is as many bytes as its tensor spans, in one piece."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    c = q.KvCache("f16", 2, 64, 16, z(8 * 8192, dtype=torch.uint8), z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32))
    x = z(2, 256)
    for ws, kw in ((z(1).expand(1 << 20), {}), (z(64, 64)[:, :8], {}), (z(1 << 12)[::2], {}),
                   (z(100), dict(ws_bytes=401)), (z(100)[50:], dict(ws_bytes=204))):
        with pytest.raises(ValueError, match="workspace"):
            q.qmv_attn_decode(c, 1, 4, x, 0.1, z(2, 256), 64, workspace=ws, stream=0, **kw)
        with pytest.raises(ValueError, match="workspace"):
            q.qmv_attn_prefill(c, 2, 4, x, 0.1, z(2, 256), 64, workspace=ws, stream=0, **kw)
    for ws, kw in ((z(64, 64), {}), (z(100), dict(ws_bytes=400)), (z(100)[50:], dict(ws_bytes=200)), (None, {})):
        with pytest.raises(ValueError, match="not on a GPU"):
            q.qmv_attn_decode(c, 1, 4, x, 0.1, z(2, 256), 64, workspace=ws, stream=0, **kw)


def test_binding_explicit_strides():
    """Strides given beside a tensor: the rows must lie in its storage, and a
    stride that the tensor's own shape says must be that."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    pages, table, lens = z(8 * 8192, dtype=torch.uint8), z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    c = q.KvCache("f16", 2, 64, 16, pages, table, lens)
    k = z(2, 128)
    flat = z(1000)
    for a, ld in ((flat, 873), (flat[1:], 872), (flat[900:], 128), (z(1, 100), 128), (z(4), 128), (flat.half(), 128)):
        for kw in (dict(k=a, v=k, ldk=ld), dict(k=k, v=a, ldv=ld)):
            with pytest.raises(ValueError, match="k must|v must|k holds|v holds"):
                q.qmv_kv_append(c, 2, stream=0, **kw)
    for a, ld in ((flat, 745), (z(1, 300), 256), (flat[600:], 256)):
        with pytest.raises(ValueError, match="q holds"):
            q.qmv_attn_decode(c, 1, 4, a, 0.1, z(2, 256), 64, ldq=ld, stream=0)
        with pytest.raises(ValueError, match="q holds"):
            q.qmv_attn_prefill(c, 2, 4, a, 0.1, z(2, 256), 64, ldq=ld, stream=0)
    with pytest.raises(ValueError, match="acc"):
        q.qmv_attn_decode(c, 1, 4, z(2, 256), 0.1, z(2, 256), 64, acc=z(2, 2, 64), ld_acc=80, stream=0)
    acc, kept, acc_out, n = z(2, 2, 64), z(2, 2, 8, dtype=torch.int32), z(2, 2, 8), z(2, dtype=torch.int32)
    for kw in (dict(dst_ld=5), dict(ld_acc=65), dict(ld_out=9)):
        with pytest.raises(ValueError, match="dst_table|acc"):
            q.qmv_kv_evict(c, table, 8, 0, 0, acc, kept, acc_out, n, stream=0, **kw)
    # what fits
    for a, ld in ((flat, 872), (flat, 128), (flat[744:], 128), (z(3, 512)[1:, 100:], 512)):
        with pytest.raises(ValueError, match="not on a GPU"):
            q.qmv_kv_append(c, 2, a, a, ldk=ld, ldv=ld, stream=0)
    with pytest.raises(ValueError, match="not on a GPU"):
        q.qmv_kv_evict(c, table, 8, 0, 0, acc, kept, acc_out, n, dst_ld=4, ld_acc=64, ld_out=8, stream=0)


def test_cache_of_host_tensors():
    """Calls over tensors that are not on a GPU end on the host; a cache's
    tensors cannot be exchanged behind its addresses."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    pages, table, lens = z(8 * 8192, dtype=torch.uint8), z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    c = q.KvCache("f16", 2, 64, 16, pages, table, lens)
    k, x = z(2, 128), z(2, 256)
    with pytest.raises(ValueError, match="not on a GPU"):
        q.qmv_kv_append(c, 2, k, k, stream=0)
    with pytest.raises(ValueError, match="not on a GPU"):
        q.qmv_attn_decode(c, 1, 4, x, 0.1, z(2, 256), 64, stream=0)
    with pytest.raises(ValueError, match="not on a GPU"):
        q.qmv_attn_prefill(c, 2, 4, x, 0.1, z(2, 256), 64, stream=0)
    with pytest.raises(ValueError, match="not on a GPU"):
        q.qmv_kv_evict(c, table, 8, 0, 0, z(2, 2, 64), z(2, 2, 8, dtype=torch.int32), z(2, 2, 8), lens, stream=0)
    for name in ("table", "seq_len", "pages", "n_seq"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


# ---- the reference itself -------------------------------------------------------

def test_reference_by_hand():
    """One head of 64 columns, three positions, by hand: logits 0, ln 2, ln 3."""
    c = ref.Cache("f16", 1, 64, 16, 2, [[1, 0]], [3])
    for p in range(3):
        k, v = np.zeros(64, np.float32), np.zeros(64, np.float32)
        k[0], v[p] = p, p + 1.0
        c.write(0, p, 0, k, v)
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, 0] = 1.0
    out, tol, acc, _ = ref.attention(c, [0, 1], x, np.log(2.0), 3, acc=np.zeros((1, 1, 4)))
    assert np.allclose(acc[0, 0], [1 / 7, 2 / 7, 4 / 7, 0]) and np.allclose(out[0, 0, :4], [1 / 7, 4 / 7, 12 / 7, 0])
    out, _, _, _ = ref.attention(c, [0, 1], x, np.log(2.0), 3, window=1, sinks=1)
    assert np.allclose(out[0, 0, :4], [0.2, 0, 12 / 5, 0])
    out, _, _, _ = ref.attention(c, [0, 4], np.repeat(x, 4, 0), 1.0, 3)     # more tokens than positions
    assert np.all(out[0] == 0) and out[1, 0, 0] == 1.0
    # the layout: page 1 holds K row 2 at slot 2 and V column 2 at [0][2][2]
    raw = c.pool[1, 0].view(np.float16)
    assert raw[2 * 64] == 2.0 and raw[16 * 64 + 2 * 16 + 2] == 3.0


def test_reference_i8_and_bf16_rows():
    x = np.array([0.0, 127.0, -63.5, 0.49] + [0.0] * 60, np.float32)
    code, d = ref.encode_row("i8", x)
    assert d == 1.0 and list(code[:4]) == [0, 127, -64, 0]
    code, d = ref.encode_row("i8", np.zeros(64, np.float32))
    assert d == 0 and not code.any()
    y = np.array([1.0, 1.00390625, 1.01171875, -3.1415927], np.float32)
    assert list(ref.from_bf16(ref.round_bf16(y))) == [1.0, 1.0, 1.015625, -3.140625]


def test_reference_evict():
    c = ref.Cache("i8", 1, 64, 16, 4, [[0]], [6])
    for p in range(6):
        c.write(0, p, 0, np.full(64, p + 1, np.float32), np.full(64, -p - 1, np.float32))
    acc = np.array([[[0, 5, 1, 5, 1, 0, 9, 9]]], np.float32)
    kept, a, n = ref.evict(c, np.array([[2]], np.int32), 4, 1, 1, acc)
    assert list(kept[0, 0]) == [0, 1, 3, 5] and list(a[0, 0]) == [0, 5, 5, 0] and n[0] == 4
    c.table, c.seq_len = np.array([[2]], np.int32), n
    K, V, there = c.rows(0, 0, 4)
    assert np.allclose(K[:, 0], [1, 2, 4, 6]) and np.allclose(V[:, 7], [-1, -2, -4, -6]) and there.all()
