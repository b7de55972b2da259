"""What stands around a layer's attention as measurable cases: a plain form in
torch, the library's calls, and the same results in 64 bits.

A case is one step of one operator:

  pages     a batch's pages kept on the GPU: tokens that a step gives up are
            released with their pages, the next step's are reserved, with the
            first row of each sequence, the rows' positions and their slots
  rope      norms of queries and keys for each head and the rotation of the
            position, in one pass
  append    the same for new tokens, whose keys and values go to a paged cache
  write4    new tokens' keys and values into a cache held in 4 bits, and the
            values that they stand for there
  attend4   attention over a cache held in 4 bits: the last n (1 to 16) tokens
            of each sequence, or whole and chunked prompts

Sizes are the layer shapes of the workloads this repository runs elsewhere:
9 query / 3 key-value heads of 64 (the 576-wide model), 32 / 8 of 64 (hidden
2048) and 32 / 8 of 128 (hidden 4096).

A page of a 4-bit cache holds, for each key-value head, the codes of K
[page][hd/2], those of V [page/16][hd/2][16], then the f16 scales of K
[page][hd/32] and of V [hd/32][page].  A byte has the codes of columns
32 b + c (low) and 32 b + c + 16 (high), c < 16; each four positions of V lie
in the order 0, 2, 1, 3.  A value is scale * (code - 8).
"""
import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
ID_BYTES = {"f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, **kw):
    return dict(kw, name=name) if name else kw


def _pages(name, seqs, page, length, add, ragged, drop):
    """`drop` of the sequences are over: theirs are new prompts of up to `add` tokens, the others
    add the same number for drafted tokens (all of them rejected before)."""
    return _case(name, op="pages", seqs=seqs, page=page, len=length, add=add, ragged=ragged, drop=drop)


def _rope(name, rows, heads, kv, hd, rot, pairs, norm, far):
    return _case(name, op="rope", rows=rows, heads=heads, kv=kv, hd=hd, rot=rot, pairs=pairs, norm=norm, far=far)


def _append(name, t, heads, kv, hd, page, seqs, n, length, pairs, norm, ragged):
    return _case(name, op="append", t=t, heads=heads, kv=kv, hd=hd, rot=hd, page=page, seqs=seqs, n=n, len=length,
                 pairs=pairs, norm=norm, ragged=ragged)


def _write4(name, kv, hd, page, seqs, n, length, ragged):
    return _case(name, op="write4", kv=kv, hd=hd, page=page, seqs=seqs, n=n, len=length, ragged=ragged)


def _attend4(name, call, heads, kv, hd, page, seqs, n, length, window=0, sinks=0, ragged=False):
    return _case(name, op="attend4", call=call, heads=heads, kv=kv, hd=hd, page=page, seqs=seqs, n=n, len=length,
                 window=window, sinks=sinks, ragged=ragged)


def listed():
    return [
        # one decode step of 64 sequences, a token each: pure latency
        _pages("pages_step", 64, 64, 4000, 1, True, 0),
        # 256 sequences check 8 drafted tokens each, after the last ones were all rejected
        _pages("pages_drafts", 256, 16, 6001, 8, True, 0),
        # 24 sequences ended, and new prompts of up to 7001 tokens take their places
        _pages("pages_prompts", 96, 16, 7001, 7001, True, 24),
        # the joined form in a decode step of 16 sequences
        _append("append_step", "f16", 32, 8, 128, 64, 16, 1, 2048, "halves", True, False),
        # ... and for prompts of different lengths, Q, K and V read out of the stacked rows
        _append("append_prompts", "bf16", 32, 8, 128, 64, 4, 2100, 2100, "halves", True, True),
        # queries and keys of a model without such norms, adjacent pairs, half of the columns turned, far positions
        _rope("rope_far", 3001, 32, 8, 64, 32, "adjacent", False, 1000000),
        # prompts into a 4-bit cache
        _write4("write4_prompts", 8, 128, 64, 4, 2100, 2100, True),
        # the smallest model's attention early in a chat: latency
        _attend4("decode4_small", "decode", 9, 3, 64, 16, 1, 1, 301),
        # a serving batch with mixed context lengths: the cache stream
        _attend4("decode4_batch", "decode", 32, 8, 128, 64, 32, 1, 8150, ragged=True),
        # one user with a very long context: split over the length
        _attend4("decode4_long", "decode", 32, 8, 128, 128, 1, 1, 131071),
        # eight drafted tokens checked at once in a sliding window with sinks
        _attend4("verify4_window", "decode", 32, 8, 64, 32, 8, 8, 20011, window=4096, sinks=4),
        # a long prompt of the 4096-wide model, full causal attention
        _attend4("prefill4_long", "prefill", 32, 8, 128, 64, 1, 4096, 4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["pages", "rope", "append", "write4", "attend4", "attend4"])
    heads, kv, hd = rng.choice([(9, 3, 64), (32, 8, 64), (32, 8, 128), (8, 8, 64), (16, 2, 128), (12, 4, 96)])
    page = rng.choice([16, 32, 64, 128])
    pairs, norm = rng.choice(["halves", "adjacent"]), rng.random() < 0.6
    seqs = _log(rng, 1, 32)
    if op == "pages":
        seqs = _log(rng, 1, 300)
        length = _log(rng, 20, 7000)
        drop = rng.choice([0, rng.randint(0, min(seqs, 24))])
        return _pages("", seqs, page, length, _log(rng, 1, length) if drop else rng.randint(1, 16), rng.random() < 0.5,
                      drop)
    if op == "rope":
        rot = rng.choice([hd, hd, hd // 2, 16])
        return _rope("", _log(rng, 1, 3000), heads, kv, hd, rot, pairs, norm, _log(rng, 10, 2000000))
    if op in ("append", "write4"):
        seqs = rng.randint(1, 8)
        length = _log(rng, 17, 1500)
        n = rng.choice([1, _log(rng, 1, length)])
        if op == "write4":
            return _write4("", kv, hd, page, seqs, n, length, rng.random() < 0.5)
        return _append("", rng.choice(["f16", "bf16"]), heads, kv, hd, page, seqs, n, length, pairs, norm,
                       rng.random() < 0.5)
    if rng.random() < 0.6:
        length = _log(rng, 33, min(131071, 200000 // seqs))
        n = rng.choice([1, 1, 1, rng.randint(2, 16)])
        call = "decode"
    else:
        seqs = rng.randint(1, 3)
        length = _log(rng, 20, 4000 // seqs)
        n = rng.choice([length, _log(rng, 17, length)])
        call = "prefill"
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, length), rng.randint(0, 9))])
    return _attend4("", call, heads, kv, hd, page, seqs, n, length, window, sinks, rng.random() < 0.5)


def _lengths(c):
    """Cached positions of each sequence, the new tokens among them."""
    if not c["ragged"]:
        return [c["len"]] * c["seqs"]
    return [max(1, c["len"] - s * c["len"] // (2 * c["seqs"]) - 3 * s) for s in range(c["seqs"])]


def _news(c):
    """New tokens of each sequence: decode takes the same number for all."""
    if c["op"] == "attend4" and c["call"] == "decode":
        return [c["n"]] * c["seqs"]
    return [min(c["n"], length) for length in _lengths(c)]


def _adds(c):
    """pages: positions each sequence keeps, and tokens it adds."""
    keep, add = [], []
    for s, length in enumerate(_lengths(c)):
        over = s % max(1, c["seqs"] // max(1, c["drop"])) == 0 and s // max(1, c["seqs"] // max(1, c["drop"])) < c["drop"]
        keep.append(0 if over else length)
        add.append(min(length, c["add"]) if over else c["add"] if c["drop"] == 0 else 1)
    return keep, add


def _head_bytes(c):
    if c["op"] in ("write4", "attend4"):
        return c["page"] * c["hd"] * 9 // 8
    return 2 * c["page"] * c["hd"] * ID_BYTES[c["t"]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _views4(c, pages):
    """The parts of a 4-bit pool: codes of K and V, scales of K and V, all [n_pages][kv]..."""
    page, hd = c["page"], c["hd"]
    pool = pages.view(-1, c["kv"], _head_bytes(c))
    half, sc = page * hd // 2, page * hd // 16
    k = pool[..., :half].unflatten(-1, (page, hd // 2))
    v = pool[..., half:2 * half].unflatten(-1, (page // 16, hd // 2, 16))
    ks = pool[..., 2 * half:2 * half + sc].view(torch.float16).unflatten(-1, (page, hd // 32))
    vs = pool[..., 2 * half + sc:].view(torch.float16).unflatten(-1, (hd // 32, page))
    return k, v, ks, vs


def _views16(c, pages):
    """K [n_pages][kv][page][hd] and V [n_pages][kv][page/16][hd][16] of a 16-bit pool."""
    pool = pages.view(DTYPE[c["t"]]).view(-1, c["kv"], 2 * c["page"] * c["hd"])
    k, v = pool.split(c["page"] * c["hd"], dim=-1)
    return k.unflatten(-1, (c["page"], c["hd"])), v.unflatten(-1, (c["page"] // 16, c["hd"], 16))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "pages":
        return _prepare_pages(c, g)
    s = {"case": c}
    if c["op"] == "rope":
        n = c["rows"]
        s["pos"] = torch.randint(0, c["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
    else:
        _prepare_cache(c, g, s)
        n = s["tokens"]
    if c["op"] == "attend4":
        s["q"] = 1.5 * torch.randn(n, c["heads"] * c["hd"], generator=g, device="cuda")
        s["out"] = torch.empty(n, c["heads"] * c["hd"], device="cuda")
        return s
    # rows of the stacked QKV product, Q, K and V as column ranges of it
    hq, hk = c.get("heads", 0) * c["hd"], c["kv"] * c["hd"]
    qkv = torch.randn(n, hq + 2 * hk, generator=g, device="cuda")
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if c["op"] == "write4":
        s["k_out"], s["v_out"] = torch.empty(2, n, hk, device="cuda")
        return s
    s["q_out"], s["k_out"] = torch.empty(n, hq, device="cuda"), torch.empty(n, hk, device="cuda")
    norms = 1 + 0.2 * torch.randn(2, c["hd"], generator=g, device="cuda")
    s["q_norm"], s["k_norm"] = (norms[0], norms[1]) if c["norm"] else (None, None)
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    s["freq"] = 500000.0 ** (-2 * i / c["rot"])
    s["eps"] = 1e-5
    return s


def _prepare_pages(c, g):
    keep, add = _adds(c)
    seqs, page = c["seqs"], c["page"]
    held = [-(-(k + a) // page) for k, a in zip(keep, add)]
    per = max(held) + 2
    n_pages = sum(held) + 37
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((seqs, per), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(per, device="cuda")
    mine = at[None, :] < torch.tensor(held, device="cuda")[:, None]
    table[mine] = ids[:sum(held)]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:37] = ids[sum(held):]
    n = sum(add)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    return {"case": c, "table": table, "n_pages": n_pages, "free": free, "count": i32([37]), "rows": n,
            "seq_len": i32([k + a for k, a in zip(keep, add)]), "keep": i32(keep), "add": i32(add),
            "granted": i32([0] * seqs), "start": i32([0] * (seqs + 1)),
            "pos": torch.empty(n, dtype=torch.int32, device="cuda"),
            "slot": torch.empty(n, dtype=torch.int64, device="cuda"),
            # the pool that the table speaks of: neither call looks into it
            "pages": torch.empty(n_pages * 2 * page * 64 * 2, dtype=torch.uint8, device="cuda")}


def _prepare_cache(c, g, s):
    page, seqs = c["page"], c["seqs"]
    lens, news = _lengths(c), _news(c)
    per_seq = -(-c["len"] // page)
    n_pages = seqs * per_seq
    pages = torch.empty(n_pages * c["kv"] * _head_bytes(c), dtype=torch.uint8, device="cuda")
    if c["op"] in ("write4", "attend4"):     # every slot holds something, as pages used before do
        k, v, ks, vs = _views4(c, pages)
        for codes, scale in ((k, ks), (v, vs)):
            codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
            d = 0.15 + 0.15 * torch.rand(scale.shape, generator=g, device="cuda")
            d *= torch.randint(0, 2, d.shape, generator=g, device="cuda") * 2 - 1
            scale.copy_(d.to(torch.bfloat16))
    else:
        pages.view(DTYPE[c["t"]]).copy_(torch.randn(pages.numel() // 2, generator=g, device="cuda"))
    table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(seqs, per_seq)
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    s.update(pages=pages, table=table, lens=lens, news=news, tokens=start[-1],
             seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    s["start_arg"] = s["start"] if len(set(news)) > 1 else None      # None: as many tokens for each sequence


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"pages": _turn_pages, "rope": _rope_rows, "append": _append_rows, "write4": _write_rows,
            "attend4": _attend}[state["case"]["op"]](state)


def _run_own(s):
    import gguf_dequant_matvec_amd as q
    c = s["case"]
    op = c["op"]
    if "ready" not in s:             # what a program keeps: handles of the cache and the rotation, the workspace
        s["ready"] = True
        if op == "pages":
            s["cache"] = q.KvCache("f16", 1, 64, c["page"], s["pages"], s["table"], s["seq_len"])
        elif op != "rope":
            s["cache"] = q.KvCache(c.get("t", "q4"), c["kv"], c["hd"], c["page"], s["pages"], s["table"], s["seq_len"])
        if op in ("rope", "append"):
            s["rope"] = q.QkRope(s["freq"], c["rot"], c["pairs"], s["q_norm"], s["k_norm"], s["eps"])
        if op == "attend4":
            args = (c["heads"], c["len"], c["window"], c["sinks"])
            need = (q.qmv_attn_decode_workspace(s["cache"], c["n"], *args) if c["call"] == "decode" else
                    q.qmv_attn_prefill_workspace(s["cache"], s["tokens"], *args))
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    if op == "pages":
        q.qmv_kv_release(s["cache"], s["keep"], s["free"], s["count"])
        q.qmv_kv_reserve(s["cache"], s["add"], s["free"], s["count"], s["rows"], s["granted"], s["start"],
                         pos=s["pos"], slot=s["slot"])
        return _pages_out(s)
    if op == "rope":
        q.qmv_qk_norm_rope(s["rope"], c["hd"], c["rows"], s["pos"], c["heads"], s["q"], s["q_out"], c["kv"], s["k"],
                           s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "append":
        q.qmv_kv_append_rope(s["cache"], s["rope"], s["tokens"], c["heads"], s["q"], s["q_out"], s["k"], s["v"],
                             start=s["start_arg"])
        return [s["q_out"], s["pages"].view(DTYPE[c["t"]])]
    if op == "write4":
        q.qmv_kv_append(s["cache"], s["tokens"], s["k"], s["v"], start=s["start_arg"])
        q.qmv_kv_read(s["cache"], s["tokens"], s["k_out"], s["v_out"], start=s["start_arg"])
        return [s["k_out"], s["v_out"]]
    scale = c["hd"] ** -0.5
    if c["call"] == "decode":
        q.qmv_attn_decode(s["cache"], c["n"], c["heads"], s["q"], scale, s["out"], c["len"], window=c["window"],
                          sinks=c["sinks"], workspace=s["ws"])
    else:
        q.qmv_attn_prefill(s["cache"], s["tokens"], c["heads"], s["q"], scale, s["out"], c["len"],
                           start=s["start_arg"], window=c["window"], sinks=c["sinks"], workspace=s["ws"])
    return s["out"]


def _pages_out(s):
    return [s["table"], s["seq_len"], s["free"], s["count"], s["granted"], s["start"], s["pos"], s["slot"]]


def _turn_pages(s):
    """Pages behind the kept lengths go back on the free stack, the first of them on top; then every
    sequence that the table, the stack and the rows have room for gets its tokens, in order."""
    c = s["case"]
    page, table, free, count = c["page"], s["table"], s["free"], s["count"]
    n_pages, cap = s["n_pages"], table.shape[1] * page
    at = torch.arange(table.shape[1], device="cuda")

    def pages_of(length):
        return (length + page - 1) // page

    length = s["seq_len"].long().clamp(0, cap)
    new = torch.where(s["keep"] >= 0, torch.minimum(length, s["keep"].long()), length)
    gone = (at >= pages_of(new)[:, None]) & (at < pages_of(length)[:, None])
    back = gone & (table >= 0) & (table < n_pages)
    rank = back.flatten().cumsum(0)
    to = count + rank[-1] - rank
    ok = back.flatten() & (to < n_pages)
    longer = torch.cat([free, free[:1]])                     # the last entry takes what is not pushed
    longer[torch.where(ok, to, n_pages)] = table.flatten()
    free.copy_(longer[:-1])
    count.copy_((count + rank[-1]).clamp(max=n_pages))
    table.masked_fill_(gone, -1)
    s["seq_len"].copy_(new)

    length, add = new, s["add"].long()
    fits = (add > 0) & (length + add <= cap)
    need = torch.where(fits, pages_of(length + add) - pages_of(length), 0)
    rows = torch.where(fits, add, 0).cumsum(0)
    given = fits & (rows <= s["rows"]) & ((need == 0) | (need.cumsum(0) <= count))
    granted, need = torch.where(given, add, 0), torch.where(given, need, 0)
    start = torch.nn.functional.pad(granted.cumsum(0), (1, 0))
    k = at - pages_of(length)[:, None]
    pick = (count - 1 - (need.cumsum(0) - need)[:, None] - k).clamp(0, n_pages - 1)
    table.copy_(torch.where((k >= 0) & (k < need[:, None]), free[pick], table))
    count.sub_(need.sum())
    length = length + granted
    s["seq_len"].copy_(length)
    s["granted"].copy_(granted)
    s["start"].copy_(start)
    r = torch.arange(s["rows"], device="cuda")
    live = r < start[-1]
    seq = torch.searchsorted(start[1:], r, right=True).clamp(max=c["seqs"] - 1)
    pos = length[seq] - (start[seq + 1] - r)
    pg = table[seq, (pos // page).clamp(min=0)].long()
    s["pos"].copy_(torch.where(live, pos, -1))
    s["slot"].copy_(torch.where(live & (pg >= 0) & (pg < n_pages), pg * page + pos % page, -1))
    return _pages_out(s)


def _turn(s, x, heads, weight, pos):
    """x [rows][heads * hd] normed for each head and turned by its rows' positions."""
    c = s["case"]
    x = x.unflatten(-1, (heads, c["hd"]))
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
    angle = pos.double()[:, None, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    r = c["rot"]
    turned = x[..., :r]
    a, b = turned.chunk(2, -1) if c["pairs"] == "halves" else (turned[..., 0::2], turned[..., 1::2])
    parts = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.cat(parts, -1) if c["pairs"] == "halves" else torch.stack(parts, -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).flatten(1)


def _rope_rows(s):
    c = s["case"]
    s["q_out"].copy_(_turn(s, s["q"], c["heads"], s["q_norm"], s["pos"]))
    s["k_out"].copy_(_turn(s, s["k"], c["kv"], s["k_norm"], s["pos"]))
    return [s["q_out"], s["k_out"]]


def _new_positions(s):
    """Sequence and position of every new token, in row order."""
    start = s["start"].long()
    rows = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), rows, right=True)
    return seq, s["seq_len"].long()[seq] - (start[seq + 1] - rows)


def _append_rows(s):
    c = s["case"]
    seq, pos = _new_positions(s)
    s["q_out"].copy_(_turn(s, s["q"], c["heads"], s["q_norm"], pos))
    keys = _turn(s, s["k"], c["kv"], s["k_norm"], pos)
    k, v = _views16(c, s["pages"])
    page, slot = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    k[page, :, slot] = keys.unflatten(-1, (c["kv"], c["hd"])).to(k.dtype)
    v[page, :, slot // 16, :, slot % 16] = s["v"].unflatten(-1, (c["kv"], c["hd"])).to(v.dtype)
    return [s["q_out"], s["pages"].view(DTYPE[c["t"]])]


def _write_rows(s):
    """Blocks of 32 values of a row: the scale is -1/8 of the value of largest size (the positive one of
    two), rounded to 8 bits of significand, then to f16, at most 2720; the codes are the nearest ones."""
    c = s["case"]
    seq, pos = _new_positions(s)
    page, slot = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    kc, vc, ks, vs = _views4(c, s["pages"])
    order = (slot & ~3) | ((slot & 1) << 1) | ((slot >> 1) & 1)
    for x, out in ((s["k"], s["k_out"]), (s["v"], s["v_out"])):
        x = x.unflatten(-1, (c["kv"], c["hd"] // 32, 32))
        hi, lo = x.amax(-1), x.amin(-1)
        d = (torch.where(hi >= -lo, hi, lo) * -0.125).to(torch.bfloat16).float().clamp(-2720, 2720).half()
        f = d.float()[..., None]
        code = torch.where(f == 0, 0, (x / f).round()).clamp(-8, 7)
        u = (code + 8).to(torch.uint8)
        byte = (u[..., :16] | u[..., 16:] << 4).flatten(-2)
        if out is s["k_out"]:
            kc[page, :, slot] = byte
            ks[page, :, slot] = d
        else:
            vc[page, :, slot // 16, :, order % 16] = byte
            vs[page, :, :, slot] = d
        out.copy_((code * f).flatten(1))
    return [s["k_out"], s["v_out"]]


def _values4(codes, scale):
    """codes [..., hd/2] and scales [..., hd/32] as values [..., hd]."""
    b = codes.unflatten(-1, (-1, 16))
    u = torch.cat([b & 15, b >> 4], -1).float() - 8
    return (u * scale[..., None].float()).flatten(-2)


def _attend(s):
    """softmax(scale q k^T) v over the visible positions, all sequences padded to the longest."""
    c = s["case"]
    kv, hd, seqs, g = c["kv"], c["hd"], c["seqs"], c["heads"] // c["kv"]
    kc, vc, ks, vs = _views4(c, s["pages"])
    table = s["table"].long()
    length = table.shape[1] * c["page"]
    k = _values4(kc[table], ks[table]).transpose(1, 2).reshape(seqs, kv, length, hd)
    vb = vc[table].transpose(-1, -2).unflatten(-2, (4, 4))[..., [0, 2, 1, 3], :].flatten(-4, -2)
    v = _values4(vb, vs[table].transpose(-1, -2)).transpose(1, 2).reshape(seqs, kv, length, hd)
    seq, pos = _new_positions(s)
    most = max(s["news"])
    j = torch.arange(s["tokens"], device="cuda") - s["start"].long()[seq]
    q = torch.zeros(seqs, most, kv, g, hd, device="cuda")
    q[seq, j] = s["q"].view(-1, kv, g, hd)
    at = torch.full((seqs, most), -1, device="cuda")
    at[seq, j] = pos
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(seqs, kv, most * g, hd), k.transpose(2, 3)).mul_(hd ** -0.5)
    key = torch.arange(length, device="cuda")
    sees = key <= at[..., None]
    if c["window"] > 0:
        sees &= (key > at[..., None] - c["window"]) | (key < c["sinks"])
    sees = sees[:, None, :, None]
    x = x.view(seqs, kv, most, g, length).masked_fill_(~sees, -torch.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    x /= x.sum(-1, keepdim=True).clamp_(min=1e-30)
    o = torch.matmul(x.view(seqs, kv, most * g, length), v).view(seqs, kv, most, g, hd)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4)[seq, j].flatten(1))
    return s["out"]


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def _visible(c, p):
    """How many positions the query at position p sees."""
    if c["window"] <= 0 or p < 0:
        return max(0, p + 1)
    return min(p + 1, c["window"]) + min(c["sinks"], max(0, p + 1 - c["window"]))


def work(case):
    c = case
    if c["op"] == "pages":
        keep, add = _adds(c)
        turned = sum(-(-(k + a) // c["page"]) - -(-k // c["page"]) for k, a in zip(keep, add))
        return {"bytes": 12 * sum(add) + 24 * c["seqs"] + 24 * turned, "flops": 0}
    kv, hd = c["kv"], c["hd"]
    if c["op"] == "rope":
        return {"bytes": c["rows"] * (8 * (c["heads"] + kv) * hd + 4), "flops": 0}
    tokens = sum(_news(c))
    if c["op"] == "append":
        return {"bytes": tokens * (8 * c["heads"] * hd + 8 * kv * hd + 4 * kv * hd), "flops": 0}
    row = 2 * kv * hd * 9 // 16              # K and V of one cached position
    if c["op"] == "write4":
        return {"bytes": tokens * (8 * kv * hd + 2 * row + 8 * kv * hd), "flops": 0}
    read = flops = 0
    for length, n in zip(_lengths(c), _news(c)):
        flops += 4 * c["heads"] * hd * sum(_visible(c, length - n + j) for j in range(n))
        p0 = max(0, length - n)
        read += length if c["window"] <= 0 else min(length, c["window"] + n - 1 + min(c["sinks"], max(0, p0 + 1 - c["window"])))
    return {"bytes": read * row + 8 * tokens * c["heads"] * hd, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    return {"pages": _exact_pages, "rope": _exact_rope, "append": _exact_append, "write4": _exact_write,
            "attend4": _exact_attend}[c["op"]](c, s)


def _exact_pages(c, s):
    """One page after the other, on the host."""
    page, n_pages = c["page"], s["n_pages"]
    table, free = s["table"].tolist(), s["free"].tolist()
    stack = free[:int(s["count"])]
    lens, keep, add = s["seq_len"].tolist(), s["keep"].tolist(), s["add"].tolist()
    for b in reversed(range(c["seqs"])):
        first, end = -(-min(lens[b], keep[b]) // page), -(-lens[b] // page)
        for j in reversed(range(first, end)):
            stack.append(table[b][j])
            table[b][j] = -1
        lens[b] = min(lens[b], keep[b])
    free[:len(stack)] = stack
    granted, start, pos, slot = [], [0], [], []
    for b in range(c["seqs"]):
        for p in range(lens[b], lens[b] + add[b]):
            if p % page == 0:
                table[b][p // page] = stack.pop()
            pos.append(p)
            slot.append(table[b][p // page] * page + p % page)
        lens[b] += add[b]
        granted.append(add[b])
        start.append(start[-1] + add[b])

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    return [i32(table), i32(lens), i32(free), i32([len(stack)]), i32(granted), i32(start), i32(pos),
            torch.tensor(slot, dtype=torch.int64, device="cuda")]


def _exact_turn(c, s, x, weight, pos):
    """Pairs as complex numbers, multiplied by e^(i t)."""
    x = x.double().reshape(x.shape[0], -1, c["hd"])
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / c["hd"] + s["eps"]).sqrt() * weight.double()
    out = x.clone()
    i = torch.arange(c["rot"] // 2, device="cuda")
    a, b = (i, i + c["rot"] // 2) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
    t = pos.double()[:, None] * s["freq"]
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(t), t)[:, None]
    out[..., a], out[..., b] = z.real, z.imag
    return out.reshape(x.shape[0], -1)


def _exact_rope(c, s):
    return [_exact_turn(c, s, s["q"], s["q_norm"], s["pos"]), _exact_turn(c, s, s["k"], s["k_norm"], s["pos"])]


def _places(c, s):
    """Position, page and slot of every new token, one after the other on the host."""
    table = s["table"].tolist()
    pos, pg = [], []
    for b in range(c["seqs"]):
        for p in range(s["lens"][b] - s["news"][b], s["lens"][b]):
            pos.append(p)
            pg.append(table[b][p // c["page"]])
    pos = torch.tensor(pos, device="cuda")
    return pos, torch.tensor(pg, device="cuda"), pos % c["page"]


def _exact_append(c, s):
    """The pool as numbers, new rows by flat index; new values before they are rounded."""
    kv, page, hd = c["kv"], c["page"], c["hd"]
    flat = s["pages"].view(DTYPE[c["t"]]).double()
    pos, pg, slot = _places(c, s)
    base = (pg * (kv * 2 * page * hd))[:, None, None] + torch.arange(kv, device="cuda")[None, :, None] * (2 * page * hd)
    slot = slot[:, None, None]
    d = torch.arange(hd, device="cuda")[None, None, :]
    flat[base + slot * hd + d] = _exact_turn(c, s, s["k"], s["k_norm"], pos).view(-1, kv, hd)
    flat[base + page * hd + (slot // 16) * (hd * 16) + d * 16 + slot % 16] = s["v"].double().reshape(-1, kv, hd)
    return [_exact_turn(c, s, s["q"], s["q_norm"], pos), flat]


def _exact_write(c, s):
    """The nearest of a block's sixteen values, by the quotient as 32 bits hold it."""
    out = []
    for x in (s["k"], s["v"]):
        x = x.double().reshape(-1, 32)
        big = x.abs().amax(1, keepdim=True)
        sign = torch.where((x == big).any(1, keepdim=True), 1.0, -1.0)
        d = (sign * big / -8).to(torch.bfloat16).double().clamp(-2720, 2720).half().double()
        ratio = (x / torch.where(d == 0, torch.inf, d)).float().double()
        out.append((torch.round(ratio).clamp(-8, 7) * d).view(s["tokens"], -1))
    return out


def _cached(c, s, b, h, length):
    """K and V rows 0..length-1 of one sequence and head in 64 bits."""
    page, hd = c["page"], c["hd"]
    raw = s["pages"].view(-1, c["kv"], _head_bytes(c))[s["table"][b].long(), h]
    n, half, sc = raw.shape[0], page * hd // 2, page * hd // 16
    col = torch.arange(hd, device="cuda")
    byte, shift = col // 32 * 16 + col % 16, col % 32 // 16 * 4
    p = torch.arange(page, device="cuda")[:, None]
    k = raw[:, p * (hd // 2) + byte] >> shift & 15
    place = torch.tensor([0, 2, 1, 3], device="cuda")[p % 4] + p % 16 // 4 * 4
    v = raw[:, half + p // 16 * (8 * hd) + byte * 16 + place] >> shift & 15
    ks = raw[:, 2 * half:2 * half + sc].contiguous().view(torch.float16).double()[:, p * (hd // 32) + col // 32]
    vs = raw[:, 2 * half + sc:].contiguous().view(torch.float16).double()[:, col // 32 * page + p]
    return ((k.double() - 8) * ks).view(n * page, hd)[:length], ((v.double() - 8) * vs).view(n * page, hd)[:length]


def _exact_attend(c, s):
    out = torch.zeros(s["tokens"], c["heads"], c["hd"], dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv"]
    row0 = 0
    for b in range(c["seqs"]):
        n, length = s["news"][b], s["lens"][b]
        where = torch.arange(length, device="cuda")
        query = torch.arange(length - n, length, device="cuda")
        hidden = where[None, :] > query[:, None]
        if c["window"]:
            hidden |= (where[None, :] + c["window"] <= query[:, None]) & (where[None, :] >= c["sinks"])
        for h in range(c["kv"]):
            keys, values = _cached(c, s, b, h, length)
            for i in range(h * group, (h + 1) * group):
                qi = s["q"][row0:row0 + n, i * c["hd"]:(i + 1) * c["hd"]].double()
                logit = qi @ keys.T * c["hd"] ** -0.5
                logit[hidden] = float("-inf")
                out[row0:row0 + n, i] = torch.nan_to_num(torch.softmax(logit, 1)) @ values
        row0 += n
    return out.view(s["tokens"], -1)
