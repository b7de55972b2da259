"""The cache and attention calls as measurable cases: a plain form in torch, the
library's calls, and the same results in 64 bits.

A case is one call of one operator:

  append   new tokens' keys and values written into a paged cache
  decode   attention of the last n (1 to 16) tokens of each sequence over its
           cache, with the optional running sums of attention weight
  prefill  causal attention of whole or chunked prompts over the cache
  evict    the cache cut to `keep` positions by accumulated weight

Sizes are the layer shapes of the workloads this repository runs elsewhere:
9 query / 3 key-value heads of 64 (the 576-wide model), 32 / 8 of 64 (hidden
2048) and 32 / 8 of 128 (hidden 4096).

A cache is one byte tensor of pages.  A page holds, for each key-value head,
K [page][hd], then V in blocks of 16 positions [page/16][hd][16], and for
8-bit caches the f32 scale of every K row and of every V row.
"""
import torch

own = False

GGUF = {"f16": 1, "bf16": 30, "i8": 24}
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "i8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, t, heads, kv, hd, page, seqs, n, length, window=0, sinks=0, acc=False, keep=0, ragged=False):
    c = dict(op=op, t=t, heads=heads, kv=kv, hd=hd, page=page, seqs=seqs, n=n, len=length, window=window,
             sinks=sinks, acc=acc, keep=keep, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 16 sequences: 16 rows of K and V, pure latency
        _case("append_step", "append", "f16", 32, 8, 128, 64, 16, 1, 2048),
        # prompts of different lengths in one batch, K and V read out of the stacked QKV rows
        _case("append_prompts", "append", "bf16", 32, 8, 128, 64, 4, 2100, 2100, ragged=True),
        # the smallest model's attention early in a chat: latency
        _case("decode_small", "decode", "f16", 9, 3, 64, 16, 1, 1, 301),
        # a serving batch with mixed context lengths: the cache stream
        _case("decode_batch", "decode", "f16", 32, 8, 128, 64, 32, 1, 8150, ragged=True),
        # one user with a very long context in an 8-bit cache: split over the length
        _case("decode_long_i8", "decode", "i8", 32, 8, 128, 128, 1, 1, 131071),
        # eight drafted tokens checked at once in a sliding window with sinks
        _case("verify_window", "decode", "bf16", 32, 8, 64, 32, 8, 8, 20011, window=4096, sinks=4),
        # decode that also collects the weights an eviction goes by
        _case("decode_weights", "decode", "f16", 32, 8, 64, 64, 4, 1, 4352, acc=True),
        # a short question to the smallest model
        _case("prefill_small", "prefill", "f16", 9, 3, 64, 16, 1, 97, 97),
        # a long prompt of the 4096-wide model, full causal attention
        _case("prefill_long", "prefill", "f16", 32, 8, 128, 64, 1, 4096, 4096),
        # ragged prompts through a window with sinks, 8-bit cache
        _case("prefill_window_i8", "prefill", "i8", 32, 8, 64, 128, 3, 5000, 5000, window=1024, sinks=4, ragged=True),
        # a cache that outgrew its budget by one slack of 256
        _case("evict_batch", "evict", "f16", 32, 8, 128, 64, 8, 0, 4352, sinks=4, window=512, keep=4096),
        # a small model's cache cut in half
        _case("evict_small", "evict", "bf16", 9, 3, 64, 16, 1, 0, 1001, sinks=4, window=64, keep=500),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "evict"])
    heads, kv, hd = rng.choice([(9, 3, 64), (32, 8, 64), (32, 8, 128), (8, 8, 64), (16, 2, 128)])
    page = rng.choice([16, 32, 64, 128])
    t = rng.choice(["f16", "bf16", "i8"])
    if op == "append":
        t = rng.choice(["f16", "bf16"])
        seqs = rng.randint(1, 8)
        length = _log(rng, 17, 1500)
        n = rng.choice([1, _log(rng, 1, length)])
        return _case("", op, t, heads, kv, hd, page, seqs, n, length, ragged=rng.random() < 0.5)
    if op == "decode":
        seqs = _log(rng, 1, 32)
        length = _log(rng, 33, min(131071, 200000 // seqs))
        n = rng.choice([1, 1, 1, rng.randint(2, 16)])
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, length), rng.randint(0, 9))])
        return _case("", op, t, heads, kv, hd, page, seqs, n, length, window, sinks, rng.random() < 0.3,
                     ragged=rng.random() < 0.5)
    if op == "prefill":
        seqs = rng.randint(1, 3)
        length = _log(rng, 20, 4000 // seqs)
        n = rng.choice([length, _log(rng, 17, length)])
        window, sinks = rng.choice([(0, 0), (_log(rng, 16, length), rng.randint(0, 9))])
        return _case("", op, t, heads, kv, hd, page, seqs, n, length, window, sinks, ragged=rng.random() < 0.5)
    t = rng.choice(["f16", "bf16"])
    seqs = rng.randint(1, 8)
    length = _log(rng, 100, 4300)
    keep = rng.randint(length // 3, length - 1)
    first = rng.randint(0, 8)
    return _case("", op, t, heads, kv, hd, page, seqs, 0, length, rng.randint(0, (keep - first) // 2), first,
                 keep=keep, ragged=rng.random() < 0.5)


def _lengths(c):
    """Cached positions of each sequence, the new tokens among them."""
    if not c["ragged"]:
        return [c["len"]] * c["seqs"]
    return [max(1, c["len"] - s * c["len"] // (2 * c["seqs"]) - 3 * s) for s in range(c["seqs"])]


def _news(c):
    """New tokens of each sequence: decode takes the same number for all."""
    if c["op"] == "decode":
        return [c["n"]] * c["seqs"]
    return [min(c["n"], length) for length in _lengths(c)]


def _head_bytes(c):
    return 2 * c["page"] * c["hd"] * SIZE[c["t"]] + (8 * c["page"] if c["t"] == "i8" else 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _views(c, pages):
    """K [n_pages][kv][page][hd], V [n_pages][kv][page/16][hd][16] and the row scales (8-bit only) of a pool."""
    kv, page, hd = c["kv"], c["page"], c["hd"]
    pool = pages.view(-1, kv, _head_bytes(c))
    part = page * hd * SIZE[c["t"]]
    k = pool[..., :part].view(DTYPE[c["t"]]).unflatten(-1, (page, hd))
    v = pool[..., part:2 * part].view(DTYPE[c["t"]]).unflatten(-1, (page // 16, hd, 16))
    if c["t"] != "i8":
        return k, v, None, None
    ks = pool[..., 2 * part:2 * part + 4 * page].view(torch.float32)
    vs = pool[..., 2 * part + 4 * page:].view(torch.float32)
    return k, v, ks, vs


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kv, page, hd, heads, seqs = c["kv"], c["page"], c["hd"], c["heads"], c["seqs"]
    lens, news = _lengths(c), _news(c)
    per_seq = -(-c["len"] // page)
    n_src = seqs * per_seq
    keep_pages = -(-c["keep"] // page)
    n_pages = n_src + seqs * keep_pages
    pages = torch.empty(n_pages * kv * _head_bytes(c), dtype=torch.uint8, device=dev)
    k, v, ks, vs = _views(c, pages)
    for view, scale in ((k, ks), (v, vs)):       # every slot holds something, as pages used before do
        if c["t"] == "i8":
            view.copy_(torch.randint(-127, 128, view.shape, generator=g, device=dev, dtype=torch.int8))
            scale.copy_(0.02 + 0.02 * torch.rand(scale.shape, generator=g, device=dev))
        else:
            view.copy_(torch.randn(view.shape, generator=g, device=dev, dtype=torch.float32))
    table = torch.randperm(n_src, generator=g, device=dev).to(torch.int32).view(seqs, per_seq)
    s = {"case": c, "pages": pages, "n_pages": n_pages, "table": table, "lens": lens, "news": news,
         "seq_len": torch.tensor(lens, dtype=torch.int32, device=dev)}
    tokens = sum(news)
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
    s["tokens"], s["scale"], s["n_src"] = tokens, hd ** -0.5, n_src
    s["start_arg"] = s["start"] if len(set(news)) > 1 else None      # None: as many tokens for each sequence
    if c["op"] == "append":
        # rows of the stacked QKV product, K and V as column ranges of it
        qkv = torch.randn(tokens, (heads + 2 * kv) * hd, generator=g, device=dev)
        s["k"] = qkv[:, heads * hd:(heads + kv) * hd]
        s["v"] = qkv[:, (heads + kv) * hd:]
    elif c["op"] == "evict":
        s["dst"] = (n_src + torch.randperm(seqs * keep_pages, generator=g, device=dev)).to(torch.int32).view(seqs, -1)
        s["acc"] = torch.rand(seqs, kv, c["len"], generator=g, device=dev).square_()
        s["kept"] = torch.empty(seqs, kv, c["keep"], dtype=torch.int32, device=dev)
        s["acc_out"] = torch.empty(seqs, kv, c["keep"], device=dev)
        s["len_out"] = torch.empty(seqs, dtype=torch.int32, device=dev)
    else:
        s["q"] = 1.5 * torch.randn(tokens, heads * hd, generator=g, device=dev)
        s["out"] = torch.empty(tokens, heads * hd, device=dev)
        s["acc"] = torch.rand(seqs, kv, c["len"], generator=g, device=dev) if c["acc"] else None
    s["cells"] = _out_pages(c, pages, n_src if c["op"] == "evict" else 0)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "decode": _attend, "prefill": _attend, "evict": _evict}[state["case"]["op"]](state)


def _run_own(s):
    import gguf_dequant_matvec_amd as q
    c = s["case"]
    if "cache" not in s:             # what a program keeps: the cache's handle and its workspace
        s["cache"] = q.KvCache(c["t"], c["kv"], c["hd"], c["page"], s["pages"], s["table"], s["seq_len"])
        need = 0
        if c["op"] == "decode":
            need = q.qmv_attn_decode_workspace(s["cache"], c["n"], c["heads"], c["len"], c["window"], c["sinks"],
                                               c["acc"])
        elif c["op"] == "prefill":
            need = q.qmv_attn_prefill_workspace(s["cache"], s["tokens"], c["heads"], c["len"], c["window"], c["sinks"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    cache = s["cache"]
    if c["op"] == "append":
        q.qmv_kv_append(cache, s["tokens"], s["k"], s["v"], start=s["start_arg"])
        return s["cells"]
    if c["op"] == "decode":
        q.qmv_attn_decode(cache, c["n"], c["heads"], s["q"], s["scale"], s["out"], c["len"], window=c["window"],
                          sinks=c["sinks"], acc=s["acc"], workspace=s["ws"])
        return [s["out"], s["acc"]]
    if c["op"] == "prefill":
        q.qmv_attn_prefill(cache, s["tokens"], c["heads"], s["q"], s["scale"], s["out"], c["len"], start=s["start_arg"],
                           window=c["window"], sinks=c["sinks"], workspace=s["ws"])
        return [s["out"], None]
    q.qmv_kv_evict(cache, s["dst"], c["keep"], c["sinks"], c["window"], s["acc"], s["kept"], s["acc_out"], s["len_out"])
    return [s["cells"], s["kept"], s["acc_out"], s["len_out"]]


def _out_pages(c, pages, first):
    """The pages from `first` on as the values they hold."""
    return pages.view(-1, c["kv"] * _head_bytes(c))[first:].view(DTYPE[c["t"]])


def _new_positions(s):
    """Sequence and position of every new token, in row order."""
    start, n = s["start"].long(), s["tokens"]
    rows = torch.arange(n, device="cuda")
    seq = torch.searchsorted(start[1:].contiguous(), rows, right=True)
    return seq, s["seq_len"].long()[seq] - (start[seq + 1] - rows)


def _append(s):
    c = s["case"]
    k, v, _, _ = _views(c, s["pages"])
    seq, pos = _new_positions(s)
    page = s["table"].long()[seq, pos // c["page"]]
    slot = pos % c["page"]
    k[page, :, slot] = s["k"].unflatten(-1, (c["kv"], c["hd"])).to(k.dtype)
    v[page, :, slot // 16, :, slot % 16] = s["v"].unflatten(-1, (c["kv"], c["hd"])).to(v.dtype)
    return s["cells"]


def _attend(s):
    """softmax(scale q k^T) v over the visible positions, all sequences padded to the longest."""
    c = s["case"]
    kv, hd, seqs, g = c["kv"], c["hd"], c["seqs"], c["heads"] // c["kv"]
    k, v, ks, vs = _views(c, s["pages"])
    table = s["table"].long()
    length = table.shape[1] * c["page"]
    k = k[table].float().transpose(1, 2).reshape(seqs, kv, length, hd)
    v = v[table].float().permute(0, 2, 1, 3, 5, 4).reshape(seqs, kv, length, hd)
    if ks is not None:
        k = k * ks[table].transpose(1, 2).reshape(seqs, kv, length, 1)
        v = v * vs[table].transpose(1, 2).reshape(seqs, kv, length, 1)
    seq, pos = _new_positions(s)
    most = max(s["news"])
    j = torch.arange(s["tokens"], device="cuda") - s["start"].long()[seq]
    q = torch.zeros(seqs, most, kv, g, hd, device="cuda")
    q[seq, j] = s["q"].view(-1, kv, g, hd)
    at = torch.full((seqs, most), -1, device="cuda")
    at[seq, j] = pos
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(seqs, kv, most * g, hd), k.transpose(2, 3)).mul_(s["scale"])
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
    if s["acc"] is not None:
        s["acc"] += x.sum((2, 3))[..., :c["len"]]
    return [s["out"], s["acc"]]


def _evict(s):
    c = s["case"]
    kv, keep, first, recent = c["kv"], c["keep"], c["sinks"], c["window"]
    lens = s["seq_len"].long()[:, None, None]
    at = torch.arange(c["len"], device="cuda")
    always = (at < first) | (at >= lens - recent)
    score = s["acc"].masked_fill(always, torch.inf).masked_fill(at >= lens, -torch.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]   # ties: the lower position
    order = torch.where(torch.arange(keep, device="cuda") < lens, order, c["len"])
    order = torch.sort(order, dim=-1).values
    live = order < lens
    src = order.clamp(max=c["len"] - 1)
    head = torch.arange(kv, device="cuda")[None, :, None]
    seq = torch.arange(c["seqs"], device="cuda")[:, None, None]
    k, v, _, _ = _views(c, s["pages"])
    page, slot = s["table"].long()[seq, src // c["page"]], src % c["page"]
    kk, vv = k[page, head, slot][live], v[page, head, slot // 16, :, slot % 16][live]
    seq, head, i = live.nonzero().unbind(1)
    page, slot = s["dst"].long()[seq, i // c["page"]], i % c["page"]
    k[page, head, slot] = kk
    v[page, head, slot // 16, :, slot % 16] = vv
    s["kept"].copy_(torch.where(live, order, -1))
    s["acc_out"].copy_(s["acc"].gather(-1, src).masked_fill_(~live, 0))
    s["len_out"].copy_(lens.flatten().clamp(max=keep))
    return [s["cells"], s["kept"], s["acc_out"], s["len_out"]]


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
    kv, hd, heads = c["kv"], c["hd"], c["heads"]
    row = 2 * kv * (hd * SIZE[c["t"]] + (4 if c["t"] == "i8" else 0))    # K and V of one cached position
    lens, news = _lengths(c), _news(c)
    tokens = sum(news)
    if c["op"] == "append":
        return {"bytes": tokens * (8 * kv * hd + row), "flops": 0}
    if c["op"] == "evict":
        kept = sum(min(c["keep"], length) for length in lens)
        return {"bytes": 2 * kept * row + 4 * kv * (sum(lens) + 2 * c["seqs"] * c["keep"]), "flops": 0}
    read = flops = 0
    for length, n in zip(lens, news):
        flops += 4 * heads * hd * sum(_visible(c, length - n + j) for j in range(n))
        p0 = max(0, length - n)
        read += length if c["window"] <= 0 else min(length, c["window"] + n - 1 + min(c["sinks"], max(0, p0 + 1 - c["window"])))
    extra = 8 * kv * sum(lens) if c["acc"] else 0
    return {"bytes": read * row + 8 * tokens * heads * hd + extra, "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    out = torch.zeros(s["tokens"], c["heads"], c["hd"], dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if s["acc"] is not None else None
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
                weight = torch.nan_to_num(torch.softmax(logit, 1))
                out[row0:row0 + n, i] = weight @ values
                if acc is not None:
                    acc[b, h, :length] += weight.sum(0)
        row0 += n
    return [out.view(s["tokens"], -1), acc]


def _cached(c, s, b, h, length):
    """K and V rows 0..length-1 of one sequence and head in 64 bits, read page by page."""
    kv, page, hd, t = c["kv"], c["page"], c["hd"], c["t"]
    size = _head_bytes(c)
    raw = s["pages"].view(s["n_pages"], kv, size)[s["table"][b].long(), h].contiguous()
    n, part = raw.shape[0], page * hd * SIZE[t]
    k = raw[:, :part].contiguous().view(DTYPE[t]).double().view(n * page, hd)
    v = raw[:, part:2 * part].contiguous().view(DTYPE[t]).double().view(n * page // 16, hd, 16)
    v = v.transpose(1, 2).reshape(n * page, hd)
    if t == "i8":
        scales = raw[:, 2 * part:].contiguous().view(torch.float32).double().view(n, 2, page)
        k = k * scales[:, 0].reshape(-1, 1)
        v = v * scales[:, 1].reshape(-1, 1)
    return k[:length], v[:length]


def _exact_append(c, s):
    """The pool as numbers, the new rows put in one token at a time (by flat index, for all heads)."""
    dt = DTYPE[c["t"]]
    flat = s["pages"].view(dt).double()
    kv, page, hd = c["kv"], c["page"], c["hd"]
    table = s["table"].tolist()
    row, k0 = [], []
    for b in range(c["seqs"]):
        for j in range(s["news"][b]):
            p = s["lens"][b] - s["news"][b] + j
            row.append(p % page)
            k0.append(table[b][p // page])
    slot = torch.tensor(row, device="cuda")[:, None, None]
    base = torch.tensor(k0, device="cuda")[:, None, None] * (kv * 2 * page * hd)
    base = base + torch.arange(kv, device="cuda")[None, :, None] * (2 * page * hd)
    d = torch.arange(hd, device="cuda")[None, None, :]
    flat[base + slot * hd + d] = s["k"].to(dt).double().reshape(-1, kv, hd)
    flat[base + page * hd + (slot // 16) * (hd * 16) + d * 16 + slot % 16] = s["v"].to(dt).double().reshape(-1, kv, hd)
    return flat.view(s["n_pages"], -1)


def _exact_evict(c, s):
    dt, kv, page, hd, keep = DTYPE[c["t"]], c["kv"], c["page"], c["hd"], c["keep"]
    flat = s["pages"].view(dt).double()
    acc = s["acc"].cpu()
    kept = torch.full((c["seqs"], kv, keep), -1, dtype=torch.int32)
    acc_out = torch.zeros(c["seqs"], kv, keep, dtype=torch.float64)
    table, dst = s["table"].long(), s["dst"].long()
    d = torch.arange(hd, device="cuda")[None, :]
    for b in range(c["seqs"]):
        length = s["lens"][b]
        for h in range(kv):
            score = acc[b, h, :length].double()
            sure = [p for p in range(length) if p < c["sinks"] or p >= length - c["window"]]
            if length <= keep:
                chosen = list(range(length))
            else:
                free = sorted(set(range(length)) - set(sure), key=lambda p: (-float(score[p]), p))
                chosen = sorted(sure + free[:keep - len(sure)])
            m = len(chosen)
            at = torch.tensor(chosen)
            kept[b, h, :m] = at.int()
            acc_out[b, h, :m] = score[at]
            at = at.cuda()
            to = torch.arange(m, device="cuda")

            def base(tab, p):
                return ((tab[b][p // page] * kv + h) * (2 * page * hd))[:, None]

            def v_at(p):
                return page * hd + ((p % page) // 16 * (hd * 16) + p % 16)[:, None] + d * 16

            flat[base(dst, to) + (to % page * hd)[:, None] + d] = flat[base(table, at) + (at % page * hd)[:, None] + d]
            flat[base(dst, to) + v_at(to)] = flat[base(table, at) + v_at(at)]
    return [flat.view(s["n_pages"], -1)[s["n_src"]:], kept, acc_out, torch.tensor([min(n, keep) for n in s["lens"]], dtype=torch.int32)]
