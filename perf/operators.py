"""Cases of the serving operators around the paged 8-bit cache, with their plain forms.

Four operators, as a serving program strings them together:

* ``prefill``  attention of a prompt (or of a chunk of one) over bf16 keys and
  values, with the score modifiers: tanh cap, distance bias, window, documents,
  bidirectional prefix (``lrkv_prefill_attn``);
* ``append``   quantising new key and value rows into the pages of the 8-bit
  cache, one scale per page and head, and reading them back as bf16
  (``lrkv_paged_append``, ``lrkv_paged_read``);
* ``attn``     attention of one or a few new tokens over the pages
  (``lrkv_paged_attn``);
* ``pages``    forking, freeing, copying and compacting pages (``lrkv_pages_*``).

``own`` false: the plain forms, elementary torch operations in 32 bits.
``own`` true: the calls a user makes of this package.
"""
import math

import torch

own = False

D = 128                       # head dimension
QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100            # a scale below this is stored as zero
BIG = 3.3895313892515355e38   # largest finite bf16


# ---- cases -----------------------------------------------------------------------------


def listed():
    return [
        # a handful of short chat prompts of different lengths: latency
        dict(name="prefill_short_ragged", op="prefill", B=3, Hq=32, Hkv=8, t_q=203, t_k=203, ragged=True,
             softcap=0.0, window=0, slopes=False, docs=1, prefix=0),
        # an 8K prompt on the Llama-3.1-8B head layout
        dict(name="prefill_8k_causal", op="prefill", B=1, Hq=32, Hkv=8, t_q=8192, t_k=8192, ragged=False,
             softcap=0.0, window=0, slopes=False, docs=1, prefix=0),
        # documents packed into one row, capped scores
        dict(name="prefill_docs_softcap", op="prefill", B=1, Hq=32, Hkv=8, t_q=8192, t_k=8192, ragged=False,
             softcap=50.0, window=0, slopes=False, docs=5, prefix=0),
        # the second half of a 16K prompt on the multi-head layout, distance bias and a prefix that sees itself
        dict(name="prefill_chunk_16k_mha", op="prefill", B=1, Hq=32, Hkv=32, t_q=8192, t_k=16384, ragged=False,
             softcap=0.0, window=0, slopes=True, docs=1, prefix=500),
        # one chat at 8K, one new token: the latency of a decode step
        dict(name="attn_8k_one_token", op="attn", B=1, Hq=32, Hkv=8, t_q=1, ctx=8192, ragged=False, code="int8",
             page=64, softcap=0.0, window=0, slopes=False),
        # sixteen chats of 8K to 16K, capped scores
        dict(name="attn_b16_softcap", op="attn", B=16, Hq=32, Hkv=8, t_q=1, ctx=16384, ragged=True, code="e4m3",
             page=32, softcap=30.0, window=0, slopes=False),
        # checking five drafted tokens a sequence, distance bias, odd lengths
        dict(name="attn_draft5_bias", op="attn", B=7, Hq=32, Hkv=8, t_q=5, ctx=5003, ragged=True, code="int8",
             page=16, softcap=0.0, window=0, slopes=True),
        # the longest context of the LLaMA-7B multi-head layout
        dict(name="attn_131072_mha", op="attn", B=1, Hq=32, Hkv=32, t_q=1, ctx=131072, ragged=False, code="int8",
             page=128, softcap=0.0, window=0, slopes=False),
        # one new token for each of sixteen chats
        dict(name="append_b16_one_token", op="append", B=16, Hkv=8, t_new=1, ctx=9001, ragged=True, code="int8",
             page=64),
        # the rows of a 32K prompt on the multi-head layout
        dict(name="append_32k_mha", op="append", B=1, Hkv=32, t_new=32768, ctx=100, ragged=False, code="e4m3",
             page=64),
        # four samples from each of four prompts, then dropped again: all layers
        dict(name="pages_fork_free", op="pages", kind="fork", layers=32, Hkv=8, page=64, seqs=4, copies=4, ctx=4001,
             code="int8"),
        # closing the holes that every second chat left in the pool when it ended
        dict(name="pages_compact", op="pages", kind="compact", layers=8, Hkv=8, page=32, seqs=32, copies=1, ctx=3001,
             code="int8"),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "append", "attn", "attn", "pages"])
    Hkv, g = rng.choice([(1, 4), (8, 4), (8, 4), (8, 1), (32, 1), (4, 8), (2, 3)])
    if op == "prefill":
        B, t_q = rng.choice([1, 1, 2, 5]), _log_int(rng, 3, 9000)
        t_k = t_q if rng.random() < 0.7 else min(16384, t_q + _log_int(rng, 1, 8000))
        while B * Hkv * g * t_q * t_k > 32 * 8192 * 16384 // 2:      # the cost of the largest listed one
            B, t_q, t_k = max(1, B // 2), max(1, t_q * 2 // 3), max(1, t_k * 2 // 3)
        t_k = max(t_q, t_k)
        kind = rng.choice(["plain", "cap", "window", "bias", "docs", "prefix"])
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, t_q=t_q, t_k=t_k, ragged=rng.random() < 0.5,
                    softcap=rng.choice([20.0, 50.0]) if kind == "cap" else 0.0,
                    window=_log_int(rng, 1, 5000) if kind == "window" else 0, slopes=kind == "bias",
                    docs=rng.randint(2, 9) if kind == "docs" else 1,
                    prefix=rng.randint(1, t_k) if kind == "prefix" else 0)
    if op == "attn":
        B, ctx, t_q = rng.choice([1, 2, 5, 16, 33]), _log_int(rng, 9, 131072), rng.choice([1, 1, 1, 2, 3, 8])
        ctx = max(t_q, min(ctx, 131072 * 32 // (B * Hkv)))
        kind = rng.choice(["plain", "cap", "window", "bias"])
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, t_q=t_q, ctx=ctx, ragged=rng.random() < 0.5,
                    code=rng.choice(["int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]),
                    softcap=30.0 if kind == "cap" else 0.0, window=_log_int(rng, 1, 9000) if kind == "window" else 0,
                    slopes=kind == "bias")
    if op == "append":
        B = rng.choice([1, 2, 7, 16])
        t_new = rng.choice([1, 1, 2, 5]) if rng.random() < 0.4 else _log_int(rng, 1, 32768)
        t_new = max(1, min(t_new, 32768 * 32 // (B * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, t_new=t_new, ctx=_log_int(rng, 1, 9000), ragged=rng.random() < 0.5,
                    code=rng.choice(["int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]))
    kind = rng.choice(["fork", "compact", "copy"])
    return dict(op=op, kind=kind, layers=rng.choice([1, 4, 8]), Hkv=rng.choice([1, 2, 8]),
                page=rng.choice([16, 32, 64, 128]), seqs=rng.randint(1, 24), copies=rng.randint(1, 4),
                ctx=_log_int(rng, 5, 3000), code=rng.choice(["int8", "e4m3"]))


# ---- what a case's sequences look like -------------------------------------------------


def _spread(n, top, ragged):
    """Lengths of n sequences: all `top`, or from `top` down to half of it in odd steps."""
    if not ragged:
        return [top] * n
    return [max(1, top - (top // 2) * b // max(1, n - 1) - (b & 1 if top > 4 else 0)) for b in range(n)]


def _prefill_lengths(c):
    """(query rows, keys) of every sequence: the queries are the last positions."""
    q = _spread(c["B"], c["t_q"], c["ragged"])
    return q, [n + c["t_k"] - c["t_q"] for n in q]


def _rows_seen(c):
    """Per sequence, the first key and the prefix's end for every query row (whole numbers on the host)."""
    out = []
    for n, T in zip(*_prefill_lengths(c)):
        docs = c["docs"]
        cuts = [T * i * i // (docs * docs) for i in range(docs)]         # uneven documents
        first, end, at = [], [], 0
        for pos in range(T - n, T):
            while at + 1 < docs and pos >= cuts[at + 1]:
                at += 1
            first.append(cuts[at])
            end.append(min(c["prefix"], T))
        out.append((first, end))
    return out


def _attn_lengths(c):
    return [max(n, c["t_q"]) for n in _spread(c["B"], c["ctx"], c["ragged"])]


def _page_counts(c):
    lens = _spread(c["seqs"], c["ctx"], c["seqs"] > 1)
    return lens, [-(-n // c["page"]) for n in lens]


def work(c):
    op = c["op"]
    if op == "prefill":
        pairs = 0
        q, k = _prefill_lengths(c)
        for n, T, (first, end) in zip(q, k, _rows_seen(c)):
            for i, pos in enumerate(range(T - n, T)):
                lo = max(first[i], pos - c["window"] + 1 if c["window"] else 0)
                pairs += max(0, max(pos, end[i] - 1) - lo + 1)
        return {"bytes": 2 * D * (2 * sum(q) * c["Hq"] + 2 * sum(k) * c["Hkv"]), "flops": 4 * D * pairs * c["Hq"]}
    if op == "attn":
        lens = _attn_lengths(c)
        seen = [min(n, c["window"] + c["t_q"] - 1) if c["window"] else n for n in lens]
        pages = sum(-(-n // c["page"]) for n in seen)
        rows = c["B"] * c["t_q"] * c["Hq"]
        return {"bytes": sum(seen) * c["Hkv"] * 2 * D + pages * (8 * c["Hkv"] + 4) + rows * D * 4,
                "flops": 4 * D * sum(seen) * c["t_q"] * c["Hq"]}
    if op == "append":
        rows = sum(_spread(c["B"], c["t_new"], c["ragged"])) * c["Hkv"]
        # bf16 rows in, codes out, codes in again, bf16 rows out: keys and values
        return {"bytes": rows * 2 * (2 * D + D + D + 2 * D), "flops": rows * 8 * D}
    lens, counts = _page_counts(c)
    per_page = c["layers"] * c["Hkv"] * (c["page"] * D * 2 + 8)
    if c["kind"] == "fork":
        moved = sum(n % c["page"] != 0 for n in lens) * c["copies"]
        words = c["copies"] * sum(counts) * 4
    elif c["kind"] == "copy":
        moved, words = sum(counts), 2 * sum(counts)
    else:
        live = sum(n for i, n in enumerate(counts) if i % 2 == 0)
        moved, words = max(1, live // 2), 2 * sum(counts)     # about half of them lie behind the last hole
    return {"bytes": 2 * moved * per_page + 4 * words, "flops": 0}


# ---- inputs ----------------------------------------------------------------------------


def _codes(gen, code, shape):
    """Random 8-bit codes as they lie in a cache (a bell of about a third of the range), as bytes."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    x = (x * (QMAX[code] / 3.5)).clamp_(-QMAX[code], QMAX[code])
    return (x.round_().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)).view(torch.uint8)


def _pool(gen, code, layers, n_pages, Hkv, page):
    s = dict(k=_codes(gen, code, (layers, n_pages, Hkv, page, D)), v=_codes(gen, code, (layers, n_pages, Hkv, page, D)))
    for n in ("scale_k", "scale_v"):
        u = torch.rand((layers, n_pages, Hkv), generator=gen, device="cuda")
        s[n] = (2.5 + 2.0 * u) / QMAX[code]
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = dict(c=c)
    if c["op"] == "prefill":
        B, Hq, Hkv, t_q, t_k = c["B"], c["Hq"], c["Hkv"], c["t_q"], c["t_k"]
        st["q"] = _normal(gen, B, t_q, Hq, D, std=2.0)
        st["k"], st["v"] = _normal(gen, B, t_k, Hkv, D), _normal(gen, B, t_k, Hkv, D)
        q, k = _prefill_lengths(c)
        st["q_len"], st["kv_len"] = _ints(q), _ints(k)
        first = torch.zeros(B, t_q, dtype=torch.int32)
        end = torch.zeros(B, t_q, dtype=torch.int32)
        for b, (f, e) in enumerate(_rows_seen(c)):
            first[b, :len(f)], end[b, :len(e)] = torch.tensor(f, dtype=torch.int32), torch.tensor(e, dtype=torch.int32)
        st["first_key"] = first.cuda() if c["docs"] > 1 else None
        st["prefix_end"] = end.cuda() if c["prefix"] else None
        st["slopes"] = _slopes(Hq) if c["slopes"] else None
        st["out"] = torch.zeros(B, t_q, Hq, D, dtype=torch.bfloat16, device="cuda")
    elif c["op"] in ("attn", "append"):
        B, Hkv, page = c["B"], c["Hkv"], c["page"]
        if c["op"] == "attn":
            t_new, Hq = c["t_q"], c["Hq"]
            before = [n - t_new for n in _attn_lengths(c)]
        else:
            t_new, Hq = c["t_new"], Hkv
            before = _spread(B, c["ctx"], c["ragged"])
            st["t_new_b"] = _ints(_spread(B, t_new, c["ragged"]))
        max_pages = (max(before) + t_new) // page + 2
        n_pages = B * max_pages
        st.update(_pool(gen, c["code"], 1, n_pages, Hkv, page))
        st["page_table"] = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).view(B, max_pages)
        st["seq_len"] = _ints(before)
        st["refs"] = torch.ones(n_pages, dtype=torch.int32, device="cuda")
        if c["op"] == "attn":
            st["q"] = _normal(gen, B, t_new, Hq, D, std=2.0)
            st["slopes"] = _slopes(Hq) if c["slopes"] else None
            st["out"] = torch.zeros(B, t_new, Hq, D, dtype=torch.bfloat16, device="cuda")
        else:
            spread = 0.5 + 1.5 * torch.rand(B, t_new, Hkv, 1, generator=gen, device="cuda")    # loud and quiet tokens
            st["k_new"] = (_normal(gen, B, t_new, Hkv, D) * spread).to(torch.bfloat16)
            st["v_new"] = _normal(gen, B, t_new, Hkv, D)
            st["first"] = _ints([n // page * page for n in before])                  # the touched pages, read back
            st["count"] = st["seq_len"] + st["t_new_b"] - st["first"]
            t_read = t_new + page - 1
            st["k_out"] = torch.zeros(B, t_read, Hkv, D, dtype=torch.bfloat16, device="cuda")
            st["v_out"] = torch.zeros_like(st["k_out"])
    else:
        _prepare_pages(c, st, gen)
        B = st["page_table"].shape[0]
        Hq, Hkv, page, max_pages = c["Hkv"], c["Hkv"], c["page"], st["page_table"].shape[1]
        n_pages = st["refs"].shape[0]
    if own:
        import decode_attention_lrkv_b200 as L
        if c["op"] == "prefill":
            st["score"] = L.Score(softcap=c["softcap"], window=c["window"], slopes=st["slopes"],
                                  first_key=st["first_key"], prefix_end=st["prefix_end"])
        else:
            dims = L.PagedDims(B=B, Hq=Hq, Hkv=Hkv, d=D, page=page, n_pages=n_pages, max_pages=max_pages,
                               n_layers=c.get("layers", 1), code=c["code"])
            st["dims"], st["cache"] = dims, L.PagedCache(dims, **{n: st[n] for n in (
                "k", "v", "scale_k", "scale_v", "page_table", "seq_len", "refs")})
            if c["op"] == "attn":
                st["score"] = L.Score(softcap=c["softcap"], window=c["window"], slopes=st["slopes"])
                st["ws"] = L.make_paged_workspace(dims, c["t_q"])
            else:
                st["ws"] = L.make_paged_workspace(dims)
    return st


def _prepare_pages(c, st, gen):
    """A pool in use: sequences on scattered pages, and the call's lists."""
    n, page = c["seqs"], c["page"]
    lens, counts = _page_counts(c)
    extra = n * c["copies"] if c["kind"] == "fork" else 0
    n_pages = sum(counts) * (2 if c["kind"] == "copy" else 1) + extra + 8
    max_pages = max(counts) + 1
    st.update(_pool(gen, c["code"], c["layers"], n_pages, c["Hkv"], page))
    perm = torch.randperm(n_pages, generator=gen, device="cuda").cpu()
    table = torch.full((n + extra, max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    seq_len = torch.zeros(n + extra, dtype=torch.int32)
    at = 0
    for i, (T, m) in enumerate(zip(lens, counts)):
        mine = perm[at:at + m]
        at += m
        if c["kind"] == "compact" and i % 2:        # a chat that has ended: its pages are holes
            continue
        table[i, :m], seq_len[i], refs[mine] = mine.to(torch.int32), T, 1
    st["page_table"], st["refs"], st["seq_len"] = table.cuda(), refs.cuda(), seq_len.cuda()
    if c["kind"] == "fork":
        st["src"] = _ints([i // c["copies"] for i in range(extra)])
        st["dst"] = _ints([n + i for i in range(extra)])
    elif c["kind"] == "copy":
        m = sum(counts)
        st["src"], st["dst"] = perm[:m].to(torch.int32).cuda(), perm[m:2 * m].to(torch.int32).cuda()
    else:
        st["table0"], st["refs0"] = st["page_table"].clone(), st["refs"].clone()


# ---- one pass --------------------------------------------------------------------------


def run(st):
    c = st["c"]
    if own:
        return _run_own(c, st)
    if c["op"] == "prefill":
        return _plain_prefill(c, st)
    if c["op"] == "attn":
        return _plain_attn(c, st)
    if c["op"] == "append":
        return _plain_append(c, st)
    return _plain_pages(c, st)


def _run_own(c, st):
    import decode_attention_lrkv_b200 as L
    if c["op"] == "prefill":
        L.lrkv_prefill_attn(st["q"], st["k"], st["v"], st["out"], q_len=st["q_len"], kv_len=st["kv_len"],
                            score=st["score"])
        return st["out"]
    dims, cache, ws = st["dims"], st["cache"], st["ws"]
    if c["op"] == "attn":
        L.lrkv_paged_attn(dims, cache, 0, st["q"], st["out"], score=st["score"], ws=ws)
        return st["out"]
    if c["op"] == "append":
        L.lrkv_paged_append(dims, cache, 0, st["k_new"], st["v_new"], t_new_b=st["t_new_b"])
        L.lrkv_paged_read(dims, cache, 0, st["first"], st["count"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if c["kind"] == "copy":
        L.lrkv_pages_copy(dims, cache, st["src"], st["dst"], ws=ws)
        return {n: st[n] for n in ("k", "v", "scale_k", "scale_v")}
    if c["kind"] == "fork":
        L.lrkv_pages_fork(dims, cache, st["src"], st["dst"], ws=ws)
        forked = {"table": st["page_table"].clone(), "refs": st["refs"].clone(), "lens": st["seq_len"].clone()}
        L.lrkv_pages_free(dims, cache, st["dst"])
        return {**forked, "refs_after": st["refs"], "k": st["k"], "v": st["v"], "scale_k": st["scale_k"],
                "scale_v": st["scale_v"]}
    st["page_table"].copy_(st["table0"])      # the same holes every time
    st["refs"].copy_(st["refs0"])
    L.lrkv_pages_compact(dims, cache, ws=ws)
    return {"table": st["page_table"], "refs": st["refs"], **_live(st)}


def _live(st):
    return {n: st[n] for n in ("k", "v", "scale_k", "scale_v")}


def _attend(q, k, v, lo, hi, pos, T, softcap, slopes):
    """Softmax attention in fp32: q [B,t_q,Hq,d], k and v [B,T,Hkv,d] fp32; row i of sequence b sees keys lo..hi."""
    B, t_q, Hq, d = q.shape
    Hkv = k.shape[2]
    q = q.float().view(B, t_q, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)         # [B,Hkv,g,t_q,d]
    s = torch.matmul(q, k.permute(0, 2, 3, 1).unsqueeze(2))                      # [B,Hkv,g,t_q,T]
    s.mul_(1.0 / math.sqrt(d))
    if softcap:
        s.div_(softcap).tanh_().mul_(softcap)
    j = torch.arange(T, device=q.device, dtype=torch.int32)
    if slopes is not None:
        dist = (pos[:, :, None] - j).abs().float()                               # [B,t_q,T]
        s.addcmul_(slopes.view(1, Hkv, Hq // Hkv, 1, 1), dist[:, None, None], value=-1.0)
    hidden = (j < lo[:, :, None]) | (j > hi[:, :, None])
    s.masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min_(-3e38)
    s.sub_(m).exp_()
    o = torch.matmul(s, v.permute(0, 2, 1, 3).unsqueeze(2)) / s.sum(-1, keepdim=True).clamp_min_(1e-37)
    return o.permute(0, 3, 1, 2, 4).reshape(B, t_q, Hq, d)


def _plain_prefill(c, st):
    B, t_q, t_k = c["B"], c["t_q"], c["t_k"]
    i = torch.arange(t_q, device="cuda", dtype=torch.int32)
    pos = (st["kv_len"] - st["q_len"])[:, None] + i
    lo = torch.zeros_like(pos) if st["first_key"] is None else st["first_key"].clone()
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    hi = pos if st["prefix_end"] is None else torch.maximum(pos, st["prefix_end"] - 1)
    hi = torch.minimum(hi, st["kv_len"][:, None] - 1)
    o = _attend(st["q"], st["k"].float(), st["v"].float(), lo, hi, pos, t_k, c["softcap"], st["slopes"])
    return torch.where((i < st["q_len"][:, None])[:, :, None, None], o.to(torch.bfloat16), st["out"])


def _values(st, code, name, layer, pages):
    """fp32 values [B, positions, Hkv, d] of the pages [B, n] of one layer."""
    codes = st[name].view(torch.int8 if code == "int8" else torch.float8_e4m3fn)[layer][pages].float()
    x = codes * st["scale_" + name][layer][pages][..., None, None]
    B, n, Hkv, page, d = x.shape
    return x.permute(0, 1, 3, 2, 4).reshape(B, n * page, Hkv, d)


def _plain_attn(c, st):
    pages = st["page_table"].long()
    T = pages.shape[1] * c["page"]
    pos = st["seq_len"][:, None] + torch.arange(c["t_q"], device="cuda", dtype=torch.int32)
    lo = pos - c["window"] + 1 if c["window"] else torch.zeros_like(pos)
    k, v = _values(st, c["code"], "k", 0, pages), _values(st, c["code"], "v", 0, pages)
    return _attend(st["q"], k, v, lo, pos, pos, T, c["softcap"], st["slopes"]).to(torch.bfloat16)


def _round_codes(x, code):
    """x, in units of its scale, as codes (nearest, ties to even), in fp32."""
    x = x.clamp(-QMAX[code], QMAX[code])
    return x.round() if code == "int8" else x.to(torch.float8_e4m3fn).float()


def _plain_append(c, st):
    B, t_new, page, code = c["B"], c["t_new"], c["page"], c["code"]
    start, n = st["seq_len"].long(), st["t_new_b"].long()
    W = (t_new + page - 2) // page + 1                                           # pages that a row can touch
    at = (start // page)[:, None] + torch.arange(W, device="cuda")
    pages = st["page_table"].long().gather(1, at)                                # [B,W]
    r = torch.arange(W * page, device="cuda") - (start % page)[:, None]          # row of the call, by place
    new = ((r >= 0) & (r < n[:, None])).view(B, W, 1, page, 1)
    old = (r < 0).view(B, W, 1, page, 1)
    kind = torch.int8 if code == "int8" else torch.float8_e4m3fn
    _put(st, "k", pages, r, new, old, kind, c)
    _put(st, "v", pages, r, new, old, kind, c)
    return {"k": _plain_read(c, st, "k"), "v": _plain_read(c, st, "v")}


def _put(st, name, pages, r, new, old, kind, c):
    B, t_new, page, code = c["B"], c["t_new"], c["page"], c["code"]
    W, Hkv = pages.shape[1], c["Hkv"]
    x = st[name + "_new"].float().nan_to_num(0.0, BIG, -BIG)
    x = x.gather(1, r.clamp(0, t_new - 1)[:, :, None, None].expand(-1, -1, Hkv, D))
    x = x.view(B, W, page, Hkv, D).permute(0, 1, 3, 2, 4)                        # [B,W,Hkv,page,d]
    amax = torch.where(new, x.abs(), torch.zeros_like(x)).amax((-1, -2))
    had = st["scale_" + name][0][pages]                                          # [B,W,Hkv]
    before = torch.where(old[..., 0].any(-1).expand_as(had), had, torch.zeros_like(had))
    s = torch.maximum(before, amax / torch.full_like(amax, QMAX[code]))       # a true quotient: ties go by it
    s = torch.where(s < TINY, torch.zeros_like(s), s)
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = st[name].view(kind)[0][pages].float()
    again = torch.where((s > before)[..., None, None], _round_codes(codes * (before * inv)[..., None, None], code), codes)
    got = torch.where(new, _round_codes(x * inv[..., None, None], code), torch.where(old, again, codes))
    st[name].view(kind)[0][pages] = got.to(kind)
    st["scale_" + name][0][pages] = torch.where(new[..., 0].any(-1).expand_as(s), s, had)


def _plain_read(c, st, name):
    page, t = c["page"], st["k_out"].shape[1]
    i = torch.arange(t, device="cuda")
    place = st["first"].long()[:, None] + i
    pages = st["page_table"].long().gather(1, (place // page).clamp_max(st["page_table"].shape[1] - 1))
    kind = torch.int8 if c["code"] == "int8" else torch.float8_e4m3fn
    x = st[name].view(torch.uint8)[0][pages, :, place % page].view(kind).float()  # [B,t,Hkv,d]
    x = (x * st["scale_" + name][0][pages][..., None]).to(torch.bfloat16)
    return torch.where((i < st["count"][:, None])[:, :, None, None], x, st[name + "_out"])


def _move(st, src, dst):
    """Copies whole pages of every layer."""
    st["k"][:, dst], st["v"][:, dst] = st["k"][:, src], st["v"][:, src]
    st["scale_k"][:, dst], st["scale_v"][:, dst] = st["scale_k"][:, src], st["scale_v"][:, src]


def _plain_pages(c, st):
    page = c["page"]
    if c["kind"] == "copy":
        _move(st, st["src"].long(), st["dst"].long())
        return {n: st[n] for n in ("k", "v", "scale_k", "scale_v")}
    table, refs, lens = st["page_table"], st["refs"], st["seq_len"]
    if c["kind"] == "fork":
        src, dst = st["src"].long(), st["dst"].long()
        T = lens[src]
        full = T // page
        slot = torch.arange(table.shape[1], device="cuda")
        rows = torch.where(slot < full[:, None], table[src], torch.full_like(table[src], -1))
        refs.index_add_(0, rows.clamp_min(0).view(-1).long(), (rows >= 0).to(torch.int32).view(-1))
        part = (T % page != 0).nonzero()[:, 0]                                   # forks that need a page of their own
        fresh = (refs == 0).nonzero()[:part.shape[0], 0]
        at = full[part].long()
        _move(st, table[src[part], at].long(), fresh)
        rows[part, at] = fresh.to(torch.int32)
        refs[fresh] = 1
        table[dst], lens[dst] = rows, T
        forked = {"table": table.clone(), "refs": refs.clone(), "lens": lens.clone()}
        mine = table[dst]
        refs.index_add_(0, mine.clamp_min(0).view(-1).long(), -(mine >= 0).to(torch.int32).view(-1))
        table[dst] = -1
        lens[dst] = 0
        return {**forked, "refs_after": refs, "k": st["k"], "v": st["v"], "scale_k": st["scale_k"],
                "scale_v": st["scale_v"]}
    table.copy_(st["table0"])
    refs.copy_(st["refs0"])
    live = refs > 0
    n = live.sum()
    index = torch.arange(refs.shape[0], device="cuda")
    src, dst = (live & (index >= n)).nonzero()[:, 0], (~live & (index < n)).nonzero()[:, 0]
    _move(st, src, dst)
    to = index.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table))
    return {"table": table, "refs": refs, **_live(st)}


# ---- the same results from the definitions, in 64 bits ---------------------------------


def exact(c, seed):
    if c["op"] == "pages":
        return None                        # whole numbers only: they have to be equal
    st = prepare(c, seed)
    return {"prefill": _exact_prefill, "attn": _exact_attn, "append": _exact_append}[c["op"]](c, st)


def _exact_rows(c, q, k, v, h, first, end, T, n):
    """Rows of one sequence and query head: q [n,d], k and v [T,d], all fp64."""
    pos = torch.arange(T - n, T, device="cuda")[:, None]
    key = torch.arange(T, device="cuda")[None, :]
    s = q @ k.T / math.sqrt(D)
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    if c["slopes"]:
        s = s - float(torch.tensor(2.0 ** (-8.0 * (h + 1) / c["Hq"]))) * (pos - key).abs()
    seen = (key <= pos) | (key < end[:, None])
    seen &= key >= first[:, None]
    if c["window"]:
        seen &= pos - key < c["window"]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.max(1, keepdim=True).values.clamp_min(-1e300))
    return (p @ v) / p.sum(1, keepdim=True).clamp_min(1e-300)


def _exact_prefill(c, st):
    out = st["out"].double()
    g = c["Hq"] // c["Hkv"]
    q_len, kv_len = _prefill_lengths(c)
    seen = _rows_seen(c)
    for b in range(c["B"]):
        n, T = q_len[b], kv_len[b]
        first, end = (torch.tensor(x, device="cuda") for x in seen[b])
        for h in range(c["Hq"]):
            out[b, :n, h] = _exact_rows(c, st["q"][b, :n, h].double(), st["k"][b, :T, h // g].double(),
                                        st["v"][b, :T, h // g].double(), h, first, end, T, n)
    return out


def _exact_cache(c, st, name, b, h, T):
    """Values [T, d] of one sequence and kv head, fp64."""
    kind = torch.int8 if c["code"] == "int8" else torch.float8_e4m3fn
    ids = st["page_table"][b, :-(-T // c["page"])].long()
    x = st[name].view(kind)[0][ids, h].double() * st["scale_" + name][0][ids, h].double()[:, None, None]
    return x.reshape(-1, D)[:T]


def _exact_attn(c, st):
    out = st["out"].double()
    g, n = c["Hq"] // c["Hkv"], c["t_q"]
    zero = torch.zeros(n, dtype=torch.long, device="cuda")
    for b, T in enumerate(_attn_lengths(c)):
        for kv in range(c["Hkv"]):
            k, v = (_exact_cache(c, st, name, b, kv, T) for name in "kv")
            for h in range(kv * g, kv * g + g):
                out[b, :, h] = _exact_rows(c, st["q"][b, :, h].double(), k, v, h, zero, zero, T, n)
    return out


def _single(x):
    """fp64 values rounded to fp32 (a quotient or product of fp32 values, taken in fp64, rounds here once)."""
    return x.to(torch.float32).double()


def _exact_append(c, st):
    page, Q, code = c["page"], QMAX[c["code"]], c["code"]
    kind = torch.int8 if code == "int8" else torch.float8_e4m3fn
    got = {"k": st["k_out"].double(), "v": st["v_out"].double()}
    counts = _spread(c["B"], c["t_new"], c["ragged"])
    starts = _spread(c["B"], c["ctx"], c["ragged"])
    for name in "kv":
        for b, (start, n) in enumerate(zip(starts, counts)):
            x = st[name + "_new"][b, :n].double()
            first, stop = start // page * page, -(-(start + n) // page) * page
            rows = torch.zeros(stop - first, c["Hkv"], D, dtype=torch.float64, device="cuda")
            rows[start - first:start - first + n] = x
            blocks = rows.view(-1, page, c["Hkv"], D)
            s = _single(blocks.abs().amax((1, 3)) / Q)                           # [blocks, Hkv]
            held = start - first
            if held:
                id0 = int(st["page_table"][b, first // page])
                before = st["scale_" + name][0, id0].double()
                s[0] = torch.maximum(s[0], before)
            s = torch.where(s < TINY, torch.zeros_like(s), s)
            inv = torch.where(s > 0, _single(1.0 / s), torch.zeros_like(s))
            t = _single(blocks * inv[:, None, :, None]).clamp(-Q, Q)
            codes = t.round() if code == "int8" else t.to(torch.float32).to(kind).double()
            if held:
                had = st[name].view(kind)[0, id0].double()[:, :held]             # [Hkv, held, d]
                t = _single(had * _single(before * inv[0])[:, None, None]).clamp(-Q, Q)
                t = t.round() if code == "int8" else t.to(torch.float32).to(kind).double()
                again = torch.where((s[0] > before)[:, None, None], t, had)
                codes[0, :held] = again.permute(1, 0, 2)
            value = (codes * s[:, None, :, None]).reshape(-1, c["Hkv"], D)
            m = start + n - first
            got[name][b, :m] = value[:m]
    return got
