"""lrkv_paged_append, _read and _attn against the definitions (bounds: serve_testutil)."""
import pytest
import torch

import decode_attention_lrkv_b200 as L
from oracle import serve as R
from tests import serve_testutil as U

pytestmark = pytest.mark.gpu
CANARY = 123.0


def make(B, Hq, Hkv, page, lens, code, room=8, n_layers=1, seed=1, codes=None):
    """A cache of sequences of the given lengths on scattered pages, with random contents."""
    max_pages = (max(lens) + room) // page + 1
    n_pages = B * max_pages + 3
    D = L.PagedDims(B=B, Hq=Hq, Hkv=Hkv, d=128, page=page, n_pages=n_pages, max_pages=max_pages, n_layers=n_layers,
                    code=code)
    c = L.PagedCache(D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k, c.v):
        x = (torch.randn(t.shape, generator=g, device="cuda") * R.QMAX[code] / 3.5).clamp(-R.QMAX[code], R.QMAX[code])
        t.copy_((x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)).view(torch.uint8))
    for t in (c.scale_k, c.scale_v):
        t.copy_((2.5 + 2 * torch.rand(t.shape, generator=g, device="cuda")) / R.QMAX[code])
    perm = torch.randperm(n_pages, generator=g, device="cuda")[:B * max_pages]
    c.page_table.copy_(perm.to(torch.int32).view(B, max_pages))
    c.refs[perm] = 1
    c.seq_len.copy_(U.ints(lens))
    return D, c


def values(c, name, layer, b, h, T):
    """fp64 values [T, d] that the cache holds."""
    D = c.dims
    ids = c.page_table[b, :-(-T // D.page)].long()
    x = getattr(c, name).view(R.KIND[D.code])[layer, ids, h].double()
    return (x * getattr(c, "scale_" + name)[layer, ids, h].double()[:, None, None]).reshape(-1, 128)[:T]


def attn(D, c, q, t_q_b=None, score=None, layer=0, ws=None, out=None):
    out = torch.full_like(q, CANARY) if out is None else out
    ws = L.make_paged_workspace(D, q.shape[1]) if ws is None else ws
    L.lrkv_paged_attn(D, c, layer, q, out, t_q_b=None if t_q_b is None else U.ints(t_q_b), score=score, ws=ws)
    torch.cuda.synchronize()
    return out


def check(out, D, c, q, t_q_b=None, score=None, layer=0):
    score, g, t_q = score or L.Score(), D.Hq // D.Hkv, q.shape[1]
    err = size = 0.0
    for b in range(D.B):
        n = t_q if t_q_b is None else t_q_b[b]
        start = int(c.seq_len[b])
        T = start + n
        pos = torch.arange(start, T, device="cuda")
        for kv in range(D.Hkv):
            k, v = values(c, "k", layer, b, kv, T), values(c, "v", layer, b, kv, T)
            for h in range(kv * g, kv * g + g):
                # weights are rounded to f16 (2^-11), below 2^-14 to steps of 2^-24; queries enter exactly
                # but for 2^-28 of a row's largest element; int8 codes enter the sums with 1152 added
                shift = 1152.0 if D.code == "int8" else 0.0
                sk = float(c.scale_k[layer].max())
                e = 2 * 128 * 2.0 ** -24 * shift * q[b, :n, h].double().abs().sum(1) * sk * (score.scale or 128 ** -0.5)
                e = e + 2.0 ** -28 * q[b, :n, h].double().abs().amax(1, keepdim=True)[:, 0] * \
                    (k.abs().sum(1).max() if T else 0) * (score.scale or 128 ** -0.5)
                a, s = U.check_rows(out[b, :n, h], q[b, :n, h], k, v, pos, T, score, h, b, 2 * 2.0 ** -11,
                                    floor=2.0 ** -25 + shift * 2.0 ** -24 / 127, extra_score=e)
                err, size = err + a, size + s
        assert bool((out[b, n:] == CANARY).all())
    assert err <= size * U.U ** 2 + 1e-30, (err / size) ** 0.5


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000])
def test_single_token_lengths(before, page, code):
    D, c = make(1, 8, 2, page, [before], code)
    q = U.normal(3, 1, 1, 8, 128, std=2.0)
    check(attn(D, c, q), D, c, q)
    assert int(c.dev_status[0]) == 0


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,t_q", [(1, 1, 1), (3, 1, 1), (8, 8, 3), (7, 1, 1), (16, 2, 2), (6, 2, 5), (8, 2, 6),
                                        (8, 1, 4), (8, 1, 64), (5, 1, 13), (4, 4, 64)])
def test_heads_and_rows(Hq, Hkv, t_q, code):
    """From one row of a kv head to row blocks of several CTAs."""
    lens = [700, 0, 45]
    D, c = make(3, Hq, Hkv, 32, lens, code, room=t_q)
    q = U.normal(4, 3, t_q, Hq, 128, std=2.0)
    check(attn(D, c, q), D, c, q)
    some = [t_q, max(0, t_q - 1), 0]
    check(attn(D, c, q, some), D, c, q, some)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_ragged_batches_split_over_many_ctas(page, code):
    lens = [5000, 0, 3, 2999, 64, 1, 4096]
    D, c = make(7, 8, 2, page, lens, code)
    q = U.normal(5, 7, 3, 8, 128, std=2.0)
    ws = L.make_paged_workspace(D, 3)
    first = attn(D, c, q, ws=ws)
    check(first, D, c, q)
    assert torch.equal(attn(D, c, q, ws=ws), first)         # the workspace is as it was, the result the same


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,Hkv,t_q", [(8, 2, 3), (8, 2, 4), (4, 1, 5), (8, 1, 4), (8, 1, 9)])
def test_rows_of_a_cache_larger_than_l2(Hq, Hkv, t_q, page, code):
    """12 to 72 rows of a kv head, in blocks of up to 32: the table has room for a long context."""
    lens = [900, 2, 0, 333]
    D, c = make(4, Hq, Hkv, page, lens, code, room=t_q)
    wide = L.PagedDims(B=4, Hq=Hq, Hkv=Hkv, d=128, page=page, n_pages=D.n_pages, max_pages=8000000 // page, code=code)
    table = torch.full((4, wide.max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, :D.max_pages] = c.page_table
    w = L.PagedCache(wide, k=c.k, v=c.v, scale_k=c.scale_k, scale_v=c.scale_v, refs=c.refs, seq_len=c.seq_len,
                     page_table=table)
    q = U.normal(4, 4, t_q, Hq, 128, std=2.0)
    for s in (L.Score(), L.Score(window=250, slopes=U.slopes(Hq), softcap=30.0)):
        some = [t_q, t_q, t_q - 1, 0]
        check(attn(wide, w, q, some, s), D, c, q, some, s)


def test_long_context():
    D, c = make(1, 4, 1, 128, [70000], "int8")
    q = U.normal(6, 1, 1, 4, 128, std=2.0)
    check(attn(D, c, q), D, c, q)


def test_many_short_sequences():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 90, (1200,), generator=g).tolist()
    D, c = make(1200, 2, 1, 16, lens, "e4m3")
    q = U.normal(7, 1200, 2, 2, 128, std=2.0)
    some = [(i * 7) % 3 for i in range(1200)]
    out = attn(D, c, q, some)
    for b in range(1200):
        assert bool((out[b, some[b]:] == CANARY).all())
    pick = list(range(0, 1200, 37)) + [1199]
    sub = L.PagedDims(B=len(pick), Hq=2, Hkv=1, d=128, page=16, n_pages=D.n_pages, max_pages=D.max_pages, code="e4m3")
    view = L.PagedCache(sub, k=c.k, v=c.v, scale_k=c.scale_k, scale_v=c.scale_v, refs=c.refs,
                        page_table=c.page_table[pick].contiguous(), seq_len=c.seq_len[pick].contiguous())
    check(out[pick], sub, view, q[pick], [some[b] for b in pick])


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("score", [dict(softcap=20.0), dict(softcap=2.0), dict(softcap=1e5), dict(window=1), dict(window=33), dict(window=500),
                                   dict(scale=0.3), dict(bias=True), dict(bias=True, softcap=30.0, window=700)], ids=str)
def test_score_modifiers(score, code):
    score = dict(score)
    D, c = make(3, 8, 2, 16, [900, 31, 0], code)
    s = L.Score(slopes=U.slopes(8) if score.pop("bias", False) else None, **score)
    q = U.normal(8, 3, 4, 8, 128, std=2.0)
    check(attn(D, c, q, score=s), D, c, q, score=s)


def test_documents_and_prefix():
    D, c = make(2, 4, 2, 32, [600, 40], "int8")
    q = U.normal(9, 2, 5, 4, 128, std=2.0)
    first = U.ints([[0, 300, 602, 10 ** 9, 604], [41, 41, 41, 41, 0]])   # past a row's position: it sees nothing
    end = U.ints([[0, 605, 0, 0, 3], [0, 0, 45, 44, 0]])
    for s in (L.Score(first_key=first), L.Score(prefix_end=end), L.Score(first_key=first, prefix_end=end)):
        out = attn(D, c, q, score=s)
        check(out, D, c, q, score=s)
    assert bool((attn(D, c, q, score=L.Score(first_key=first))[0, 3] == 0).all())
    none = L.Score(first_key=torch.full((2, 5), 10 ** 9, dtype=torch.int32, device="cuda"))
    assert bool((attn(D, c, q, score=none) == 0).all())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_what_lies_behind_a_sequence_is_not_used(code):
    D, c = make(2, 4, 2, 64, [70, 64], code, room=64)
    q = U.normal(10, 2, 1, 4, 128)
    want = attn(D, c, q)
    for b, T in ((0, 71), (1, 65)):
        last = int(c.page_table[b, T // 64])
        for t in (c.k, c.v):
            t[:, last, :, T % 64:] = 0x7F                    # NaN as e4m3
        c.page_table[b, T // 64 + 1:] = 10 ** 9              # entries that no token needs
    assert torch.equal(attn(D, c, q), want)
    assert int(c.dev_status[0]) == 0


@pytest.mark.parametrize("code,page", [("int8", 16), ("e4m3", 16), ("int8", 64), ("e4m3", 128)])
def test_bad_pages_are_skipped(code, page):
    D, c = make(1, 4, 1, page, [6 * page + 3], code)
    q = U.normal(11, 1, 1, 4, 128)
    c.k[:, D.n_pages - 1], c.v[:, D.n_pages - 1] = 0x7F, 0x7F
    c.page_table[0, 1], c.page_table[0, 4] = -1, D.n_pages
    out = attn(D, c, q)
    assert int(c.dev_status[0]) == L.DEV_BAD_PAGE
    T = 6 * page + 4
    keep = [i for i in range(T) if i // page not in (1, 4)]
    c.page_table[0, 1] = c.page_table[0, 4] = 0
    for h in range(4):
        k, v = values(c, "k", 0, 0, 0, T)[keep], values(c, "v", 0, 0, 0, T)[keep]
        at = torch.tensor([len(keep) - 1], device="cuda")
        ref = R.attend(q[0, :, h], k, v, at, torch.zeros_like(at), at)
        U.close(out[0, :, h], ref, (2 * 2.0 ** -11, U.score_error(ref, 0) + 5e-3, 2.0 ** -24 + 1e-6))


def test_table_shorter_than_the_sequence():
    D, c = make(1, 4, 1, 16, [30], "int8", room=1)           # two pages: 32 positions
    c.seq_len.fill_(31)
    q = U.normal(12, 1, 3, 4, 128)
    out = attn(D, c, q)                                      # rows at 31, 32, 33; keys 0 .. 31
    assert int(c.dev_status[0]) == L.DEV_SEQ_OVERFLOW
    k, v = values(c, "k", 0, 0, 0, 32), values(c, "v", 0, 0, 0, 32)
    pos = torch.tensor([31, 32, 33], device="cuda")
    for h in range(4):
        ref = R.attend(q[0, :, h], k, v, pos, torch.zeros_like(pos), pos.clamp_max(31))
        U.close(out[0, :, h], ref, (2 * 2.0 ** -11, U.score_error(ref, 0) + 5e-3, 2.0 ** -24 + 1e-6))
    c.dev_status.zero_()
    attn(D, c, q, [4])
    assert int(c.dev_status[0]) & L.DEV_BAD_COUNT


def test_scales_and_queries_far_from_one():
    for scale, q_std in ((1e-30, 1.0), (1e4, 1e-4), (1e-6, 1e6), (0.0, 1.0)):
        D, c = make(1, 4, 1, 32, [200], "int8")
        c.scale_k.mul_(scale)
        c.scale_v.mul_(1e-20)
        c.scale_v[0, ::2] *= 1e12                            # pages whose values differ by 12 orders
        q = U.normal(13, 1, 1, 4, 128, std=q_std)
        q[..., :64] *= 2.0 ** -9
        check(attn(D, c, q), D, c, q)


def test_pool_past_4_gib():
    """Pages whose codes lie past 2^32 bytes."""
    page, Hkv = 128, 8
    n_pages = 2 ** 32 // (page * Hkv * 128) + 40
    D = L.PagedDims(B=1, Hq=16, Hkv=Hkv, d=128, page=page, n_pages=n_pages, max_pages=4, code="e4m3")
    shape = (1, n_pages, Hkv, page, 128)
    c = L.PagedCache(D, k=torch.empty(shape, dtype=torch.uint8, device="cuda"),
                     v=torch.empty(shape, dtype=torch.uint8, device="cuda"))
    c.page_table.copy_(U.ints([[n_pages - 1, 5, n_pages - 30, n_pages - 2]]))
    new = U.normal(14, 1, 400, Hkv, 128), U.normal(15, 1, 400, Hkv, 128)
    L.lrkv_paged_append(D, c, 0, *new)
    back = torch.zeros_like(new[0]), torch.zeros_like(new[1])
    L.lrkv_paged_read(D, c, 0, None, U.ints([400]), *back)
    for x, y in zip(new, back):
        assert float((x.float() - y.float()).abs().max()) <= 2 ** -4 * float(x.float().abs().max())
    c.seq_len.fill_(399)
    q = U.normal(16, 1, 1, 16, 128)
    check(attn(D, c, q), D, c, q)


# ---- append and read -----------------------------------------------------------------


def mirror_append(D, host, layer, new, start, n, table):
    """The append of one sequence on host copies {k, v, scale_k, scale_v}."""
    for name, rows in new.items():
        for page_i in range(start // D.page, -(-(start + n) // D.page)):
            first = page_i * D.page
            if page_i >= D.max_pages or n == 0:
                continue
            pid = int(table[page_i])
            if not 0 <= pid < D.n_pages:
                continue
            lo, hi = max(start, first), min(start + n, first + D.page)
            for h in range(D.Hkv):
                codes = host[name].view(R.KIND[D.code])[layer, pid, h].float()
                got, s = R.append_page(codes, host["scale_" + name][layer, pid, h], rows[lo - start:hi - start, h],
                                       lo - first, D.code)
                host[name].view(R.KIND[D.code])[layer, pid, h] = got.to(R.KIND[D.code])
                host["scale_" + name][layer, pid, h] = s


def same(D, c, host):
    for name in ("k", "v"):
        assert torch.equal(c.__dict__["scale_" + name].cpu(), host["scale_" + name])
        # codes by value: the two zeros of e4m3 are one value
        a, b = (t.view(R.KIND[D.code]).float() for t in (getattr(c, name).cpu(), host[name]))
        assert torch.equal(torch.nan_to_num(a, nan=999.0), torch.nan_to_num(b, nan=999.0))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("t_new", [1, 5, 40, 300])
def test_append_is_exact(t_new, page, code):
    lens = [0, 1, page - 1, page, 3 * page + 7]
    D, c = make(5, 2, 2, page, lens, code, room=t_new, n_layers=2)
    k, v = U.normal(20, 5, t_new, 2, 128), U.normal(21, 5, t_new, 2, 128, std=0.3)
    k[1] *= 8                                                # louder than what is there: codes are rounded again
    k[4, :, 1] *= 0.01
    v[2] = 0
    some = [t_new, t_new, max(t_new - 1, 1), t_new, 0]
    host = {n: getattr(c, n).cpu().clone() for n in ("k", "v", "scale_k", "scale_v")}
    for b in range(5):
        mirror_append(D, host, 1, {"k": k[b, :some[b]].cpu(), "v": v[b, :some[b]].cpu()}, lens[b], some[b],
                      c.page_table[b].cpu())
    L.lrkv_paged_append(D, c, 1, k, v, t_new_b=U.ints(some))
    torch.cuda.synchronize()
    same(D, c, host)
    assert int(c.dev_status[0]) == 0 and c.seq_len.tolist() == lens


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_of_odd_values(code):
    """Infinities, NaN, zeros, subnormals and the largest numbers; ties."""
    D, c = make(4, 1, 1, 16, [3, 16, 0, 5], code, room=16)
    x = U.normal(22, 4, 16, 1, 128)
    x[0, 0, 0, 0], x[0, 1, 0, 1], x[0, 2, 0, 2] = float("inf"), float("nan"), float("-inf")
    x[1] *= 2.0 ** -120                                      # a scale that counts as zero
    x[2] = torch.arange(128, device="cuda").to(torch.bfloat16) - 63.5
    x[2, :, 0, 0] = 127
    x[3] = 3e38
    host = {n: getattr(c, n).cpu().clone() for n in ("k", "v", "scale_k", "scale_v")}
    for b in range(4):
        mirror_append(D, host, 0, {"k": x[b].cpu(), "v": -x[b].cpu()}, int(c.seq_len[b]), 16, c.page_table[b].cpu())
    L.lrkv_paged_append(D, c, 0, x, -x)
    torch.cuda.synchronize()
    same(D, c, host)


def test_append_past_the_table_and_onto_bad_pages():
    D, c = make(3, 1, 1, 16, [20, 20, 20], "int8", room=10)  # two pages a sequence
    c.page_table[1, 1] = -1
    c.page_table[2, 1] = D.n_pages + 5
    k = U.normal(23, 3, 40, 1, 128)
    host = {n: getattr(c, n).cpu().clone() for n in ("k", "v", "scale_k", "scale_v")}
    for b in range(3):
        mirror_append(D, host, 0, {"k": k[b].cpu(), "v": k[b].cpu()}, 20, 40, c.page_table[b].cpu())
    L.lrkv_paged_append(D, c, 0, k, k)
    torch.cuda.synchronize()
    same(D, c, host)
    assert int(c.dev_status[0]) == L.DEV_SEQ_OVERFLOW | L.DEV_BAD_PAGE


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_read_is_exact(page, code):
    D, c = make(4, 3, 3, page, [200, 333, 64, 9], code)
    first, count = [0, 130, 63, 3], [200, 203, 1, 0]
    k, v = (torch.full((4, 210, 3, 128), CANARY, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.lrkv_paged_read(D, c, 0, U.ints(first), U.ints(count), k, v)
    torch.cuda.synchronize()
    for b in range(4):
        for h in range(3):
            for name, got in (("k", k), ("v", v)):
                # an 8-bit code times an fp32 scale, rounded to fp32 and then to bf16, as specified
                ids = c.page_table[b].long()
                x = getattr(c, name).view(R.KIND[code])[0, ids, h].float() * getattr(c, "scale_" + name)[0, ids, h][:, None, None]
                x = x.reshape(-1, 128)[first[b]:first[b] + count[b]].to(torch.bfloat16)
                assert torch.equal(got[b, :count[b], h], x)
        assert bool((k[b, count[b]:] == CANARY).all()) and bool((v[b, count[b]:] == CANARY).all())
    c.page_table[0, 0] = -1
    k.fill_(CANARY)
    L.lrkv_paged_read(D, c, 0, None, U.ints([page + 1, 0, 0, 999]), k, v)
    torch.cuda.synchronize()
    assert bool((k[0, :page] == CANARY).all()) and not bool((k[0, page] == CANARY).all())
    assert int(c.dev_status[0]) & (L.DEV_BAD_PAGE | L.DEV_BAD_COUNT) == L.DEV_BAD_PAGE | L.DEV_BAD_COUNT


def test_two_captured_graphs_with_a_workspace_each():
    D, c = make(2, 8, 2, 32, [3000, 500], "int8", room=16)
    q = U.normal(30, 2, 1, 8, 128, std=2.0)
    want = attn(D, c, q)
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [L.make_paged_workspace(D) for _ in range(2)]
    graphs = [U.graph_of(lambda i=i: L.lrkv_paged_attn(D, c, 0, q, outs[i], ws=ws[i])) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # a replay sees the cache as it is then
    c.seq_len.copy_(U.ints([100, 501]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], attn(D, c, q))
