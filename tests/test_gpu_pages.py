"""lrkv_pages_* against the rules on host lists, and a whole serving run."""
import random

import pytest
import torch

import decode_attention_lrkv_b200 as L
from oracle import serve as R
from tests import serve_testutil as U
from tests.test_gpu_paged import attn, check

pytestmark = pytest.mark.gpu


def filled(B, page, n_pages, max_pages, n_layers=2, Hkv=2, code="int8", seed=1):
    D = L.PagedDims(B=B, Hq=2 * Hkv, Hkv=Hkv, d=128, page=page, n_pages=n_pages, max_pages=max_pages, n_layers=n_layers,
                    code=code)
    c = L.PagedCache(D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8))
    for t in (c.scale_k, c.scale_v):
        t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
    return D, c, L.make_paged_workspace(D)


def host(c):
    return R.Pool(c.page_table.tolist(), c.refs.tolist(), c.seq_len.tolist(), c.dims.page)


def same(c, pool, before):
    """Counts, table, lengths and status as the rules say; pages moved and no others touched."""
    torch.cuda.synchronize()
    assert c.page_table.tolist() == pool.table
    assert c.refs.tolist() == pool.refs
    assert c.seq_len.tolist() == pool.len
    assert int(c.dev_status[0]) == pool.status
    for name, was in before.items():
        want = was.clone()
        for s, d in pool.moves:
            want[:, d] = was[:, s]
        assert torch.equal(getattr(c, name), want)
    pool.moves = []


def contents(c):
    return {n: getattr(c, n).clone() for n in ("k", "v", "scale_k", "scale_v")}


def set_state(c, table, refs, lens):
    c.page_table.copy_(U.ints(table))
    c.refs.copy_(U.ints(refs))
    c.seq_len.copy_(U.ints(lens))


def random_state(c, seed, share=0.0):
    """Sequences of random lengths on scattered pages, the first pages of some shared."""
    D, rng = c.dims, random.Random(seed)
    free = list(range(D.n_pages))
    rng.shuffle(free)
    table, refs, lens = [], [0] * D.n_pages, []
    for b in range(D.B):
        n = rng.choice([0, 0, rng.randint(1, D.max_pages * D.page)])
        row = []
        if n and b and rng.random() < share:
            for p in table[rng.randrange(b)][:min(rng.randint(0, 3), n // D.page)]:
                if p < 0:
                    break
                row.append(p)
        while len(row) < -(-n // D.page) and free:
            row.append(free.pop())
        n = min(n, len(row) * D.page)
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (D.max_pages - len(row)))
        lens.append(n)
    set_state(c, table, refs, lens)


@pytest.mark.parametrize("B,page,n_pages,max_pages", [(1, 16, 5, 5), (7, 16, 40, 9), (30, 32, 200, 12), (1500, 16, 9001, 7)])
def test_reserve_advance_free(B, page, n_pages, max_pages):
    D, c, ws = filled(B, page, n_pages, max_pages, n_layers=1, Hkv=1)
    rng = random.Random(B)
    pool, before = host(c), contents(c)
    for step in range(12):
        counts = [rng.choice([0, 1, 1, 2, 17, 40]) for _ in range(B)]
        if step % 3 == 2:
            seqs = [rng.randrange(B) for _ in range(max(1, B // 2))]
            L.lrkv_pages_free(D, c, U.ints(seqs))
            pool.free(seqs)
            same(c, pool, before)
        one = step % 2 == 0
        t = max(counts)
        L.lrkv_pages_reserve(D, c, t, None if one else U.ints(counts))
        counts = [t] * B if one else counts
        pool.reserve(counts)
        same(c, pool, before)
        fits = [n if all(p >= 0 for p in pool.table[b][:min(-(-(pool.len[b] + n) // page), max_pages)]) else 0
                for b, n in enumerate(counts)]
        L.lrkv_pages_advance(D, c, t, U.ints(fits))
        over = any(pool.len[b] + n > max_pages * page for b, n in enumerate(fits))
        pool.advance(fits)
        pool.status |= 0x2 if over else 0
        same(c, pool, before)


def test_reserve_twice_takes_pages_once():
    D, c, ws = filled(2, 16, 10, 4)
    for _ in range(2):
        L.lrkv_pages_reserve(D, c, 20)
    assert c.page_table.tolist() == [[0, 1, -1, -1], [2, 3, -1, -1]] and c.refs.tolist() == [1] * 4 + [0] * 6
    L.lrkv_pages_reserve(D, c, 33, U.ints([33, 99]))          # the second count is out of range: 33
    assert c.page_table.tolist() == [[0, 1, 4, -1], [2, 3, 5, -1]]
    assert int(c.dev_status[0]) == L.DEV_BAD_COUNT


@pytest.mark.parametrize("n_layers,Hkv,page", [(1, 1, 16), (3, 2, 32), (2, 8, 128)])
def test_fork(n_layers, Hkv, page):
    D, c, ws = filled(12, page, 80, 8, n_layers, Hkv)
    for seed in range(6):
        random_state(c, seed, share=0.5)
        c.dev_status.zero_()
        pool, before = host(c), contents(c)
        rng = random.Random(seed)
        n = rng.choice([1, 5, 40])
        src, dst = [rng.randint(-1, 12) for _ in range(n)], [rng.randint(-1, 12) for _ in range(n)]
        L.lrkv_pages_fork(D, c, U.ints(src), U.ints(dst), ws=ws)
        pool.fork(src, dst)
        same(c, pool, before)


def test_fork_when_the_pool_runs_out():
    D, c, ws = filled(6, 16, 6, 4)
    set_state(c, [[1, 3, -1, -1]] + [[-1] * 4] * 5, [0, 1, 0, 1, 0, 0], [20, 0, 0, 0, 0, 0])
    c.refs.copy_(U.ints([0, 1, 1, 1, 1, 0]))                   # two are free
    pool, before = host(c), contents(c)
    L.lrkv_pages_fork(D, c, U.ints([0] * 4), U.ints([5, 2, 4, 1]), ws=ws)
    pool.fork([0] * 4, [5, 2, 4, 1])
    assert pool.status == L.DEV_NO_PAGES
    same(c, pool, before)


def test_fork_then_free_leaves_the_pool_as_it_was():
    D, c, ws = filled(8, 32, 60, 6)
    random_state(c, 3)
    c.seq_len[5:] = 0
    c.page_table[5:] = -1
    refs = torch.zeros(D.n_pages, dtype=torch.int32, device="cuda")
    for p in c.page_table[:5].flatten().tolist():
        if p >= 0:
            refs[p] += 1
    c.refs.copy_(refs)
    L.lrkv_pages_fork(D, c, U.ints([0, 1, 1]), U.ints([5, 6, 7]), ws=ws)
    L.lrkv_pages_free(D, c, U.ints([7, 5, 6]))
    assert torch.equal(c.refs, refs) and int(c.dev_status[0]) == 0


@pytest.mark.parametrize("n_pages", [5, 64, 1000, 9000])
def test_compact(n_pages):
    D, c, ws = filled(10, 16, n_pages, 40, n_layers=2, Hkv=1)
    for seed in range(4):
        random_state(c, seed, share=0.3)
        pool, before = host(c), contents(c)
        for _ in range(2):                                    # the second time there is nothing to do
            L.lrkv_pages_compact(D, c, ws=ws)
            pool.compact()
            same(c, pool, before)
            before = contents(c)
        live = sum(r > 0 for r in pool.refs)
        assert all(r > 0 for r in pool.refs[:live]) and not any(pool.refs[live:])


def test_compact_of_empty_and_full_pools():
    D, c, ws = filled(2, 16, 7, 4)
    for refs in ([0] * 7, [1] * 7, [0] * 6 + [1], [1] + [0] * 6):
        set_state(c, [[-1] * 4] * 2, refs, [0, 0])
        pool, before = host(c), contents(c)
        L.lrkv_pages_compact(D, c, ws=ws)
        pool.compact()
        same(c, pool, before)


@pytest.mark.parametrize("n", [1, 3, 30, 500])
def test_copy(n):
    D, c, ws = filled(2, 32, 700, 4, n_layers=3)
    for seed in range(3):
        rng = random.Random(seed + n)
        ids = list(range(700))
        rng.shuffle(ids)
        src, dst = [rng.choice(ids[:200]) for _ in range(n)], ids[200:200 + n]
        if seed:                                              # entries that break the rules
            for _ in range(n // 3 + 1):
                i = rng.randrange(n)
                what = rng.randrange(4)
                if what == 0:
                    src[i] = rng.choice([-1, 700, 10 ** 9])
                elif what == 1:
                    dst[i] = rng.choice([-1, 700, -10 ** 9])
                elif what == 2:
                    dst[i] = dst[rng.randrange(n)]
                else:
                    src[i] = dst[rng.randrange(n)]
        c.dev_status.zero_()
        pool, before = host(c), contents(c)
        L.lrkv_pages_copy(D, c, U.ints(src), U.ints(dst), ws=ws)
        pool.copy(src, dst)
        same(c, pool, before)


def test_calls_leave_the_workspace_as_they_need_it():
    """Attention, fork, copy and compact in turn on one workspace, captured and replayed."""
    D, c, ws = filled(6, 32, 90, 12, n_layers=1, Hkv=2)
    random_state(c, 5)
    c.k.random_(0, 100)
    c.v.random_(0, 100)
    c.seq_len[4:], c.page_table[4:] = 0, -1
    refs = torch.zeros(90, dtype=torch.int32)
    for p in c.page_table.flatten().tolist():
        if p >= 0:
            refs[p] += 1
    c.refs.copy_(refs)
    q, out = U.normal(1, 6, 1, 4, 128), torch.zeros(6, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    src, dst, free = U.ints([0, 1, 9, 1]), U.ints([4, 5, 3, 4]), U.ints([4, 5])
    far = U.ints([0, 0]), U.ints([88, 88])

    def step():
        L.lrkv_pages_fork(D, c, src, dst, ws=ws)
        L.lrkv_paged_attn(D, c, 0, q, out, ws=ws)
        L.lrkv_pages_free(D, c, free)
        L.lrkv_pages_compact(D, c, ws=ws)
        L.lrkv_pages_copy(D, c, *far, ws=ws)

    step()
    torch.cuda.synchronize()
    first, state = out.clone(), (c.page_table.tolist(), c.refs.tolist(), c.seq_len.tolist())
    g = U.graph_of(step)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert (c.page_table.tolist(), c.refs.tolist(), c.seq_len.tolist()) == state


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_a_serving_run(code):
    """Prompts are prefilled, cached in 8 bits, forked, extended token by token (once with drafted
    tokens), freed and compacted; a later chunk of a prompt attends to what is read back."""
    B, Hq, Hkv, page, n_layers = 5, 8, 2, 16, 2
    D = L.PagedDims(B=B, Hq=Hq, Hkv=Hkv, d=128, page=page, n_pages=60, max_pages=20, n_layers=n_layers, code=code)
    c, ws = L.PagedCache(D), L.make_paged_workspace(D, 4)
    score = L.Score(softcap=30.0, window=150)
    prompt = [100, 37, 0, 0, 0]
    t = max(prompt)
    n = U.ints(prompt)

    def tokens(seed, t):
        return U.normal(seed, B, t, Hq, 128, std=2.0), U.normal(seed + 1, B, t, Hkv, 128), U.normal(seed + 2, B, t, Hkv, 128)

    # prompts
    L.lrkv_pages_reserve(D, c, t, n)
    for layer in range(n_layers):
        q, k, v = tokens(10 * layer, t)
        out = torch.zeros_like(q)
        L.lrkv_prefill_attn(q, k, v, out, q_len=n, kv_len=n, score=score)
        L.lrkv_paged_append(D, c, layer, k, v, t_new_b=n)
    L.lrkv_pages_advance(D, c, t, n)
    # two samples from the first prompt
    L.lrkv_pages_fork(D, c, U.ints([0, 0]), U.ints([2, 4]), ws=ws)
    assert c.seq_len.tolist() == [100, 37, 100, 0, 100]
    # decode steps, one of them with drafted tokens
    for step, t_new in enumerate((1, 1, 4, 1)):
        counts = [t_new, t_new, t_new, 0, 1]
        L.lrkv_pages_reserve(D, c, t_new, U.ints(counts))
        for layer in range(n_layers):
            q, k, v = tokens(100 * step + 10 * layer + 50, t_new)
            L.lrkv_paged_append(D, c, layer, k, v, t_new_b=U.ints(counts))
            out = attn(D, c, q, counts, score, layer, ws)
            check(out, D, c, q, counts, score, layer)
        L.lrkv_pages_advance(D, c, t_new, U.ints(counts))
    assert c.seq_len.tolist() == [107, 44, 107, 0, 104]
    shared = c.page_table[0, :6].tolist()
    assert c.page_table[2, :6].tolist() == shared and c.refs[shared].tolist() == [3] * 6
    # the first prompt's owner ends; the pool closes up; the others go on
    before = [attn(D, c, q, [0, 1, 1, 0, 1], score, 1, ws)]
    L.lrkv_pages_free(D, c, U.ints([0]))
    L.lrkv_pages_compact(D, c, ws=ws)
    after = attn(D, c, q, [0, 1, 1, 0, 1], score, 1, ws)
    assert torch.equal(before[0], after)
    live = int((c.refs > 0).sum())
    assert bool((c.refs[:live] > 0).all()) and int(c.page_table.max()) == live - 1
    # a second chunk for sequence 1: its keys and values are read back and attended to beside the new ones
    old, new = 44, 70
    kk, vv = (torch.zeros(B, old + new, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.lrkv_paged_read(D, c, 1, None, U.ints([0, old, 0, 0, 0]), kk, vv)
    q, k, v = tokens(999, new)
    kk[1, old:], vv[1, old:] = k[1], v[1]
    out = torch.zeros_like(q)
    L.lrkv_prefill_attn(q[1:2], kk[1:2], vv[1:2], out[1:2], score=score)
    pos = torch.arange(old, old + new, device="cuda")
    for h in range(Hq):
        U.check_rows(out[1, :, h], q[1, :, h], kk[1, :, h // 4], vv[1, :, h // 4], pos, old + new, score, h, 0, U.U)
    assert int(c.dev_status[0]) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    D, c, ws = filled(2, 16, 4, 2)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    other = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=32, n_pages=4, max_pages=2, n_layers=2)
    with pytest.raises(ValueError, match="shape"):
        L.lrkv_paged_append(D, c, 0, bf(2, 1, 4, 128), bf(2, 1, 4, 128))
    with pytest.raises(ValueError, match="made for"):
        L.lrkv_pages_reserve(other, c, 1)
    with pytest.raises(ValueError, match="CUDA"):
        L.lrkv_pages_free(D, c, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="uint8"):
        L.lrkv_pages_compact(D, c, ws=ws.view(torch.int32))
    with pytest.raises(ValueError, match="dst"):
        L.lrkv_pages_copy(D, c, U.ints([0, 1]), U.ints([2]), ws=ws)
    with pytest.raises(ValueError, match="slopes"):
        L.lrkv_paged_attn(D, c, 0, bf(2, 1, 4, 128), bf(2, 1, 4, 128), score=L.Score(slopes=U.slopes(3)), ws=ws)
    with pytest.raises(ValueError, match="CUDA"):
        L.lrkv_prefill_attn(bf(1, 4, 4, 128), bf(1, 4, 2, 128), bf(1, 4, 2, 128).cpu(), bf(1, 4, 4, 128))
    with pytest.raises(L.LrkvError):
        L.lrkv_paged_attn(D, c, 2, bf(2, 1, 4, 128), bf(2, 1, 4, 128), ws=ws)
    with pytest.raises(L.LrkvError):
        L.lrkv_pages_compact(D, c)


@pytest.mark.parametrize("scored", [False, True])
def test_both_paths_of_the_binding_do_the_same(scored):
    """Ordinary calls are marshalled in C++; an explicit stream takes the Python path."""
    from decode_attention_lrkv_b200 import serve as S
    here = torch.cuda.current_stream()
    results = []
    for stream in (None, here):
        D, c, ws = filled(6, 16, 90, 12, n_layers=2)
        for t in (c.k, c.v):
            t.zero_()
        q, k, v = U.normal(1, 6, 40, 4, 128), U.normal(2, 6, 40, 2, 128), U.normal(3, 6, 40, 2, 128)
        n = U.ints([40, 3, 17, 0, 0, 0])
        score = L.Score(slopes=U.slopes(4), window=30) if scored else L.Score(softcap=20.0)
        out, out1 = torch.zeros_like(q), torch.zeros(6, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
        kk, vv = torch.zeros_like(k), torch.zeros_like(v)
        kw = dict(stream=stream)
        L.lrkv_prefill_attn(q, k, v, out, q_len=n, kv_len=n, score=score, **kw)
        L.lrkv_pages_reserve(D, c, 41, n + 1, **kw)
        L.lrkv_paged_append(D, c, 1, k, v, t_new_b=n, **kw)
        L.lrkv_pages_advance(D, c, 40, n, **kw)
        L.lrkv_paged_read(D, c, 1, None, n, kk, vv, **kw)
        L.lrkv_pages_fork(D, c, U.ints([0, 1]), U.ints([4, 5]), ws=ws, **kw)
        L.lrkv_pages_free(D, c, U.ints([1]), **kw)
        L.lrkv_pages_compact(D, c, ws=ws, **kw)
        L.lrkv_pages_copy(D, c, U.ints([0]), U.ints([80]), ws=ws, **kw)
        L.lrkv_paged_append(D, c, 1, k[:, :1].contiguous(), v[:, :1].contiguous(), **kw)
        L.lrkv_paged_attn(D, c, 1, q[:, :1].contiguous(), out1, score=score, ws=ws, **kw)
        torch.cuda.synchronize()
        results.append([out, out1, kk, vv, *(getattr(c, f).clone() for f in c.FIELDS)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    # what each of them takes
    assert S._calls.counts(1, D, c, 0, None, None) == 0 and S._calls.counts(1, D, c, 0, None, here) == -1
    twin = L.PagedDims(**{f: getattr(D, f) for f in ("B", "Hq", "Hkv", "d", "page", "n_pages", "max_pages", "n_layers", "code")})
    assert S._calls.counts(1, twin, c, 0, None, None) == -1      # equal, but another object
    L.lrkv_pages_advance(twin, c, 0)
    assert S._calls.append(D, c, 1, k.float(), v, None, None) == -1
    assert S._calls.append(D, c, 2 ** 40, k, v, None, None) == -1
    assert S._calls.append(D, c, 7, k, v, None, None) == L.LRKV_ERR_INVALID_ARG
    assert S._calls.append(D, object(), 1, k, v, None, None) == -1 and S._calls.append(D) == -1
    assert S._calls.attn(D, c, 1, q, q.cpu(), None, score, ws, None) == -1
    assert S._calls.attn(D, c, 1, q, out, None, 3, ws, None) == -1
    assert S._calls.prefill(q, k, v[:, :5], out, None, None, None, None, None, None) == -1
    assert S._calls.lists(3, D, c, None, None, ws.view(torch.int8), None) == -1
