"""Calls of the serving operators that the other tests do not make: wrong devices, sequences whose
pages ran out, rejected drafts, weights far below the largest one, numbers that are not finite."""
import random

import pytest
import torch

import decode_attention_lrkv_b200 as L
from oracle import serve as R
from tests import serve_testutil as U
from tests.test_gpu_paged import attn, check, make, mirror_append, values
from tests.test_gpu_paged import same as same_codes
from tests.test_gpu_pages import contents, filled, host, random_state, same, set_state

pytestmark = pytest.mark.gpu
CANARY = 123.0


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("name", L.PagedCache.FIELDS)
def test_a_cache_with_a_tensor_of_the_host_is_refused(name):
    D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=4, max_pages=2)
    c, ws, one = L.PagedCache(D), L.make_paged_workspace(D), U.ints([0])
    c.__dict__[name] = getattr(c, name).cpu()
    here = torch.cuda.current_stream()
    for kw in ({}, {"stream": here}):
        for call in (lambda: L.lrkv_paged_append(D, c, 0, bf(2, 1, 2, 128), bf(2, 1, 2, 128), **kw),
                     lambda: L.lrkv_paged_read(D, c, 0, None, U.ints([1, 1]), bf(2, 1, 2, 128), bf(2, 1, 2, 128), **kw),
                     lambda: L.lrkv_paged_attn(D, c, 0, bf(2, 1, 4, 128), bf(2, 1, 4, 128), ws=ws, **kw),
                     lambda: L.lrkv_pages_reserve(D, c, 1, **kw), lambda: L.lrkv_pages_advance(D, c, 1, **kw),
                     lambda: L.lrkv_pages_fork(D, c, one, one, ws=ws, **kw), lambda: L.lrkv_pages_free(D, c, one, **kw),
                     lambda: L.lrkv_pages_copy(D, c, one, one, ws=ws, **kw), lambda: L.lrkv_pages_compact(D, c, ws=ws, **kw)):
            with pytest.raises(ValueError, match="CUDA tensor"):
                call()


# ---- sequences that got no pages -----------------------------------------------------


@pytest.mark.parametrize("B,page,max_pages", [(1, 16, 3), (9, 16, 40), (40, 128, 5), (300, 32, 70)])
def test_advance_stops_where_pages_are_missing(B, page, max_pages):
    D, c, ws = filled(B, page, B * max_pages + 5, max_pages, n_layers=1, Hkv=1)
    for seed in range(6):
        rng = random.Random(seed)
        random_state(c, seed)
        table = c.page_table.tolist()
        for b in range(B):
            have = rng.randint(0, max_pages)
            table[b][:have] = [rng.randrange(D.n_pages) for _ in range(have)]
            if rng.random() < 0.3:
                table[b][rng.randrange(max_pages)] = rng.choice([-1, D.n_pages, 10 ** 9, -5])
        c.page_table.copy_(U.ints(table))
        c.dev_status.zero_()
        pool, before = host(c), contents(c)
        counts = [rng.choice([0, 1, 2, page, rng.randint(0, page * max_pages)]) for _ in range(B)]
        one = seed == 5
        L.lrkv_pages_advance(D, c, max(counts), None if one else U.ints(counts))
        pool.advance([max(counts)] * B if one else counts)
        same(c, pool, before)


def test_a_pool_that_runs_out_in_the_middle_of_a_run():
    """The steps of a serving loop on a pool that is full: once another sequence has gone, the one
    that had to wait goes on where it stopped, and sees nothing of what its new page held before."""
    D = L.PagedDims(B=2, Hq=4, Hkv=2, d=128, page=16, n_pages=3, max_pages=4)
    c, ws = L.PagedCache(D), L.make_paged_workspace(D)
    k, v = U.normal(1, 2, 32, 2, 128), U.normal(2, 2, 32, 2, 128) * 50
    n = U.ints([16, 32])
    L.lrkv_pages_reserve(D, c, 32, n)
    L.lrkv_paged_append(D, c, 0, k, v, t_new_b=n)
    L.lrkv_pages_advance(D, c, 32, n)
    assert c.seq_len.tolist() == [16, 32] and int(c.dev_status[0]) == 0
    one = U.ints([1, 0])

    def step(seed):
        L.lrkv_pages_reserve(D, c, 1, one)
        k1, v1 = U.normal(seed, 2, 1, 2, 128), U.normal(seed + 1, 2, 1, 2, 128)
        L.lrkv_paged_append(D, c, 0, k1, v1, t_new_b=one)
        q = U.normal(seed + 2, 2, 1, 4, 128)
        out = attn(D, c, q, [1, 0], ws=ws)
        L.lrkv_pages_advance(D, c, 1, one)
        return q, out, k1, v1

    for i in range(2):
        step(10 + i)
        assert c.seq_len.tolist() == [16, 32] and c.page_table[0].tolist() == [0, -1, -1, -1]
    assert int(c.dev_status[0]) == L.DEV_NO_PAGES | L.DEV_BAD_PAGE
    c.dev_status.zero_()
    L.lrkv_pages_free(D, c, U.ints([1]))
    q, out, k1, v1 = step(20)
    assert c.seq_len.tolist() == [17, 0] and int(c.dev_status[0]) == 0
    c.seq_len[0] = 16
    check(out, D, c, q, [1, 0])
    # the new page's scale is that of its one token alone
    page = int(c.page_table[0, 1])
    assert torch.equal(c.scale_v[0, page].cpu(), (v1[0, 0].float().abs().amax(1).cpu() / torch.full((2,), 127.0)))


def test_fork_of_a_source_without_its_last_page():
    for bad in (-1, 60, 10 ** 9):
        D, c, ws = filled(5, 16, 60, 4)
        set_state(c, [[3, bad, -1, -1], [4, 5, -1, -1]] + [[-1] * 4] * 3, [0] * 3 + [1] * 3 + [0] * 54, [20, 30, 0, 0, 0])
        pool, before = host(c), contents(c)
        L.lrkv_pages_fork(D, c, U.ints([0, 1, 0]), U.ints([2, 3, 4]), ws=ws)
        pool.fork([0, 1, 0], [2, 3, 4])
        assert pool.len == [20, 30, 0, 30, 0] and pool.status == L.DEV_BAD_PAGE
        same(c, pool, before)


# ---- numbers -------------------------------------------------------------------------


def small_codes(T, page, kstd, vtop, q, seed):
    """One kv head of int8 keys of deviation 1 (kstd codes) and values of -vtop .. vtop codes."""
    n = T // page + 1
    D = L.PagedDims(B=1, Hq=q.shape[2], Hkv=1, d=128, page=page, n_pages=n, max_pages=n, code="int8")
    c = L.PagedCache(D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = (torch.randn(n * page, 128, generator=g, device="cuda") * kstd).clamp(-127, 127).round()
    v = torch.randint(-vtop, vtop + 1, (n * page, 128), generator=g, device="cuda")
    for name, x in (("k", k), ("v", v)):
        getattr(c, name).copy_(x.to(torch.int8).view(torch.uint8).view(n, page, 128)[None, :, None])
    c.scale_k.fill_(1 / kstd), c.scale_v.fill_(1.0)
    c.page_table.copy_(torch.arange(n, device="cuda")), c.seq_len.fill_(T - 1)
    return D, c, k[:T].double() * float(c.scale_k[0, 0, 0]), v[:T].double()


@pytest.mark.parametrize("T,page", [(64, 64), (8192, 16), (65536, 64), (200000, 128)])
@pytest.mark.parametrize("kstd,sign", [(36.0, False), (2.0, True)])
def test_small_codes_over_many_tokens(T, page, kstd, sign):
    """Values of a few code steps on pages whose scale a louder token has set, and queries of one
    sign: what the shift of int8 codes adds has to leave the sums without a trace.  The output is a
    sum of values of random signs, so independent errors of the weights are off it by 2^-11 / sqrt 3
    relative to it, the last rounding by 2^-8 / sqrt 3 at most (root mean square); fp32 sums of
    codes below 2^8 have ten bits to spare.  2^-8 holds for all together."""
    q = U.normal(5, 1, 1, 8, 128)
    q = q.abs() if sign else q
    D, c, k, v = small_codes(T, page, kstd, 1, q, 1)
    out = attn(D, c, q)
    pos = torch.tensor([T - 1], device="cuda")
    err = size = 0.0
    for h in range(8):
        ref = R.attend(q[0, :, h], k, v, pos, pos * 0, pos)[0]
        err, size = err + float(((out[0, :, h].double() - ref) ** 2).sum()), size + float((ref ** 2).sum())
    assert err <= size * U.U ** 2, (err / size) ** 0.5


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,t_q", [(4, 1), (4, 8)])
def test_many_weights_far_below_the_largest_one(Hq, t_q, page):
    """The first key of every 32 has a value of zero and lies 15 to 20 nats above the others, whose
    weights are all that the output is made of.  A weight of 2^-21 of the largest one or more is off
    by 2^-11 of itself, a smaller one by 2^-32 of the largest (half of f16's smallest step, lifted 2^7)."""
    T = 3000
    D = L.PagedDims(B=1, Hq=Hq, Hkv=1, d=128, page=page, n_pages=200, max_pages=200, code="e4m3")
    c = L.PagedCache(D)
    k, v = torch.zeros(200 * page, 128, device="cuda"), 1 + torch.rand(200 * page, 128, device="cuda")
    k[::32, 0], v[::32] = 16.0, 0.0
    for name, x in (("k", k), ("v", v)):
        getattr(c, name).copy_(x.to(torch.float8_e4m3fn).view(torch.uint8).view(200, page, 128)[None, :, None])
    c.scale_k.fill_(1.0), c.scale_v.fill_(1.0)
    c.page_table.copy_(torch.arange(200, device="cuda")), c.seq_len.fill_(T - t_q)
    q = bf(1, t_q, Hq, 128)
    for i, nats in enumerate((15.0, 16.0, 17.4, 20.0)):
        q[:, :, i, 0] = nats * 128 ** 0.5 / 16
    out = attn(D, c, q)
    keys, vals = k.double(), v.to(torch.float8_e4m3fn).double()
    pos = torch.arange(T - t_q, T, device="cuda")
    for h in range(Hq):
        assert float(out[0, :, h].abs().min()) > 0
        U.check_rows(out[0, :, h], q[0, :, h], keys[:T], vals[:T], pos, T, L.Score(), h, 0, 2 * 2.0 ** -11, floor=2.0 ** -32)


@pytest.mark.parametrize("t_q,t_k", [(300, 300), (40, 6000)])    # the second one splits the keys
@pytest.mark.parametrize("score", [dict(), dict(softcap=20.0), dict(window=80)], ids=str)
def test_a_prefill_hands_nan_on(t_q, t_k, score):
    """Rows with a NaN of their own, or that see a NaN key, are NaN; the others are as they were."""
    q, k, v = U.normal(1, 1, t_q, 4, 128), U.normal(2, 1, t_k, 2, 128), U.normal(3, 1, t_k, 2, 128)
    first = torch.zeros(1, t_q, dtype=torch.int32, device="cuda")
    first[0, 9] = 10 ** 9                                      # a row that sees nothing, its query NaN
    s = L.Score(first_key=first, **score)
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    L.lrkv_prefill_attn(q, k, v, want, score=s)
    at = t_k - 20                                              # seen by the last 20 rows (a window: by some)
    q[0, 3, 1], q[0, 9], k[0, at, 0, 5] = float("nan"), float("nan"), float("nan")
    L.lrkv_prefill_attn(q, k, v, got, score=s)
    nan = torch.zeros(t_q, 4, dtype=torch.bool)
    nan[3, 1] = True
    nan[t_q - 20:, :2] = True                                  # heads 0 and 1 read kv head 0
    nan = nan.cuda()
    assert bool(got[0][nan].isnan().all()) and torch.equal(got[0][~nan], want[0][~nan])
    assert bool((got[0, 9] == 0).all())
    k[:] = float("nan")                                        # nothing but NaN
    L.lrkv_prefill_attn(q, k, v, got, score=s)
    keep = torch.arange(t_q, device="cuda") != 9
    assert bool(got[0][keep].isnan().all()) and bool((got[0, 9] == 0).all())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,t_q", [([20, 3000], 3), ([5, 40], 9)])
def test_the_paged_attention_hands_nan_on(lens, t_q, code):
    D, c = make(2, 8, 2, 32, lens, code, room=t_q)
    q = U.normal(1, 2, t_q, 8, 128)
    first = torch.zeros(2, t_q, dtype=torch.int32, device="cuda")
    first[:, 1] = 10 ** 9
    s = L.Score(first_key=first)
    want = attn(D, c, q, score=s)
    nan = torch.zeros(2, t_q, 8, dtype=torch.bool, device="cuda")
    nan[0, 0, 3] = nan[1, 2, 7] = nan[:, 1] = True
    q[nan] = float("nan")
    got = attn(D, c, q, score=s)
    nan[:, 1] = False                                          # these see nothing
    assert bool(got[nan].isnan().all()) and torch.equal(got[~nan], want[~nan]) and bool((got[:, 1] == 0).all())


def test_windows_wider_than_any_sequence():
    """The widest window hides nothing, in front of the first key too (more rows than keys)."""
    q, k, v = U.normal(1, 2, 80, 4, 128), U.normal(2, 2, 60, 2, 128), U.normal(3, 2, 60, 2, 128)
    end = torch.full((2, 80), 30, dtype=torch.int32, device="cuda")
    for n in (2 ** 31 - 1, 2 ** 25 + 1, 2 ** 25, 2 ** 24):
        for e in (end, None):
            want, got = torch.zeros_like(q), torch.zeros_like(q)
            L.lrkv_prefill_attn(q, k, v, want, score=L.Score(prefix_end=e))
            L.lrkv_prefill_attn(q, k, v, got, score=L.Score(window=n, prefix_end=e))
            assert torch.equal(got, want) and bool((want[:, :20] == 0).all()) == (e is None)
    D, c = make(2, 4, 2, 32, [200, 3], "int8")
    q = U.normal(4, 2, 2, 4, 128)
    assert torch.equal(attn(D, c, q, score=L.Score(window=2 ** 31 - 1)), attn(D, c, q))


def test_a_status_word_of_another_type_is_refused():
    q, k, v = bf(1, 4, 4, 128), bf(1, 4, 2, 128), bf(1, 4, 2, 128)
    for bad in (torch.zeros(4, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda"), U.ints([])):
        with pytest.raises(ValueError, match="dev_status"):
            L.lrkv_prefill_attn(q, k, v, torch.zeros_like(q), dev_status=bad)
    L.lrkv_prefill_attn(q, k, v, torch.zeros_like(q), dev_status=U.ints([0]))


def test_the_longest_lists_of_sequences():
    D, c, ws = filled(300, 16, 900, 6, n_layers=1, Hkv=1)
    random_state(c, 1)
    n, rng = 2 ** 16, random.Random(2)
    pool, before = host(c), contents(c)
    src, dst = [rng.randint(-1, 300) for _ in range(n)], [rng.randint(-1, 300) for _ in range(n)]
    L.lrkv_pages_fork(D, c, U.ints(src), U.ints(dst), ws=ws)
    pool.fork(src, dst)
    same(c, pool, before)
    before = contents(c)
    seqs = [rng.randint(-1, 200) for _ in range(n)]
    L.lrkv_pages_free(D, c, U.ints(seqs))
    pool.free(seqs)
    same(c, pool, before)


def test_dims_are_no_score():
    D, c = make(2, 4, 2, 32, [5, 9], "int8")
    q = U.normal(1, 2, 1, 4, 128)
    with pytest.raises(TypeError, match="a Score is needed"):
        attn(D, c, q, score=D)
    with pytest.raises(TypeError, match="a Score is needed"):
        L.lrkv_prefill_attn(q, q, q, torch.zeros_like(q), score=D)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_rejected_drafts_leave_their_mark_on_a_page_that_goes_on(page, code):
    """Five drafted tokens, the last three loud; two are accepted and others appended over the rest.
    The page's scale stays what the loud ones made it, but a page that starts anew forgets them."""
    lens = [page + 4, page, 2 * page - 3]                   # on a page, at its start, over its end
    D, c = make(3, 2, 2, page, lens, code, room=12)
    before = c.scale_k.clone()
    host = {n: getattr(c, n).cpu().clone() for n in ("k", "v", "scale_k", "scale_v")}

    def append(seed, t, loud):
        k, v = U.normal(seed, 3, t, 2, 128), U.normal(seed + 1, 3, t, 2, 128)
        k[:, 2:] *= loud
        for b in range(3):
            mirror_append(D, host, 0, {"k": k[b].cpu(), "v": v[b].cpu()}, int(c.seq_len[b]), t, c.page_table[b].cpu())
        L.lrkv_paged_append(D, c, 0, k, v)
        same_codes(D, c, host)

    append(1, 5, 50.0)
    loud = c.scale_k.clone()
    c.seq_len += U.ints([2, 0, 3])                            # none of the second one's is accepted
    append(3, 3, 1.0)
    at = [int(c.page_table[b, 1]) for b in range(3)]
    assert torch.equal(c.scale_k[0, at[0]], loud[0, at[0]]) and bool((loud[0, at[0]] > before[0, at[0]]).all())
    assert bool((c.scale_k[0, at[1]] < loud[0, at[1]]).all())
    over = int(c.page_table[2, 2])                            # its first page ends with three accepted tokens
    assert bool((c.scale_k[0, over] < loud[0, over]).all())
    check(attn(D, c, U.normal(9, 3, 3, 2, 128)), D, c, U.normal(9, 3, 3, 2, 128))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_scores_past_what_fp32_counts_singly(code):
    """Scores of some 10^8, where a step of fp32 is 8 or more: a key far above the others, wherever
    it lies, is the output, and equal scores weigh the same on both sides of such a key."""
    D, c = make(1, 4, 1, 32, [3000], code)
    c.scale_v.fill_(1 / 64), c.scale_k.fill_(1.0)
    for top in (5, 1500, 2999):
        k = torch.zeros(D.max_pages * 32, 128, device="cuda")
        k[:, 0], k[top, 0] = 32.0, 64.0
        kk = k.to(torch.int8) if code == "int8" else k.to(torch.float8_e4m3fn)
        c.k[0, c.page_table[0].long(), 0] = kk.view(torch.uint8).view(D.max_pages, 32, 128)
        q = bf(1, 1, 4, 128)
        q[..., 0] = torch.tensor([2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27], device="cuda")
        out = attn(D, c, q)
        v = values(c, "v", 0, 0, 0, 3001)
        assert torch.equal(out[0, 0], v[top].to(torch.bfloat16).expand(4, 128))
    c.k[0, c.page_table[0].long(), 0] = 32 if code == "int8" else 0x60          # 32 as e4m3
    out = attn(D, c, bf(1, 1, 4, 128) + torch.tensor([2.0 ** 24] + [0.0] * 127, device="cuda").bfloat16())
    mean = v.mean(0)
    # equal weights: a rounding of them is the same for all; the sums are off by 2^-8 of a half code step
    assert bool(((out[0, 0].double() - mean).abs() <= U.U * mean.abs() + 2.0 ** -9 * v.abs().mean(0)).all())
