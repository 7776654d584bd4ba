"""lrkv_prefill_attn against the fp64 definition, element by element (bounds: serve_testutil)."""
import pytest
import torch

import decode_attention_lrkv_b200 as L
from tests import serve_testutil as U

pytestmark = pytest.mark.gpu
CANARY = 123.0


def run(q, k, v, q_len=None, kv_len=None, score=None, out=None, **kw):
    out = torch.full_like(q, CANARY) if out is None else out
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    L.lrkv_prefill_attn(q, k, v, out, q_len=None if q_len is None else U.ints(q_len),
                        kv_len=None if kv_len is None else U.ints(kv_len), score=score, dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status[0])


def check(out, q, k, v, q_len=None, kv_len=None, score=None):
    B, t_q, Hq, _ = q.shape
    g, score = Hq // k.shape[2], score or L.Score()
    err = size = 0.0
    for b in range(B):
        n, T = (t_q if q_len is None else q_len[b]), (k.shape[1] if kv_len is None else kv_len[b])
        pos = torch.arange(T - n, T, device="cuda")
        for h in range(Hq):
            e, s = U.check_rows(out[b, :n, h], q[b, :n, h], k[b, :, h // g], v[b, :, h // g], pos, T, score, h, b, U.U)
            err, size = err + e, size + s
        assert bool((out[b, n:] == CANARY).all())           # rows behind the last one: as they were
    # the roundings are uniform and independent: two of them, of a variance of u^2 / 3 each
    assert err <= size * U.U ** 2 + 1e-30, (err / size) ** 0.5


def inputs(B, Hq, Hkv, t_q, t_k, seed=1, std=2.0):
    return (U.normal(seed, B, t_q, Hq, 128, std=std), U.normal(seed + 1, B, t_k, Hkv, 128),
            U.normal(seed + 2, B, t_k, Hkv, 128))


@pytest.mark.parametrize("t", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 641])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (3, 3), (6, 2)])
def test_causal_lengths(t, Hq, Hkv):
    q, k, v = inputs(1, Hq, Hkv, t, t, seed=t)
    out, status = run(q, k, v)
    assert status == 0
    check(out, q, k, v)


@pytest.mark.parametrize("t_q,t_k", [(1, 1000), (3, 64), (100, 1100), (256, 257), (129, 2048), (5, 5000)])
def test_a_chunk_after_cached_keys(t_q, t_k):
    q, k, v = inputs(2, 4, 2, t_q, t_k, seed=t_q)
    out, status = run(q, k, v)
    assert status == 0
    check(out, q, k, v)


def test_ragged_rows_and_lengths_with_garbage_behind_them():
    q_len, kv_len = [300, 0, 1, 129, 64], [300, 77, 1, 500, 64]
    q, k, v = inputs(5, 4, 2, 300, 500)
    for b, (n, T) in enumerate(zip(q_len, kv_len)):
        q[b, n:] = float("nan")
        k[b, T:] = float("nan")
        v[b, T:] = float("inf")
    out, status = run(q, k, v, q_len, kv_len)
    assert status == 0
    check(out, q, k, v, q_len, kv_len)


def test_no_keys_and_counts_out_of_range():
    q, k, v = inputs(3, 2, 2, 40, 60)
    out, status = run(q, k, v, [40, 40, 40], [0, 60, 60])
    assert bool((out[0] == 0).all()) and status == 0        # rows that see nothing
    check(out[1:], q[1:], k[1:], v[1:])
    out, status = run(q, k, v, [-5, 99, 40], [60, 61, -1])
    assert status == L.DEV_BAD_COUNT
    assert bool((out[0] == CANARY).all()) and bool((out[2] == 0).all())
    check(out[1:2], q[1:2], k[1:2], v[1:2])
    empty = torch.empty(2, 0, 2, 128, dtype=torch.bfloat16, device="cuda")
    out, _ = run(q[:2], empty, empty.clone())
    assert bool((out == 0).all())
    run(empty, k[:2], v[:2])                                # no rows: nothing happens


@pytest.mark.parametrize("softcap,std", [(20.0, 2.0), (50.0, 2.0), (5.0, 6.0), (1.0, 30.0), (2000.0, 2.0), (1e6, 2.0)])
def test_tanh_cap(softcap, std):
    """Small and large scores take the polynomial and the exponential form."""
    q, k, v = inputs(1, 4, 2, 200, 400, std=std)
    score = L.Score(softcap=softcap)
    out, _ = run(q, k, v, score=score)
    check(out, q, k, v, score=score)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 1000])
def test_windows(window):
    q, k, v = inputs(2, 4, 2, 300, 450, seed=window)
    score = L.Score(window=window)
    out, _ = run(q, k, v, score=score)
    check(out, q, k, v, score=score)


def doc_starts(B, t_q, cuts, first=0):
    row = torch.zeros(t_q, dtype=torch.int32)
    for c in cuts:
        row[max(c - first, 0):] = c
    return row.repeat(B, 1).cuda()


def test_documents_hide_what_came_before_even_nan_keys():
    q, k, v = inputs(2, 4, 2, 500, 500)
    score = L.Score(first_key=doc_starts(2, 500, [1, 64, 65, 300, 499]), softcap=30.0)
    out, _ = run(q, k, v, score=score)
    check(out, q, k, v, score=score)
    # the tail of a padded document, which no row sees
    score.first_key[:, 210:300] = 210
    score.first_key[:, 300:] = 300
    k[:, 200:210] = float("nan")
    q_seen = torch.cat([torch.arange(200), torch.arange(210, 500)])
    score.first_key[:, 200:210] = 10 ** 6                   # rows of the padding see nothing
    out, _ = run(q, k, v, score=score)
    assert bool((out[:, 200:210] == 0).all())
    for i in range(2):
        check(out[i:i + 1], q[i:i + 1], k[i:i + 1], v[i:i + 1], score=score)
    assert bool(torch.isfinite(out[:, q_seen]).all())


def test_prefix_sees_itself():
    q, k, v = inputs(2, 4, 2, 400, 600)
    end = torch.zeros(2, 400, dtype=torch.int32, device="cuda")
    end[0], end[1, :100] = 333, 590                          # the second one for some rows alone
    score = L.Score(prefix_end=end, slopes=U.slopes(4))
    out, _ = run(q, k, v, score=score)
    check(out, q, k, v, score=score)
    end.fill_(10 ** 6)                                       # past the sequence: everything is seen
    out, _ = run(q, k, v, [400, 30], [600, 50], score=score)
    check(out, q, k, v, [400, 30], [600, 50], score=score)


def test_everything_at_once():
    q, k, v = inputs(2, 8, 2, 350, 700)
    score = L.Score(scale=0.11, softcap=25.0, window=300, slopes=U.slopes(8), first_key=doc_starts(2, 350, [400, 470], 350),
                    prefix_end=torch.full((2, 350), 480, dtype=torch.int32, device="cuda"))
    out, status = run(q, k, v, [350, 201], [700, 555], score=score)
    assert status == 0
    check(out, q, k, v, [350, 201], [700, 555], score=score)


def test_rows_that_see_nothing_are_zero():
    q, k, v = inputs(1, 2, 1, 300, 300)
    first = torch.zeros(1, 300, dtype=torch.int32, device="cuda")
    first[0, 7], first[0, 130:290] = 8, 2 ** 31 - 1
    score = L.Score(first_key=first)
    out, _ = run(q, k, v, score=score)
    assert bool((out[0, 7] == 0).all()) and bool((out[0, 130:290] == 0).all())
    check(out, q, k, v, score=score)


def test_scores_that_grow_along_the_keys():
    """Every tile raises the maximum: the running reference moves all the time."""
    q = U.normal(1, 1, 300, 2, 128)
    k = q.clone()[:, :, :1] * torch.linspace(0.1, 6.0, 300, device="cuda")[None, :, None, None].to(torch.bfloat16)
    v = U.normal(2, 1, 300, 1, 128)
    for score in (L.Score(), L.Score(scale=1.0), L.Score(scale=1e-6), L.Score(slopes=torch.full((2,), -3.0, device="cuda"))):
        out, _ = run(q, k.contiguous(), v, score=score)
        check(out, q, k, v, score=score)


def test_slices_of_a_fused_projection():
    B, t, Hq, Hkv = 2, 200, 6, 2
    fused = U.normal(5, B, t, Hq + 2 * Hkv, 128)
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv], fused[:, :, Hq + Hkv:]
    wide = torch.full((B, t + 3, Hq + 1, 136), CANARY, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :t, :Hq, :128]
    run(q, k, v, out=out)
    check(out, q, k, v)
    assert bool((wide[..., 128:] == CANARY).all()) and bool((wide[:, t:] == CANARY).all())
    heads_first = U.normal(6, B, Hq, t, 128).permute(0, 2, 1, 3)     # [B, heads, t, d] storage
    out, _ = run(heads_first, k, v, out=torch.full((B, Hq, t, 128), CANARY, dtype=torch.bfloat16,
                                                   device="cuda").permute(0, 2, 1, 3))
    check(out, heads_first, k, v)


def test_offsets_past_32_bits():
    far = 2 ** 31 + 128 * 8
    base = torch.empty(far + 300 * 128, dtype=torch.bfloat16, device="cuda")
    two = base.as_strided((2, 300, 1, 128), (far, 128, 128, 1))
    q, k, v = inputs(2, 1, 1, 300, 300)
    for name in ("k", "v", "q"):
        x = {"k": k, "v": v, "q": q}
        two.copy_(x[name])
        x[name] = two
        out, _ = run(x["q"], x["k"], x["v"], out=torch.full((2, 300, 1, 128), CANARY, dtype=torch.bfloat16, device="cuda"))
        check(out, q, k, v)
    two.fill_(CANARY)
    out, _ = run(q, k, v, out=two)
    check(out, q, k, v)


def test_graph_replay_other_streams_and_equal_results():
    q, k, v = inputs(2, 8, 2, 150, 900)
    out, want = torch.zeros_like(q), run(q, k, v)[0]
    g = U.graph_of(lambda: L.lrkv_prefill_attn(q, k, v, out))
    q2 = U.normal(77, *q.shape, std=2.0)
    want2 = run(q2, k, v)[0]
    keep = q.clone()
    for x, w in ((q2, want2), (keep, want)):
        q.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = torch.zeros_like(q)
    with torch.cuda.stream(s):
        L.lrkv_prefill_attn(q, k, v, other)
    L.lrkv_prefill_attn(q, k, v, out, stream=s)
    s.synchronize()
    assert torch.equal(other, want) and torch.equal(out, want)


@pytest.mark.parametrize("t_q,t_k", [(2100, 2100), (600, 9000)])
def test_long_prompts(t_q, t_k):
    q, k, v = inputs(1, 4, 1, t_q, t_k)
    out, _ = run(q, k, v)
    check(out, q, k, v)


@pytest.mark.parametrize("score", [dict(), dict(window=700), dict(docs=True, softcap=20.0), dict(prefix=True, bias=True)],
                         ids=str)
def test_keys_split_over_ctas(score):
    """Few rows after many keys: the keys of a row block are shared out, also where a share is empty."""
    t_q, t_k = 70, 6000
    q, k, v = inputs(2, 4, 2, t_q, t_k)
    s = dict(score)
    first = None
    if s.pop("docs", False):
        first = doc_starts(2, t_q, [5950, 5990], t_k - t_q)
        first[0, :30], first[1, 10] = 100, 10 ** 7
    end = torch.full((2, t_q), 5980, dtype=torch.int32, device="cuda") if s.pop("prefix", False) else None
    s = L.Score(slopes=U.slopes(4) if s.pop("bias", False) else None, first_key=first, prefix_end=end, **s)
    out = torch.full_like(q, CANARY)
    need = L.lrkv_prefill_workspace_size(q, k, v, out)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")     # any contents: here NaN
    args = dict(q_len=[t_q, 33], kv_len=[t_k, 5000], score=s)
    run(q, k, v, out=out, ws=ws, **args)
    check(out, q, k, v, **args)
    if first is not None:
        assert bool((run(q, k, v, score=s)[0][1, 10] == 0).all())
    with pytest.raises(L.LrkvError):
        run(q, k, v, ws=ws[:need - 16])
    again = torch.full_like(q, CANARY)
    lens = {n: U.ints(args[n]) for n in ("q_len", "kv_len")}
    g = U.graph_of(lambda: L.lrkv_prefill_attn(q, k, v, again, score=s, ws=ws, **lens))
    again.fill_(CANARY)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
