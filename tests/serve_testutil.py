"""Error bounds and reference runs shared by the serving tests on the GPU.

Let u = 2^-8 (half a bf16 step), o the exact output, A the mean of |v| under the exact
weights.  An output differs from o by at most
  weights   each is off by a relative w, so numerator and denominator together by 2 w A
            (prefill rounds the numerator's weights to bf16: w = u enters once);
  scores    an absolute error e in a score changes a weight by e^e - 1 <= 2 e, again 2 x 2 e A;
  the end   one rounding to bf16: u |o|.
A score's error: an fp32 sum of 128 products, at most 128 2^-24 sum|q k| scale (a factor of
2 for the tensor core's own order), the factors, tanh and exponential in fp32: 2^-20 of the
score's size, and for a tanh cap 2e-6 of the cap or, where every score is small against it,
of four times the largest one.
"""
import torch

from oracle import serve as R

U = 2.0 ** -8


def close(got, ref, rows_err):
    """got [n,d] bf16 against ref = attend(...) with the given weight and score errors."""
    out, size, extra, _, _ = ref
    w, e, floor = rows_err
    bound = (w + 4 * e[:, None]) * size + U * out.abs() * (1 + w) + floor * extra + 1e-30
    bad = (got.double() - out).abs() > bound * 1.001
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - out).abs() / bound).max()))


def score_error(ref, softcap):
    return 2 * 128 * 2.0 ** -24 * ref[4] + 2.0 ** -20 * (ref[3] + 1) + (2e-6 * (4 * ref[3]).clamp_max(softcap) if softcap else 0.0)


def check_rows(got, q, k, v, pos, total, score, h, b, w, floor=0.0, extra_score=0.0):
    """Rows of one sequence and head against the oracle; returns (squared error, squared output)."""
    pick = lambda t: None if t is None else t[b, :len(pos)].long()
    lo, hi = R.rows_seen(pos, total, score.window, pick(score.first_key), pick(score.prefix_end))
    ref = R.attend(q, k[:total], v[:total], pos, lo, hi, score.scale, score.softcap,
                   None if score.slopes is None else score.slopes[h])
    close(got, ref, (w, score_error(ref, score.softcap) + extra_score, floor))
    return float(((got.double() - ref[0]) ** 2).sum()), float((ref[0] ** 2).sum())


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


def graph_of(fn):
    """fn captured into a CUDA graph (after one warm-up run on a side stream)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g
