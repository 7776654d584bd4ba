"""The serving oracle against closed forms and hand-worked cases."""
import math

import torch

from oracle import serve as R


def test_attention_of_equal_scores_is_the_mean_of_what_is_seen():
    v = torch.arange(12.0).view(6, 2)
    q, k = torch.zeros(3, 2), torch.randn(6, 2)
    pos = torch.tensor([3, 4, 5])
    lo, hi = R.rows_seen(pos, 6, window=2)
    out = R.attend(q, k, v, pos, lo, hi)[0]
    assert torch.allclose(out, torch.stack([v[2:4].mean(0), v[3:5].mean(0), v[4:6].mean(0)]).double())
    lo, hi = R.rows_seen(pos, 6, first_key=torch.tensor([9, 0, 5]), prefix_end=torch.tensor([0, 6, 0]))
    out = R.attend(q, k, v, pos, lo, hi)[0]
    assert torch.allclose(out, torch.stack([torch.zeros(2), v.mean(0), v[5]]).double())


def test_modifiers_by_hand():
    q, k = torch.tensor([[2.0]]), torch.tensor([[3.0], [1.0]])
    v = torch.tensor([[1.0], [0.0]])
    pos, lo, hi = torch.tensor([1]), torch.tensor([0]), torch.tensor([1])
    a, b = 4 * math.tanh(6 / 4) - 0.5, 4 * math.tanh(2 / 4)       # distances 1 and 0
    want = math.exp(a) / (math.exp(a) + math.exp(b))
    got = R.attend(q, k, v, pos, lo, hi, scale=1.0, softcap=4.0, slope=0.5)[0]
    assert abs(float(got) - want) < 1e-12


def test_quantisation_by_hand():
    codes, s = R.append_page(torch.zeros(4, 2), torch.tensor(0.0), torch.tensor([[127.0, -63.5]]).bfloat16(), 0, "int8")
    assert float(s) == 1.0 and codes[0].tolist() == [127.0, -64.0]      # a tie goes to the even code
    codes, s = R.append_page(codes, s, torch.tensor([[254.0, 1.0]]).bfloat16(), 1, "int8")
    assert float(s) == 2.0 and codes[:2].tolist() == [[64.0, -32.0], [127.0, 0.0]]
    same, t = R.append_page(codes, s, torch.tensor([[2.0, -2.0]]).bfloat16(), 2, "int8")
    assert float(t) == 2.0 and torch.equal(same[:2], codes[:2]) and same[2].tolist() == [1.0, -1.0]
    codes, s = R.append_page(torch.ones(4, 2), torch.tensor(5.0), torch.tensor([[math.nan, 0.0]]).bfloat16(), 0, "e4m3")
    assert float(s) == 0.0 and codes[0].tolist() == [0.0, 0.0]          # a new page forgets its old scale


def test_pool_rules_by_hand():
    p = R.Pool([[3, 1, -1], [-1, -1, -1], [-1, -1, -1]], [0, 1, 0, 1, 0], [6, 0, 0], 4)
    p.fork([0, 0, 0], [1, 2, 1])
    assert p.table[1] == [3, 0, -1] and p.table[2] == [3, 2, -1] and p.refs == [1, 1, 1, 3, 0]
    assert p.moves == [(1, 0), (1, 2)] and p.status == 0x40
    p.free([0, 1, 0])
    assert p.refs == [0, 0, 1, 1, 0] and p.len == [0, 0, 6]
    p.moves = []
    p.compact()
    assert p.table[2] == [1, 0, -1] and p.refs == [1, 1, 0, 0, 0] and p.moves == [(2, 0), (3, 1)]
    p.status = 0
    p.reserve([13, 9, 6])                     # too long; three pages; one page, but none is left
    assert p.status == 0x22 and p.table[1] == [2, 3, 4] and p.table[2] == [1, 0, -1]
