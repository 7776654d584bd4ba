"""The page rules of the serving oracle where pages are missing, by hand."""
from oracle import serve as R


def test_a_sequence_does_not_advance_over_tokens_without_a_page():
    # page 4: one that has room, one whose next page is missing, one in the middle of a missing page
    p = R.Pool([[0, 1, -1], [2, -1, -1], [3, -1, 4], [5, 99, -1]], [1] * 6, [3, 2, 6, 4], 4)
    p.advance([2, 1, 2, 1])
    assert p.len == [5, 3, 6, 4] and p.status == 0x10
    p.status = 0
    p.advance([9, 5, 0, 0])
    assert p.len == [8, 4, 6, 4] and p.status == 0x12      # 14 tokens are more than three pages hold
    p = R.Pool([[0, 1]], [1, 1], [7], 4)
    p.advance([2])
    assert p.len == [8] and p.status == 0x2


def test_a_source_without_its_last_page_is_not_forked():
    p = R.Pool([[0, -1], [1, 2], [-1, -1], [-1, -1]], [1, 1, 1, 0, 0], [6, 8, 0, 0], 4)
    p.fork([0, 1], [2, 3])
    assert p.table == [[0, -1], [1, 2], [-1, -1], [1, 2]] and p.len == [6, 8, 0, 8]
    assert p.refs == [1, 2, 2, 0, 0] and p.moves == [] and p.status == 0x10
