"""Acceptance of drafted tokens by hand."""
from oracle.accept import accept


def test_chain():
    #          token:  0   1   2   3
    drafted, sampled = [9, 5, 6, 7], [5, 6, 8, 1]
    assert accept([0, 4], None, drafted, sampled) == ([3], [0, 1, 2], [5, 6, 8], [8])
    assert accept([0, 4], None, drafted, sampled, eos=6) == ([2], [0, 1], [5, 6], [6])   # nothing follows an end token
    assert accept([0, 4], None, drafted, [-1] * 4) == ([1], [0], [-1], [-1])
    assert accept([0, 0, 1, 4], None, drafted, sampled) == ([0, 1, 2], [0, 1, 2], [5, 6, 8], [-1, 5, 8])


def test_tree():
    # 0 - 1 - 3, 0 - 2 - 4 - 5, and 6, a second root
    masks = [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b110101, 0b1000000]
    drafted = [9, 5, 6, 7, 8, 7, 6]
    assert accept([0, 7], masks, drafted, [6, 7, 8, 0, 3, 0, 0]) == ([3], [0, 2, 4], [6, 8, 3], [3])
    assert accept([0, 7], masks, drafted, [5, 7, 8, 4, 3, 0, 0]) == ([3], [0, 1, 3], [5, 7, 4], [4])
    assert accept([0, 7], masks, drafted, [4, 7, 8, 4, 3, 0, 0]) == ([1], [0], [4], [4])
    twins = [0b1, 0b11, 0b101, 0b1101]                     # two children with the same token: the first
    assert accept([0, 4], twins, [0, 5, 5, 7], [5, 1, 7, 2]) == ([2], [0, 1], [5, 1], [1])
