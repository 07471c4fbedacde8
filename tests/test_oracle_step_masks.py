"""Masks of steps without parents in the oracle, by hand."""

from oracle import step as OS


def test_masks_of_chains_without_parents():
    def masks(n, words):
        return OS.assign([[0] * 9], [9], [], 0, [3], [n], n + 1, 16, None, words)[4]
    assert masks(3, 1) == [[1], [3], [7], [0]]
    assert masks(66, 1)[63:] == [[-1], [-1], [-1], [0]]
    assert masks(66, 2)[63:] == [[-1, 0], [-1, 1], [-1, 3], [0, 0]]
