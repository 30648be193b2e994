"""When a node of a tree and the same token decoded alone select the same pages.

Keys of a sequence, of which the tree's prefix has the first L and a path of the
tree the rest.  Node i of the path selects from the prefix; decoded alone, token i
selects from the first L + i positions.  With `last` of 1 or more the lists are the
same as long as the positions from L - 1 to L + i - 1 lie in one page: pages before the
last are whole and unchanged, the last one is selected without a score.  Beyond, they
may differ.  On the CPU."""
import numpy as np
import pytest

from oracle import kv8, select

DH, P, G = 16, 16, 2


def lists(codes, scale, q, length, top, first, last):
    """The pages that q [G, DH] selects from the first `length` positions."""
    pages = -(-length // P)
    box = [select.bounds(kv8.decode(codes[p * P:min(length, p * P + P)])) for p in range(pages)]
    lo, hi = (np.array([b[side] for b in box]).reshape(pages, DH) for side in (0, 1))
    return select.choose(select.scores(q, lo, hi, scale[:pages]), top, first, last)


def sequence(seed, length):
    rng = np.random.default_rng(seed)
    return kv8.encode(rng.standard_normal((length, DH)) * 60), 2.0 ** rng.integers(-1, 2, -(-length // P)), rng


@pytest.mark.parametrize("first,last", [(0, 1), (1, 1), (1, 2)])
def test_inside_the_last_page_the_lists_are_the_same(first, last):
    differ = 0
    for L in range(8 * P + 1, 9 * P + 1):          # every place of the prefix's end in a page
        codes, scale, rng = sequence(L, L + P + 4)
        for i in range(P + 4):                     # a path longer than a page
            q = rng.standard_normal((G, DH))
            tree, alone = (lists(codes, scale, q, n, 4, first, last) for n in (L, L + i))
            if (L + i - 1) // P == (L - 1) // P:
                assert tree == alone, (L, i)
            else:
                # one page more, taken without a score; the tree's last page competes
                assert -(-(L + i) // P) - 1 in alone and -(-L // P) - 1 in tree
                differ += tree != alone
    assert differ > 0                              # past the page's end nothing is promised


def test_without_a_forced_last_page_nothing_is_promised():
    differ = 0
    for L in range(8 * P + 1, 9 * P):
        codes, scale, rng = sequence(L, L + P)
        for i in range(1, 9 * P - L + 1):          # inside the page
            q = rng.standard_normal((G, DH))
            differ += lists(codes, scale, q, L, 4, 1, 0) != lists(codes, scale, q, L + i, 4, 1, 0)
    assert differ > 0
