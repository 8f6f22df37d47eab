"""What a prefix does beside documents: first keys bound rows from below alone, so a prefix that
ends inside the first document changes nothing for later ones, and a longer one shows rows
the keys of the next.
"""

import numpy as np
import pytest

from oracle.scored import visible

CUTS, L = [0, 40, 41, 100], 150                # documents 0 .. 39, 40, 41 .. 99, 100 .. 149


def _document(p):
    return max(i for i, c in enumerate(CUTS) if c <= p)


def _sees(prefix):
    """[position, key]: visible or not."""
    seen = np.zeros((L, L), bool)
    for p in range(L):
        lo, hi = visible(p, L, 0, CUTS[_document(p)], prefix)
        seen[p, lo:hi] = True
    return seen


DOCUMENTS = np.array([_document(p) for p in range(L)])
SAME = DOCUMENTS[:, None] == DOCUMENTS[None]
CAUSAL = np.tril(np.ones((L, L), bool))


@pytest.mark.parametrize("prefix", [0, 1, 17, 39, 40])
def test_a_prefix_inside_the_first_document(prefix):
    want = SAME & CAUSAL
    want[:40, :prefix] = True
    assert np.array_equal(_sees(prefix), want)


@pytest.mark.parametrize("prefix", [41, 60, 120, 150])
def test_a_longer_prefix_shows_later_documents(prefix):
    want = CAUSAL | (np.arange(L)[None] < prefix)
    want &= np.arange(L)[None] >= np.array(CUTS)[DOCUMENTS][:, None]
    assert np.array_equal(_sees(prefix), want)
    assert (_sees(prefix) & ~SAME).any()
