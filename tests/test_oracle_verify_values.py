"""Values that are no probabilities in the oracle's verdict on drafts: above 1 they count as 1,
NaN and negative ones as 0, where a draft is judged as where a token is drawn.
"""

import numpy as np
import pytest

import oracle

NAN, INF = float("nan"), float("inf")

# (uniform, the draft's own probability, the target's, whether the draft is kept)
JUDGED = [(0.625, 3.0, 1.5, 1), (0.625, 1.0, 1.0, 1),   # 0.625 < 1
          (0.625, NAN, 0.5, 1), (0.625, 0.0, 0.5, 1),   # 0 < 0.5
          (0.625, -1.0, 0.0, 0), (0.0, -1.0, 0.0, 0),   # 0 < 0 is false
          (0.625, INF, 0.5, 0), (0.25, INF, 0.5, 1),    # the draft's is 1
          (0.0, 0.5, NAN, 0), (0.5, 0.5, -INF, 0),      # the target's is 0
          (0.75, 1.0, INF, 1), (0.0, NAN, INF, 1)]      # the target's is 1


@pytest.mark.parametrize("u,q,p,kept", JUDGED)
def test_drafts_are_judged_by_what_values_count_as(u, q, p, kept):
    target = np.array([[[0.25, 0.25, p], [0.5, 0.25, 0.25]]])
    draft = np.array([[[0.25, 0.25, q]]])
    _, n = oracle.verify_drafts(target, draft, np.array([[2]]), np.array([[u, 0.5]]))
    assert n.tolist() == [kept]


def test_tokens_are_drawn_by_what_values_count_as():
    row = [NAN, 2.0, -1.0, 1.0]                # 0, 1, 0, 1
    target = np.array([[row]] * 4)
    out, _ = oracle.verify_drafts(target, None, np.empty((4, 0), int),
                                  np.array([[0.0], [0.4375], [0.5], [0.9375]]))
    assert out[:, 0].tolist() == [1, 1, 3, 3]
