"""Pins of the eviction's restatement where positions repeat or are negative:
more entries can then be protected than stay, and those rank by score too."""

import numpy as np
import pytest

import oracle.psa_oracle_serve as O


def test_protected_entries_rank_by_score_among_themselves():
    pos = np.array([0, 1, 2, 3, 4, 5, 5, 5, 6, 6, 6, 7]).reshape(1, 1, 12)
    score = np.arange(12.0).reshape(1, 1, 12)
    # protected: positions above 3, slots 4 to 11; the four of largest score
    kept, n = O.evict(score, pos, [12], 4, 0, 4)
    assert n[0] == 4 and kept[0, 0].tolist() == [8, 9, 10, 11]
    # every entry at one position: the one of lowest score goes
    kept, _ = O.evict(np.array([[[3.0, 1.0, 2.0]]]), np.zeros((1, 1, 3), int), [3], 2, 0, 1)
    assert kept[0, 0].tolist() == [0, 2]
    # below `sink`, negative ones included
    kept, _ = O.evict(np.array([[[1.0, 9.0, 2.0, 2.0]]]), np.array([[[-5, 7, -1, -2]]]), [4], 1, 1, 0)
    assert kept[0, 0].tolist() == [2]


@pytest.mark.parametrize("seed", range(20))
def test_it_is_the_lexicographic_order(seed):
    """(protected, score descending with NaN lowest, slot), by numpy's own sort."""
    rng = np.random.Generator(np.random.PCG64(seed))
    C, budget = 40, int(rng.integers(2, 40))
    recent = int(rng.integers(0, budget + 1))
    sink = int(rng.integers(0, budget - recent + 1))
    pos = rng.integers(-3, 12, (1, 1, C))
    score = rng.integers(0, 5, (1, 1, C)).astype(float)
    score[rng.random((1, 1, C)) < 0.1] = np.nan
    safe = (pos[0, 0] < sink) | (pos[0, 0] > pos.max() - recent)
    down = np.where(np.isnan(score[0, 0]), np.inf, -score[0, 0])
    stay = np.lexsort((np.arange(C), down, ~safe))[:budget]
    kept, _ = O.evict(score, pos, [C], budget, sink, recent)
    assert sorted(kept[0, 0].tolist()) == sorted(stay.tolist())
