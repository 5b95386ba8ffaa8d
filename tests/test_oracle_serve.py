"""Pins of the serving operators' float64 restatement: closed forms, textbook
softmax from another library, brute force, and planted mistakes."""

import itertools
import math

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O


def _rand(*shape, seed=0):
    return np.random.Generator(np.random.PCG64(seed)).standard_normal(shape)


def test_decode_equals_textbook_softmax_over_the_joined_keys():
    B, Bp, Hq, Hkv, T, d, P, C = 4, 2, 6, 2, 3, 16, 11, 9
    q, kc, vc = _rand(B, Hq, T, d), _rand(B, Hkv, C, d, seed=1), _rand(B, Hkv, C, d, seed=2)
    kp, vp = _rand(Bp, Hkv, P, d, seed=3), _rand(Bp, Hkv, P, d, seed=4)
    cl, pl = [9, 5, 2, 0], [11, 4]
    out, lse, _, _ = O.decode(q, kc, vc, cl, kp, vp, pl)
    for b in range(B):
        k = torch.from_numpy(np.concatenate([kp[b // 2], kc[b]], 1)).repeat_interleave(3, 0)
        v = torch.from_numpy(np.concatenate([vp[b // 2], vc[b]], 1)).repeat_interleave(3, 0)
        see = torch.zeros(T, P + C, dtype=torch.bool)
        for t in range(T):
            see[t, :pl[b // 2]] = True
            see[t, P:P + max(0, cl[b] - (T - 1 - t))] = True
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b]), k, v, attn_mask=see)
        assert np.allclose(out[b], ref.numpy(), atol=1e-12)
        z = (torch.from_numpy(q[b]) @ k.mT / math.sqrt(d)).masked_fill(~see, -math.inf)
        assert np.allclose(lse[b], torch.logsumexp(z, -1).numpy(), atol=1e-12)


def test_decode_nothing_visible():
    out, lse, _, _ = O.decode(_rand(1, 1, 2, 8), _rand(1, 1, 4, 8), _rand(1, 1, 4, 8), [1])
    assert (out[0, 0, 0] == 0).all() and lse[0, 0, 0] == -np.inf
    assert np.isfinite(lse[0, 0, 1])


def test_key_weight_is_the_column_sum_of_the_softmax():
    B, Hq, Hkv, T, d, C = 2, 4, 2, 5, 8, 7
    q, k = _rand(B, Hq, T, d), _rand(B, Hkv, C, d, seed=1)
    lens = [7, 6]
    lse = O.decode(q, k, k, lens)[1]
    got, mass = O.key_weight(q, k, lse, lens, True)
    for b in range(B):
        for h in range(Hkv):
            p = np.zeros(C)
            for hq in (2 * h, 2 * h + 1):
                z = torch.from_numpy(q[b, hq] @ k[b, h].T / math.sqrt(d))
                mask = torch.arange(C) >= lens[b] - (T - 1 - torch.arange(T))[:, None]
                p += torch.softmax(z.masked_fill(mask, -math.inf), -1).numpy().sum(0)
            assert np.allclose(got[b, h], p, atol=1e-12)
        assert abs(got[b].sum() - Hq * T) < 1e-10      # every query's weights sum to one
    assert np.array_equal(got, mass)


def test_evict_equals_brute_force():
    """Of all subsets of the right size: none sums to more, once protected
    entries count as infinite, and the order rule holds."""
    rng = np.random.Generator(np.random.PCG64(3))
    for _ in range(30):
        C, budget, sink, recent = 7, int(rng.integers(1, 7)), int(rng.integers(0, 2)), 0
        recent = int(rng.integers(0, budget - sink + 1)) if budget > sink else 0
        sink = min(sink, budget)
        score, pos = rng.integers(0, 4, (1, 1, C)).astype(float), rng.permutation(C).reshape(1, 1, C)
        kept, n = O.evict(score, pos, [C], budget, sink, recent)
        ids = kept[0, 0]
        assert n[0] == budget and len(set(ids)) == budget
        safe = {i for i in range(C) if pos[0, 0, i] < sink or pos[0, 0, i] > C - 1 - recent}
        assert safe <= set(ids)
        worth = lambda s: sum(score[0, 0, i] for i in s if i not in safe)  # noqa: E731
        best = max(worth(s) for s in itertools.combinations(range(C), budget) if safe <= set(s))
        assert worth(ids) == best
        stay = [i for i in range(budget) if i in set(ids)]
        assert all(ids[i] == i for i in stay)                    # what can stay stays
        moved = [ids[i] for i in range(budget) if ids[i] != i]
        assert moved == sorted(moved) and all(m >= budget for m in moved)


def test_evict_ties_keep_the_lower_slot_and_nan_goes_first():
    score = np.array([[[1.0, 2.0, 1.0, np.nan, 1.0]]])
    kept, _ = O.evict(score, None, [5], 3, 0, 0)
    assert kept[0, 0].tolist() == [0, 1, 2]
    kept, _ = O.evict(score[:, :, ::-1], None, [5], 4, 0, 0)
    assert kept[0, 0].tolist() == [0, 4, 2, 3]


@pytest.mark.parametrize("mistake", ["prefix of the wrong group", "causal off by one", "scale dropped"])
def test_planted_mistakes_are_seen(mistake):
    q, k = _rand(2, 1, 2, 8), _rand(2, 1, 6, 8, seed=1)
    ref = O.decode(q, k, k, [6, 5])[0]
    if mistake == "prefix of the wrong group":
        bad = O.decode(q, k[::-1], k[::-1], [6, 5])[0]
    elif mistake == "causal off by one":
        bad = O.decode(q, k, k, [5, 4])[0]
    else:
        bad = O.decode(q * math.sqrt(8), k, k, [6, 5])[0]
    assert np.abs(bad - ref).max() > 1e-3
