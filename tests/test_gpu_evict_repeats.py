"""psa_cache_evict where positions repeat or are negative and more entries are
protected than stay: the protected ones rank by score among themselves, equal
scores by slot.  Everything it gives is exact."""

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O
from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


def run(B, H, C, lens, budget, sink, recent, positions, kind="few", seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, H, C, 64, generator=g).bfloat16().cuda() for _ in range(2))
    e = torch.rand(B, H, C, generator=g)
    score = {"few": (e * 4).floor(), "tails": (e * 10 - 5).exp(), "odd": (e * 10 - 5).sinh()}[kind]
    if kind == "odd":
        score[e < 0.05] = float("nan")
        score[(e > 0.05) & (e < 0.1)] = float("inf")
        score[(e > 0.1) & (e < 0.15)] = -float("inf")
        score[(e > 0.15) & (e < 0.2)] = -0.0
    pos = positions(B, H, C, g).int()
    kept, n = O.evict(score.numpy(), pos.numpy(), lens, budget, sink, recent)
    safe = (pos < sink) | (pos > torch.stack([pos[b, :, :m].amax(-1) for b, m in enumerate(lens)])[..., None] - recent)
    more = [bool(int(safe[b, h, :m].sum()) > min(m, budget)) for b, m in enumerate(lens) for h in range(H)]
    was = [t.clone() for t in (k, v)]
    glen = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gs, gp = score.cuda(), pos.cuda()
    out = (k, v, gs, gp, glen, torch.empty(B, H, budget, dtype=torch.int32, device="cuda")) if in_place else None
    ws = psa.cache_evict_workspace(B, H, C, budget)
    got = psa.psa_cache_evict(k, v, gs, budget, pos=gp, cache_len=glen, sink=sink, recent=recent, ws=ws, out=out)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    assert np.array_equal(got[5].cpu().numpy(), kept) and got[4].tolist() == n.tolist()
    at = torch.from_numpy(kept)
    there = at >= 0
    row = at.clamp(min=0).cuda()[..., None].expand(-1, -1, -1, 64)
    for x, w in zip(got[:2], was):
        assert torch.equal(x[:, :, :budget][there.cuda()], w.gather(2, row)[there.cuda()])
    for x, w in zip(got[2:4], (score, pos)):
        a, b = x[:, :, :budget].cpu()[there], w.gather(2, at.clamp(min=0))[there]
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    return more


siblings = lambda B, H, C, g: (torch.arange(C) // 5).expand(B, H, C).contiguous()  # noqa: E731
same = lambda B, H, C, g: torch.full((B, H, C), 7)  # noqa: E731
negative = lambda B, H, C, g: torch.randint(-C, C // 8 + 1, (B, H, C), generator=g)  # noqa: E731


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["few", "tails", "odd"])
@pytest.mark.parametrize("C", [12, 700, 20000, 40000])
def test_more_protected_than_stay(C, kind, in_place):
    """One CTA, clusters with keys and positions on chip, keys alone; many over
    the budget, and one over it."""
    b = C // 3
    assert all(run(1, 2, C, [C], b, 0, b, siblings, kind, in_place=in_place))
    assert all(run(2, 1, C, [C, C - 1], b, 2, b // 2, same, kind, in_place=in_place))
    assert all(run(1, 1, C, [C], C // 4, C // 4, 0, negative, kind, in_place=in_place))
    assert all(run(2, 2, C, [C, C - 1], C - 1, 1, 2, same, kind, in_place=in_place)[:2])


def test_keys_that_do_not_fit_on_chip():
    assert all(run(1, 1, 300000, [299999], 1000, 0, 1000, siblings))
    assert all(run(1, 1, 300000, [300000], 299999, 0, 1, same, "tails"))


def test_as_many_protected_as_stay():
    """Exactly nk protected entries, and fewer with equal positions among them."""
    pos = lambda B, H, C, g: torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 7, 7]).expand(B, H, C)  # noqa: E731
    assert not any(run(1, 2, 10, [10], 3, 0, 1, pos))
    assert not any(run(1, 2, 10, [10], 4, 1, 1, pos))
    assert not any(run(1, 2, 10, [10], 9, 1, 1, pos))
    assert all(run(1, 2, 10, [10], 2, 0, 1, pos))
