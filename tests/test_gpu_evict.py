"""psa_cache_evict against its definition: everything it gives is exact."""

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O
from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


def make(B, H, C, d, dtype=torch.bfloat16, seed=0, kind="tails"):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, H, C, d, generator=g).to(dtype)
    v = torch.randn(B, H, C, d, generator=g).to(dtype)
    e = torch.rand(B, H, C, generator=g)
    score = {"tails": torch.where(e < 0.1, 0.0, (e * 10 - 5).exp()), "equal": torch.full_like(e, 2.5),
             "few": (e * 4).floor(), "odd": (e * 10 - 5).sinh()}[kind]
    if kind == "odd":   # infinities, NaN, signed zeros among negative and positive scores
        score[e < 0.05] = float("nan")
        score[(e > 0.05) & (e < 0.1)] = float("inf")
        score[(e > 0.1) & (e < 0.15)] = float("-inf")
        score[(e > 0.15) & (e < 0.2)] = 0.0
        score[(e > 0.2) & (e < 0.25)] = -0.0
    pos = torch.stack([torch.randperm(C, generator=g) for _ in range(B * H)]).view(B, H, C).int()
    return k, v, score, pos


def check(x, lens, budget, sink, recent, use_pos, in_place, c_out=None):
    k, v, score, pos = x
    B, H, C, d = k.shape
    kept, newlen = O.evict(score.numpy(), pos.numpy() if use_pos else None, lens, budget, sink, recent)
    c_out = C if in_place else (c_out or budget)
    gk, gv, gs, gp = (t.cuda() for t in x)
    glen = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = psa.cache_evict_workspace(B, H, C, budget)
    if in_place:
        before = [t.clone() for t in (gk, gv, gs, gp)]
        out = (gk, gv, gs, gp if use_pos else torch.full_like(gp, -7), glen,
               torch.empty(B, H, budget, dtype=torch.int32, device="cuda"))
        if not use_pos:
            before[3] = out[3].clone()
    else:
        fill = lambda *s, dtype: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
        out = (fill(B, H, c_out, d, dtype=k.dtype), fill(B, H, c_out, d, dtype=k.dtype),
               fill(B, H, c_out, dtype=torch.float32), fill(B, H, c_out, dtype=torch.int32),
               fill(B, dtype=torch.int32), fill(B, H, budget, dtype=torch.int32))
        before = [t.clone() for t in out[:4]]
    got = psa.psa_cache_evict(gk, gv, gs, budget, pos=gp if use_pos else None, cache_len=glen, sink=sink,
                              recent=recent, ws=ws, out=out)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    assert np.array_equal(got[5].cpu().numpy(), kept)
    assert np.array_equal(got[4].cpu().numpy(), newlen)
    bits = lambda t: t.cpu().view(torch.int32 if t.dtype == torch.float32 else  # noqa: E731
                                  torch.int16 if t.element_size() == 2 else t.dtype)
    for b in range(B):
        n = int(newlen[b])
        for h in range(H):
            at = torch.from_numpy(kept[b, h, :n])
            src = (k, v, score, pos if use_pos else torch.arange(C, dtype=torch.int32).expand(B, H, C))
            for t, s, old in zip(got[:4], src, before):
                assert torch.equal(bits(t[b, h, :n]), bits(s[b, h][at]))
                assert torch.equal(bits(t[b, h, n:]), bits(old[b, h, n:])), "slots past the length changed"


CASES = [
    # B, H, C, d, lens, budget, sink, recent, scores
    (1, 1, 1, 64, [1], 1, 0, 0, "tails"),
    (1, 2, 2, 128, [2], 1, 0, 1, "tails"),
    (2, 2, 33, 64, [33, 0], 32, 4, 8, "tails"),
    (3, 2, 130, 128, [130, 129, 64], 128, 2, 16, "few"),
    (2, 3, 1000, 64, [1000, 501], 500, 0, 0, "equal"),
    (2, 1, 1025, 128, [1025, 1024], 1024, 4, 64, "tails"),
    (1, 2, 4097, 64, [4097], 100, 50, 50, "odd"),
    (1, 1, 9001, 64, [8999], 4096, 4, 1000, "odd"),
    (1, 2, 40000, 64, [39999], 1, 0, 0, "tails"),
    (1, 1, 33000, 64, [33000], 32999, 0, 0, "few"),
    (2, 1, 20000, 64, [20000, 7000], 6999, 0, 0, "equal"),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("use_pos", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:4]) + "-" + c[8])
def test_against_the_definition(case, use_pos, in_place):
    B, H, C, d, lens, budget, sink, recent, kind = case
    check(make(B, H, C, d, kind=kind), lens, budget, sink, recent, use_pos, in_place)


def test_wider_output_cache_and_fp16():
    check(make(2, 2, 300, 64, torch.float16), [300, 200], 150, 4, 20, True, False, c_out=400)


def test_long_cache_whose_keys_do_not_fit_on_chip():
    """300000 entries over 8 CTAs: more than a CTA keeps, so every pass reads
    the scores again."""
    check(make(1, 1, 300000, 64), [299999], 2000, 4, 500, True, False)
    check(make(1, 1, 300000, 64, kind="few"), [300000], 299990, 4, 500, False, True)


def test_protected_entries_stay_whatever_their_score():
    k, v, score, pos = make(1, 1, 500, 64)
    pos = torch.arange(500, dtype=torch.int32).view(1, 1, 500).contiguous()
    score[:] = 1.0
    score[0, 0, :4] = -1.0
    score[0, 0, -16:] = float("nan")
    got = psa.psa_cache_evict(k.cuda(), v.cuda(), score.cuda(), 20, pos=pos.cuda(), sink=4, recent=16)
    assert sorted(got[3].flatten().tolist()) == list(range(4)) + list(range(484, 500))


def test_evicting_one_entry_moves_one_row():
    """In place, one entry over the budget: the last entry takes the evicted
    one's slot, every other slot keeps its entry."""
    k, v, score, pos = make(1, 1, 65, 64)
    score = torch.rand(1, 1, 65) + 1
    score[0, 0, 17] = 0.5
    pos = torch.arange(65, dtype=torch.int32).view(1, 1, 65).contiguous()
    check((k, v, score, pos), [65], 64, 0, 8, True, True)
    got = psa.psa_cache_evict(k.cuda(), v.cuda(), score.cuda(), 64, pos=pos.cuda(), recent=8)
    want = list(range(64))
    want[17] = 64
    assert got[5].flatten().tolist() == want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("C, sink, recent", [(3, 1, 1), (700, 300, 399), (50000, 4, 40000), (300000, 4, 100)])
def test_one_entry_over_the_budget(C, sink, recent, in_place):
    """One reduction picks it: over one CTA, a cluster, and keys that do not
    fit on chip; among few unprotected entries; of equal scores the last."""
    for kind in ("tails", "equal", "few"):
        check(make(2, 1, C, 64, kind=kind), [C, C - 1], C - 1, sink, recent, True, in_place)
        check(make(1, 2, C, 64, kind=kind), [C], C - 1, sink, recent, False, in_place)


def test_bad_lengths_are_clamped_and_reported():
    x = make(2, 1, 70, 64)
    ws = psa.cache_evict_workspace(2, 1, 70, 50)
    glen = torch.tensor([-3, 99], dtype=torch.int32).cuda()
    got = psa.psa_cache_evict(*(t.cuda() for t in x[:3]), 50, pos=x[3].cuda(), cache_len=glen, ws=ws)
    assert psa.psa_read_status(ws) == psa.PSA_ERR_LENGTH
    assert got[4].tolist() == [0, 50]


def test_captured_graph_follows_the_lengths():
    k, v, score, pos = (t.cuda() for t in make(2, 2, 700, 64))
    glen = torch.tensor([700, 600], dtype=torch.int32).cuda()
    ws = psa.cache_evict_workspace(2, 2, 700, 300)
    out = psa.psa_cache_evict(k, v, score, 300, pos=pos, cache_len=glen, recent=10, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        psa.psa_cache_evict(k, v, score, 300, pos=pos, cache_len=glen, recent=10, ws=ws, out=out)
    for lens in ([301, 300], [10, 0], [700, 555]):
        glen.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        kept, n = O.evict(score.cpu().numpy(), pos.cpu().numpy(), lens, 300, 0, 10)
        assert np.array_equal(out[5].cpu().numpy(), kept) and out[4].tolist() == n.tolist()
