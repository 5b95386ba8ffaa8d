"""psa_key_weight against the float64 restatement.

Tolerance: a weight e^{s - lse} is as exact, relatively, as its exponent is
absolutely.  The fp32 logit of d products is off by at most
(d + 2) 2^-24 sum_c |q_c k_c| / sqrt(d) < 2e-4 (the sum stays below 25 for
these inputs), the product with log2 e and the subtraction add 3 roundings of
values below 64 (2e-5), the exponential 2^-22; the sum's own roundings stay
below 1e-5 of it (compensated over tiles, 32 terms in a row inside one).  So
each slot is within 3e-4 of the weight added, plus a rounding of the score
it joins, 2^-23 of the result."""

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O
from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


def make(B, Bk, Hq, Hkv, T, d, C, dtype, lens, causal, seed=0, junk=float("nan")):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, T, d, generator=g).to(dtype)
    k = torch.randn(Bk, Hkv, C, d, generator=g).to(dtype)
    score = torch.rand(Bk, Hkv, C, generator=g)
    for i, m in enumerate(lens):
        k[i, :, m:] = junk
    # the queries' own log sums (rounded to fp32, an input like any other)
    n, G = B // Bk, Hq // Hkv
    kk = torch.nan_to_num(k.double())
    z = torch.einsum("bhtd,bhcd->bhtc", q.double(), kk.repeat_interleave(n, 0).repeat_interleave(G, 1)) / d ** 0.5
    end = torch.tensor(lens).repeat_interleave(n)[:, None, None, None]
    if causal:
        end = end - (T - 1 - torch.arange(T))[None, None, :, None]
    z = z.masked_fill(torch.arange(C) >= end, -float("inf"))
    return q, k, torch.logsumexp(z, -1).float(), score


def check(x, lens, causal, with_score=True, in_place=False):
    q, k, lse, score = x
    f = lambda t: np.nan_to_num(t.double().numpy())  # noqa: E731
    ref, mass = O.key_weight(f(q), f(k), lse.double().numpy(), lens, causal,
                             score.double().numpy() if with_score else None)
    ws = psa.key_weight_workspace(q.shape[0], q.shape[1], k.shape[1], q.shape[2], q.shape[3], k.shape[0], k.shape[2])
    gs = score.cuda() if with_score else None
    got = psa.psa_key_weight(q.cuda(), k.cuda(), lse.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             causal=causal, score=gs, ws=ws, out=gs if in_place else None)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    got = got.double().cpu().numpy()
    tol = 3e-4 * mass + 2.0 ** -23 * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])


CASES = [
    # B, Bk, Hq, Hkv, T, d, C, dtype, lens, causal
    (1, 1, 1, 1, 1, 64, 1, "bf16", [1], True),
    (1, 1, 4, 2, 1, 128, 129, "bf16", [129], True),
    (2, 2, 8, 2, 1, 128, 700, "bf16", [700, 255], True),
    (3, 3, 6, 2, 1, 64, 300, "fp16", [0, 256, 257], True),
    (3, 3, 6, 2, 5, 64, 300, "fp16", [3, 5, 300], True),           # fewer entries than tokens
    (2, 2, 2, 1, 100, 128, 600, "bf16", [600, 130], True),          # 200 rows, two tiles across heads
    (1, 1, 2, 2, 128, 64, 128, "bf16", [128], True),
    (1, 1, 4, 2, 300, 128, 300, "bf16", [300], True),               # a causal prefill
    (2, 2, 2, 1, 257, 64, 900, "fp16", [900, 257], True),
    (2, 2, 2, 1, 257, 64, 900, "fp16", [100, 400], True),           # more tokens than entries
    (1, 1, 2, 1, 300, 64, 500, "bf16", [499], False),
    (12, 1, 8, 2, 1, 128, 1000, "bf16", [999], False),              # a shared prefix, one tile of 48 rows
    (66, 2, 6, 1, 1, 64, 520, "bf16", [520, 130], False),           # 198 rows over two tiles, the last part filled
    (10, 1, 30, 1, 5, 64, 260, "fp16", [260], False),               # 150 rows per sequence
    (1, 1, 8, 1, 700, 128, 700, "bf16", [700], True),               # few units: query tiles split
    (4, 1, 2, 1, 200, 64, 300, "bf16", [300], True),                # causal and shared
    (2, 2, 20, 1, 1, 128, 400, "bf16", [400, 131], True),           # rows on both sides of where the kernels change
    (2, 2, 20, 1, 1, 64, 400, "fp16", [400, 131], True),
    (2, 2, 16, 1, 1, 128, 400, "fp16", [17, 399], True),
    (1, 1, 11, 1, 3, 64, 200, "bf16", [150], True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:8]) + ("-causal" if c[9] else ""))
def test_against_the_definition(case):
    B, Bk, Hq, Hkv, T, d, C, dt, lens, causal = case
    x = make(B, Bk, Hq, Hkv, T, d, C, {"bf16": torch.bfloat16, "fp16": torch.float16}[dt], lens, causal)
    check(x, lens, causal)


def test_without_a_score_and_in_place():
    x = make(2, 2, 4, 2, 3, 128, 400, torch.bfloat16, [400, 77], True)
    check(x, [400, 77], True, with_score=False)
    check(x, [400, 77], True, in_place=True)
    x = make(1, 1, 8, 1, 700, 64, 700, torch.bfloat16, [650], True)   # split query tiles
    check(x, [650], True, with_score=False)
    check(x, [650], True, in_place=True)


@pytest.mark.parametrize("case", [
    (3, 3, 4, 2, 1, 64, 300, "fp16", [300, 100, 257], True),      # few queries
    (6, 2, 16, 1, 1, 128, 700, "bf16", [700, 300], False),        # 48 rows of a tile
    (1, 1, 4, 2, 64, 128, 600, "bf16", [600], True),              # a window, whole tiles
    (2, 2, 4, 2, 256, 64, 500, "bf16", [500, 256], True),         # a prefill
    (1, 1, 8, 1, 640, 128, 640, "fp16", [640], False),            # split query tiles
], ids=str)
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_queries_without_lse_add_nothing_whatever_they_hold(case, junk):
    """Padded queries: lse = -inf, and the row's memory as it was."""
    B, Bk, Hq, Hkv, T, d, C, dt, lens, causal = case
    q, k, lse, score = make(B, Bk, Hq, Hkv, T, d, C, {"bf16": torch.bfloat16, "fp16": torch.float16}[dt], lens, causal)
    gone = torch.rand(lse.shape, generator=torch.Generator().manual_seed(5)) < 0.3
    gone[0, 0, 0], gone[-1, -1, -1] = True, False
    lse[gone] = -float("inf")
    zeros = torch.where(gone[..., None], 0, q)
    ref = torch.nan_to_num(k.double()), lse.double().numpy()
    ref, mass = O.key_weight(zeros.double().numpy(), ref[0].numpy(), ref[1], lens, causal, score.double().numpy())
    q = torch.where(gone[..., None], torch.full_like(q, junk), q)
    got = psa.psa_key_weight(q.cuda(), k.cuda(), lse.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             causal=causal, score=score.cuda()).double().cpu().numpy()
    assert (np.abs(got - ref) <= 3e-4 * mass + 2.0 ** -23 * np.abs(ref)).all()


def test_weights_of_a_query_sum_to_one():
    """Over all keys of a head the weights of its G T queries sum to G T."""
    x = make(1, 1, 8, 2, 500, 128, 2000, torch.bfloat16, [1999], True)
    got = psa.psa_key_weight(x[0].cuda(), x[1].cuda(), x[2].cuda(), torch.tensor([1999]).int().cuda(), causal=True)
    s = got.double().sum(-1).cpu().flatten()
    # every weight within 3e-4 (the bound above), so is the sum
    assert (s / 2000 - 1).abs().max() < 3e-4
    assert (got[..., 1999:] == 0).all()


def test_bit_identical_on_repeats():
    x = [t.cuda() for t in make(1, 1, 8, 1, 700, 64, 700, torch.bfloat16, [700], True)]
    a = psa.psa_key_weight(*x[:3], causal=True, score=x[3])
    for _ in range(3):
        assert torch.equal(a, psa.psa_key_weight(*x[:3], causal=True, score=x[3]))


def test_bad_lengths_are_clamped_and_reported():
    x = [t.cuda() for t in make(2, 2, 2, 1, 1, 64, 100, torch.bfloat16, [100, 100], True)]
    ws = psa.key_weight_workspace(2, 2, 1, 1, 64, 2, 100)
    bad = psa.psa_key_weight(*x[:3], torch.tensor([-1, 101]).int().cuda(), causal=True, ws=ws)
    assert psa.psa_read_status(ws) == psa.PSA_ERR_LENGTH
    good = psa.psa_key_weight(*x[:3], torch.tensor([0, 100]).int().cuda(), causal=True, ws=ws)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    assert torch.equal(bad, good) and (bad[0] == 0).all()


def test_captured_graph_follows_the_lengths():
    lens = [[300, 20], [1, 0], [257, 256]]
    x = make(2, 2, 4, 2, 1, 64, 300, torch.bfloat16, lens[0], True, junk=0.0)
    q, k, lse, score = (t.cuda() for t in x)
    n = torch.tensor(lens[0]).int().cuda()
    ws = psa.key_weight_workspace(2, 4, 2, 1, 64, 2, 300)
    out = psa.psa_key_weight(q, k, lse, n, causal=True, score=score, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        psa.psa_key_weight(q, k, lse, n, causal=True, score=score, ws=ws, out=out)
    for ls in lens:
        n.copy_(torch.tensor(ls).int())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, psa.psa_key_weight(q, k, lse, n, causal=True, score=score))
