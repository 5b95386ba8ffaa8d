"""psa_key_weight where a CTA of the tensor-core kernel takes more than one unit
of work (more pairs of key tiles than the machine has SMs): query tiles that
stay on chip for several pairs, tiles streamed past them, tiles of one head
dealt forwards and backwards, query tiles split in parts.

Reference: float64.  Tolerance as derived in test_gpu_key_weight.py (same
inputs): 3e-4 of the weight added, and a rounding of the score it joins."""

import math

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu

SMS = 148


def reference(q, k, lens, causal, score):
    """(lse of the queries in fp32, scores, weight added), float64, key set by key set."""
    B, Hq, T, d = q.shape
    Bk, Hkv, C, _ = k.shape
    n, G = B // Bk, Hq // Hkv
    lse = torch.full((B, Hq, T), -math.inf)
    mass = torch.zeros(Bk, Hkv, C, dtype=torch.float64)
    for b in range(B):
        m = lens[b // n]
        if m == 0:
            continue
        for h in range(Hkv):
            z = q[b, h * G:(h + 1) * G].double() @ k[b // n, h, :m].double().T / math.sqrt(d)
            if causal:
                z = torch.where(torch.arange(m) < m - (T - 1 - torch.arange(T))[:, None], z, -math.inf)
            l32 = torch.logsumexp(z, -1).float()
            lse[b, h * G:(h + 1) * G] = l32
            e = torch.exp(z - l32.double()[..., None])
            mass[b // n, h, :m] += torch.where(l32[..., None] == -math.inf, 0.0, e).sum((0, 1))
    there = torch.arange(C) < torch.tensor(lens)[:, None, None]
    return lse, torch.where(there, score.double() + mass, 0.0), mass


CASES = [
    # what it is, B, Bk, Hkv, G, T, d, C, lens, causal, parts
    ("one tile on chip", 3, 3, 8, 4, 32, 64, 5000, [5000, 4099, 257], True, 1),
    ("two tiles on chip", 3, 3, 8, 4, 64, 128, 5000, [4999, 0, 3000], True, 1),
    ("four tiles on chip", 2, 2, 8, 4, 120, 64, 5000, [5000, 4863], True, 1),
    ("three tiles streamed", 3, 3, 8, 3, 100, 128, 5000, [5000, 1, 4000], True, 1),
    ("six tiles streamed", 3, 3, 8, 7, 100, 64, 5000, [3333, 5000, 512], True, 1),
    ("sequences in a tile", 6, 2, 8, 4, 8, 128, 5000, [5000, 777], False, 1),
    ("tiles of one head", 4, 4, 8, 2, 300, 64, 3000, [3000, 299, 2900, 0], True, 1),
    ("prefills", 8, 8, 8, 1, 1500, 64, 1500, [1500, 1499, 700, 1500, 256, 1, 1500, 1024], True, 1),
    ("rows in parts", 1, 1, 8, 16, 100, 128, 4864, [4800], True, 2),
    ("a head's tiles in parts", 1, 1, 8, 8, 200, 64, 4864, [4864], True, 4),
]


# (the longest case in one type: the type is not what differs there)
RUNS = [pytest.param(c, t, id=f"{c[0].replace(' ', '-')}-{n}") for c in CASES
        for n, t in (("bf16", torch.bfloat16), ("fp16", torch.float16)) if n == "bf16" or c[5] <= 1000]


@pytest.mark.parametrize("case,dtype", RUNS)
def test_against_float64(case, dtype):
    _, B, Bk, Hkv, G, T, d, C, lens, causal, parts = case
    # more units than SMs, and the split that is meant
    assert Bk * Hkv * -(-C // 256) > SMS and B // Bk * G * T > 32
    size = psa.psa_key_weight_workspace_size(B, Hkv * G, Hkv, T, d, Bk, C)
    assert (size == 256) if parts == 1 else (size - 256) // (Bk * Hkv * C * 4) == parts
    g = torch.Generator().manual_seed(1)
    q = torch.randn(B, Hkv * G, T, d, generator=g).to(dtype)
    k = torch.randn(Bk, Hkv, C, d, generator=g).to(dtype)
    score = torch.rand(Bk, Hkv, C, generator=g)
    lse, want, mass = reference(q, k, lens, causal, score)
    for b, m in enumerate(lens):
        k[b, :, m:] = float("nan")
    gq, gk, gl, gs = q.cuda(), k.cuda(), lse.cuda(), score.cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = psa.key_weight_workspace(B, Hkv * G, Hkv, T, d, Bk, C)
    got = psa.psa_key_weight(gq, gk, gl, n, causal=causal, score=gs, ws=ws)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    err = (got.double().cpu() - want).abs()
    assert (err <= 3e-4 * mass + 2.0 ** -23 * want.abs()).all(), err.max()
    # and in place, with the same bits
    again = psa.psa_key_weight(gq, gk, gl, n, causal=causal, score=gs, ws=ws, out=gs)
    assert again is gs and torch.equal(gs, got)
