"""psa_key_weight: a query with lse = -inf adds nothing, whatever it holds and
whatever the keys hold."""

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B, Bk, G, T, d, C, causal", [
    (2, 2, 1, 1, 64, 300, False),     # few queries: one, two and four groups of eight
    (2, 2, 3, 4, 128, 300, True),
    (1, 1, 4, 7, 64, 500, True),
    (24, 2, 4, 1, 64, 300, False),    # a tile of 48 rows
    (1, 1, 4, 64, 128, 500, True),    # a window
    (1, 1, 2, 200, 64, 200, True),    # a prefill
], ids=str)
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_queries_without_lse_add_nothing_to_keys_of_any_value(B, Bk, G, T, d, C, causal, junk):
    g = torch.Generator().manual_seed(0)
    q = torch.randn(B, 2 * G, T, d, generator=g).bfloat16().cuda()
    k = torch.randn(Bk, 2, C, d, generator=g).bfloat16()
    k[:, 0, ::3, 5] = junk            # the first KV head's keys, whose queries have no lse
    k = k.cuda()
    lse = torch.full((B, 2 * G, T), 4.0, device="cuda")
    score = torch.rand(Bk, 2, C, generator=g).cuda()
    lse[:, :G] = -float("inf")
    got = psa.psa_key_weight(q, k, lse, causal=causal, score=score)
    assert torch.equal(got[:, 0], score[:, 0])
    # the other head's weights are there, and do not see the first one's keys
    clean = psa.psa_key_weight(q, torch.nan_to_num(k, 0.0, 0.0, 0.0), lse, causal=causal, score=score)
    assert torch.equal(got[:, 1], clean[:, 1]) and (got[:, 1, 0] > score[:, 1, 0]).all()
