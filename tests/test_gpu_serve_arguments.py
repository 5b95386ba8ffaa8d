"""What the serving calls accept does not depend on whether the native module
makes them."""

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
def test_causal_is_a_truth_value_or_0_or_1(monkeypatch, native):
    assert psa._native is not None
    if not native:
        monkeypatch.setattr(psa, "_native", None)
    g = torch.Generator().manual_seed(0)
    q, k = torch.randn(1, 2, 3, 64, generator=g).half().cuda(), torch.randn(1, 1, 20, 64, generator=g).half().cuda()
    lse = torch.zeros(1, 2, 3, device="cuda")
    yes, no = psa.psa_key_weight(q, k, lse, causal=True), psa.psa_key_weight(q, k, lse, causal=False)
    assert not torch.equal(yes, no)
    assert torch.equal(psa.psa_key_weight(q, k, lse, causal=1), yes)
    assert torch.equal(psa.psa_key_weight(q, k, lse, causal=0), no)
    for bad in (2, -1):
        with pytest.raises(psa.PSAError) as e:
            psa.psa_key_weight(q, k, lse, causal=bad)
        assert e.value.status == psa.PSA_ERR_ARG
    with pytest.raises(TypeError):
        psa.psa_key_weight(q, k, lse, causal=None)
