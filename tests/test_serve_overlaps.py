"""The workspace of psa_key_weight may not lie over a tensor of the call, as for
the other serving entry points.  Host-only."""

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

FAR = 1 << 40       # aligned to everything, never dereferenced


def weight(**kw):
    a = dict(q=1 * FAR, k=2 * FAR, lse=3 * FAR, kl=None, si=None, B=2, Hq=4, Hkv=2, T=1, d=64, Bk=2, C=100, causal=1,
             dtype=0, so=5 * FAR, ws=6 * FAR, n=1 << 62, st=None)
    a.update(kw)
    return psa.lib().psa_key_weight(*a.values())


@pytest.mark.parametrize("kw", [dict(ws=1 * FAR), dict(ws=2 * FAR + 256), dict(ws=3 * FAR), dict(kl=6 * FAR + 8),
                                dict(si=6 * FAR), dict(so=6 * FAR, si=6 * FAR), dict(so=6 * FAR + 16),
                                dict(q=6 * FAR - 512), dict(lse=6 * FAR - 4)])
def test_a_workspace_over_a_tensor_is_refused(kw):
    assert weight(**kw) == psa.PSA_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU the device check, the last one, is what refuses")
def test_what_is_not_an_overlap_goes_on_to_the_device_check():
    for kw in ({}, dict(si=5 * FAR), dict(si=4 * FAR, kl=7 * FAR), dict(q=6 * FAR - 1024), dict(q=6 * FAR + 256)):
        assert weight(**kw) == psa.PSA_ERR_DEVICE
