"""A stream of another device is refused by the serving calls, not left aside.
Host-only (a stand-in for the stream: nothing is launched)."""

import types

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

OTHER = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)


def test_a_stream_of_another_device_is_refused():
    q, k = torch.zeros(1, 1, 1, 64).half(), torch.zeros(1, 1, 8, 64).half()
    for call in (lambda: psa.psa_decode(q, k, k, stream=OTHER),
                 lambda: psa.psa_key_weight(q, k, torch.zeros(1, 1, 1), stream=OTHER),
                 lambda: psa.psa_cache_evict(k, k, torch.zeros(1, 1, 8), 2, stream=OTHER)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
