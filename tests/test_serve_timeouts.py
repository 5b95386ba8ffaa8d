"""Failure detection of the serving kernels without a GPU fault: a bounded wait
that runs out.  The test hook makes the next launch withhold one hand-off in its
first block; every wait is bounded and sees the others' give-up, so the launch
ends by itself with PSA_ERR_TIMEOUT in the status word, and the next call on the
same context gives what it gave before."""

import time

import pytest
import torch

from block_sparse_attention_psa_b200 import psa


def test_stall_hook_arguments():
    L = psa.lib()
    assert L.psa_test_stall_next_serve(2) == psa.PSA_ERR_ARG
    assert L.psa_test_stall_next_serve(1) == psa.PSA_OK
    assert L.psa_test_stall_next_serve(0) == psa.PSA_OK   # taken back: no call meets it


def stall(call, ws):
    want = call()
    assert psa.psa_read_status(ws) == psa.PSA_OK
    psa.psa_test_stall_next_serve(True)
    t0 = time.perf_counter()
    call()
    status = psa.psa_read_status(ws)          # synchronises the stream
    elapsed = time.perf_counter() - t0
    assert status == psa.PSA_ERR_TIMEOUT, psa.status_text(status)
    assert elapsed < 60.0, elapsed
    for _ in range(2):
        got = call()
        assert psa.psa_read_status(ws) == psa.PSA_OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("B, G, T, d, P, C", [
    (1, 1, 1, 64, 0, 100),          # one tile
    (3, 4, 1, 128, 0, 3000),        # caches, several tiles each
    (40, 4, 1, 128, 9000, 300),     # a prefix for a pair of row tiles, and caches
    (2, 2, 100, 64, 1000, 2000),    # several row tiles of a cache
], ids=str)
def test_decode_stops_and_the_context_survives(B, G, T, d, P, C):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = r(B, 2 * G, T, d), r(B, 2, C, d), r(B, 2, C, d)
    kp, vp = (r(1, 2, P, d), r(1, 2, P, d)) if P else (None, None)
    ws = psa.decode_workspace(B, 2 * G, 2, T, d, 1, P, C)
    stall(lambda: psa.psa_decode(q, k, v, None, kp, vp, None, ws=ws, want_lse=True), ws)


@pytest.mark.gpu
@pytest.mark.parametrize("B, Hkv, G, T, d, C, causal", [
    (1, 1, 1, 64, 64, 200, True),       # one unit
    (3, 8, 4, 32, 128, 5000, True),     # more units than SMs, query tiles kept on chip
    (3, 8, 4, 100, 128, 5000, True),    # and streamed past them
    (2, 8, 2, 700, 64, 3000, True),     # tiles of one head
    (1, 1, 8, 640, 128, 640, False),    # split query tiles
], ids=str)
def test_key_weight_stops_and_the_context_survives(B, Hkv, G, T, d, C, causal):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).half().cuda()  # noqa: E731
    q, k = r(B, Hkv * G, T, d), r(B, Hkv, C, d)
    lse = torch.full((B, Hkv * G, T), 5.0, device="cuda")
    ws = psa.key_weight_workspace(B, Hkv * G, Hkv, T, d, B, C)
    stall(lambda: (psa.psa_key_weight(q, k, lse, causal=causal, ws=ws),), ws)
