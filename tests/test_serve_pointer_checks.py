"""The serving entry points of the C ABI refuse memory that is not the current
device's for every pointer they take, before any launch: a length array left
on the host, or values of another GPU, would otherwise be read by a kernel."""

import ctypes
import os
import re

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
API = os.path.join(ROOT, "block_sparse_attention_psa_b200", "csrc", "api.cu")
SERVING = ("psa_decode", "psa_key_weight", "psa_cache_evict")


@pytest.mark.parametrize("name", SERVING)
def test_every_pointer_is_checked(name):
    src = open(API).read()
    m = re.search(r"\nint " + name + r"\(([^)]*)\) \{(.*?)\n\}", src, re.S)
    pointers = re.findall(r"\*\s*(\w+)", m.group(1))
    assert pointers.pop() == "stream" and len(pointers) >= 8 - (name == "psa_key_weight")
    checked = re.search(r"check_device\(\{([^}]*)\}\)", m.group(2)).group(1)
    assert {x.strip() for x in checked.split(",")} == set(pointers)
    assert m.group(2).index("check_device(") < m.group(2).index("launch_")


def _calls():
    """Of each entry point: its pointers by name, and the call with them."""
    dev = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    half, i32 = torch.bfloat16, torch.int32
    L = psa.lib()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    n = ws.numel()
    st = torch.cuda.current_stream().cuda_stream
    d = dict(q=dev(2, 2, 1, 64, dtype=half), k_prefix=dev(1, 2, 70, 64, dtype=half),
             v_prefix=dev(1, 2, 70, 64, dtype=half), prefix_len=dev(1, dtype=i32) + 70,
             k_cache=dev(2, 2, 40, 64, dtype=half), v_cache=dev(2, 2, 40, 64, dtype=half),
             cache_len=dev(2, dtype=i32) + 9, out=dev(2, 2, 1, 64, dtype=half), lse=dev(2, 2, 1), workspace=ws)
    yield "psa_decode", d, lambda a: L.psa_decode(
        a["q"], a["k_prefix"], a["v_prefix"], a["prefix_len"], a["k_cache"], a["v_cache"], a["cache_len"], 2, 2, 2, 1,
        64, 1, 70, 40, 0, a["out"], a["lse"], a["workspace"], n, st)
    w = dict(q=dev(2, 2, 1, 64, dtype=half), k=dev(2, 2, 40, 64, dtype=half), lse=dev(2, 2, 1),
             key_len=dev(2, dtype=i32) + 9, score_in=dev(2, 2, 40), score_out=dev(2, 2, 40), workspace=ws)
    yield "psa_key_weight", w, lambda a: L.psa_key_weight(
        a["q"], a["k"], a["lse"], a["key_len"], a["score_in"], 2, 2, 2, 1, 64, 2, 40, 1, 0, a["score_out"],
        a["workspace"], n, st)
    e = dict(k=dev(2, 2, 40, 64, dtype=half), v=dev(2, 2, 40, 64, dtype=half), score=dev(2, 2, 40),
             pos=dev(2, 2, 40, dtype=i32), cache_len=dev(2, dtype=i32) + 40, k_out=dev(2, 2, 20, 64, dtype=half),
             v_out=dev(2, 2, 20, 64, dtype=half), score_out=dev(2, 2, 20), pos_out=dev(2, 2, 20, dtype=i32),
             len_out=dev(2, dtype=i32), kept=dev(2, 2, 20, dtype=i32), workspace=ws)
    yield "psa_cache_evict", e, lambda a: L.psa_cache_evict(
        a["k"], a["v"], a["score"], a["pos"], a["cache_len"], 2, 2, 40, 64, 20, 1, 2, 20, a["k_out"], a["v_out"],
        a["score_out"], a["pos_out"], a["len_out"], a["kept"], a["workspace"], n, st)


@pytest.mark.gpu
@pytest.mark.parametrize("pinned", [False, True])
def test_host_memory_is_refused_for_every_pointer(pinned):
    host = torch.zeros((1 << 20) + 256, dtype=torch.uint8, pin_memory=pinned)
    at = (host.data_ptr() + 255) & ~255
    for name, tensors, call in _calls():
        right = {k: t.data_ptr() for k, t in tensors.items()}
        assert call(right) == psa.PSA_OK, name
        torch.cuda.synchronize()
        for k in tensors:
            before = {x: t.clone() for x, t in tensors.items()}
            assert call({**right, k: at}) == psa.PSA_ERR_ARG, (name, k)
            torch.cuda.synchronize()
            assert all(torch.equal(t, before[x]) for x, t in tensors.items()), (name, k)   # nothing ran
        assert call(right) == psa.PSA_OK, name
    torch.cuda.synchronize()
    assert not host.any()
