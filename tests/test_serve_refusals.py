"""The serving operators refuse what they cannot do on the host, before any
CUDA call: the C entry points by status code, the binding by an exception.
Host-only."""

import ctypes

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

FAR = 1 << 40       # aligned to everything, never dereferenced
FAKE = FAR // 2
BIG = 1 << 62


def decode(L, **kw):
    a = dict(q=FAKE, kp=None, vp=None, pl=None, kc=2 * FAR, vc=3 * FAR, cl=None, B=2, Hq=4, Hkv=2, T=1, d=64, Bp=1, P=0,
             C=100, dtype=0, out=4 * FAR, lse=None, ws=5 * FAR, n=BIG, st=None)
    a.update(kw)
    return L.psa_decode(*a.values())


def weight(L, **kw):
    a = dict(q=FAKE, k=FAKE, lse=FAKE, kl=None, si=None, B=2, Hq=4, Hkv=2, T=1, d=64, Bk=2, C=100, causal=1, dtype=0,
             so=FAR, ws=2 * FAR, n=BIG, st=None)
    a.update(kw)
    return L.psa_key_weight(*a.values())


def evict(L, **kw):
    a = dict(k=1 * FAR, v=2 * FAR, score=3 * FAR, pos=None, cl=None, B=2, Hkv=2, C=100, d=64, budget=50, sink=4,
             recent=8, Co=60, ko=5 * FAR, vo=6 * FAR, so=7 * FAR, po=8 * FAR, lo=9 * FAR, kept=10 * FAR, ws=11 * FAR,
             n=BIG, st=None)
    a.update(kw)
    return L.psa_cache_evict(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), psa.PSA_ERR_ARG), (dict(out=None), psa.PSA_ERR_ARG), (dict(ws=None), psa.PSA_ERR_ARG),
    (dict(kc=None), psa.PSA_ERR_ARG), (dict(vc=None), psa.PSA_ERR_ARG), (dict(kp=FAKE), psa.PSA_ERR_ARG),
    (dict(pl=FAKE), psa.PSA_ERR_ARG), (dict(P=10), psa.PSA_ERR_ARG), (dict(C=0), psa.PSA_ERR_ARG),
    (dict(B=0), psa.PSA_ERR_ARG), (dict(T=0), psa.PSA_ERR_ARG), (dict(Bp=0), psa.PSA_ERR_ARG),
    (dict(C=-1), psa.PSA_ERR_ARG), (dict(dtype=2), psa.PSA_ERR_ARG), (dict(d=96), psa.PSA_ERR_UNSUPPORTED),
    (dict(T=257), psa.PSA_ERR_UNSUPPORTED), (dict(C=(1 << 20) + 1), psa.PSA_ERR_UNSUPPORTED),
    (dict(Hq=5), psa.PSA_ERR_SHAPE), (dict(Bp=2, B=3), psa.PSA_ERR_SHAPE), (dict(B=1 << 24, Hq=4), psa.PSA_ERR_SHAPE),
    (dict(q=FAKE + 2), psa.PSA_ERR_ARG), (dict(kc=2 * FAR + 8), psa.PSA_ERR_ARG), (dict(lse=FAKE + 2), psa.PSA_ERR_ARG),
    (dict(cl=FAKE + 1), psa.PSA_ERR_ARG), (dict(ws=FAKE + 16), psa.PSA_ERR_ARG), (dict(n=1000), psa.PSA_ERR_CAPACITY),
    # outputs over inputs or each other
    (dict(out=FAKE + 64), psa.PSA_ERR_ARG), (dict(out=2 * FAR), psa.PSA_ERR_ARG), (dict(lse=3 * FAR), psa.PSA_ERR_ARG),
    (dict(lse=4 * FAR + 8), psa.PSA_ERR_ARG), (dict(cl=4 * FAR), psa.PSA_ERR_ARG), (dict(ws=2 * FAR), psa.PSA_ERR_ARG),
])
def test_decode_refuses(kw, status):
    assert decode(psa.lib(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), psa.PSA_ERR_ARG), (dict(k=None), psa.PSA_ERR_ARG), (dict(lse=None), psa.PSA_ERR_ARG),
    (dict(so=None), psa.PSA_ERR_ARG), (dict(ws=None), psa.PSA_ERR_ARG), (dict(C=0), psa.PSA_ERR_ARG),
    (dict(T=0), psa.PSA_ERR_ARG), (dict(causal=2), psa.PSA_ERR_ARG), (dict(dtype=-1), psa.PSA_ERR_ARG),
    (dict(d=32), psa.PSA_ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), psa.PSA_ERR_UNSUPPORTED),
    (dict(Hq=3), psa.PSA_ERR_SHAPE), (dict(B=3), psa.PSA_ERR_SHAPE), (dict(q=FAKE + 4), psa.PSA_ERR_ARG),
    (dict(so=FAR + 2), psa.PSA_ERR_ARG), (dict(n=255), psa.PSA_ERR_CAPACITY),
    (dict(so=FAKE), psa.PSA_ERR_ARG),                            # over the inputs
    (dict(si=FAR + 4), psa.PSA_ERR_ARG),                         # score_out half over score_in
    (dict(kl=FAR + 16), psa.PSA_ERR_ARG), (dict(ws=FAR + 256), psa.PSA_ERR_ARG),
])
def test_key_weight_refuses(kw, status):
    assert weight(psa.lib(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), psa.PSA_ERR_ARG), (dict(score=None), psa.PSA_ERR_ARG), (dict(kept=None), psa.PSA_ERR_ARG),
    (dict(lo=None), psa.PSA_ERR_ARG), (dict(po=None), psa.PSA_ERR_ARG), (dict(budget=0), psa.PSA_ERR_ARG),
    (dict(sink=-1), psa.PSA_ERR_ARG), (dict(sink=45), psa.PSA_ERR_ARG), (dict(budget=101), psa.PSA_ERR_SHAPE),
    (dict(Co=49), psa.PSA_ERR_SHAPE), (dict(d=80), psa.PSA_ERR_UNSUPPORTED),
    (dict(C=(1 << 20) + 1), psa.PSA_ERR_UNSUPPORTED), (dict(v=2 * FAR + 2), psa.PSA_ERR_ARG),
    (dict(ws=11 * FAR + 8), psa.PSA_ERR_ARG), (dict(n=300), psa.PSA_ERR_CAPACITY),
    # in place is all or nothing
    (dict(ko=1 * FAR), psa.PSA_ERR_ARG), (dict(ko=1 * FAR, vo=2 * FAR, so=3 * FAR), psa.PSA_ERR_ARG),
    (dict(ko=1 * FAR, vo=2 * FAR, so=3 * FAR, Co=100, pos=4 * FAR), psa.PSA_ERR_ARG),
    # overlaps that are not
    (dict(ko=1 * FAR + 256), psa.PSA_ERR_ARG), (dict(vo=5 * FAR + 16), psa.PSA_ERR_ARG),
    (dict(so=3 * FAR), psa.PSA_ERR_ARG), (dict(kept=3 * FAR), psa.PSA_ERR_ARG),
    (dict(cl=9 * FAR + 4), psa.PSA_ERR_ARG), (dict(pos=7 * FAR), psa.PSA_ERR_ARG),
])
def test_evict_refuses(kw, status):
    assert evict(psa.lib(), **kw) == status


def test_workspace_sizes():
    assert psa.psa_decode_workspace_size(1, 8, 2, 1, 128, 1, 0, 100) > 0
    assert psa.psa_decode_workspace_size(1, 8, 3, 1, 128, 1, 0, 100) == 0
    assert psa.psa_decode_workspace_size(4, 8, 2, 1, 128, 3, 10, 100) == 0
    assert psa.psa_key_weight_workspace_size(1, 8, 2, 1, 128, 1, 100) >= 256
    assert psa.psa_key_weight_workspace_size(1, 8, 2, 1, 96, 1, 100) == 0
    assert psa.psa_cache_evict_workspace_size(2, 2, 100, 50) >= 256 + 2 * 4 + 2 * 2 * 50 * 4
    assert psa.psa_cache_evict_workspace_size(2, 2, 100, 101) == 0
    with pytest.raises(psa.PSAError):
        psa.decode_workspace(1, 8, 3, 1, 128, C=100)
    assert psa.status_text(psa.PSA_ERR_LENGTH) != "unknown status"


def _cache(B=2, H=2, C=100, d=64, dt=torch.bfloat16):
    return torch.zeros(B, H, C, d, dtype=dt), torch.zeros(B, H, C, d, dtype=dt)


def test_decode_binding_refuses():
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    k, v = _cache()
    with pytest.raises(ValueError, match="a cache or a prefix"):
        psa.psa_decode(q)
    with pytest.raises(ValueError, match="v_cache is required"):
        psa.psa_decode(q, k)
    with pytest.raises(ValueError, match="need k_prefix"):
        psa.psa_decode(q, k, v, prefix_len=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_cache must be torch.bfloat16"):
        psa.psa_decode(q, k.half(), v)
    with pytest.raises(ValueError, match="v_cache must have shape"):
        psa.psa_decode(q, k, v[:, :, :50])
    with pytest.raises(ValueError, match="k_cache must have shape"):
        psa.psa_decode(q, *_cache(B=3))
    with pytest.raises(ValueError, match="cache_len must be torch.int32"):
        psa.psa_decode(q, k, v, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="must be bfloat16 or float16"):
        psa.psa_decode(q.float(), k.float(), v.float())
    with pytest.raises(ValueError, match="4 dimensions"):
        psa.psa_decode(q[0], k, v)
    with pytest.raises(ValueError, match="CUDA device"):
        psa.psa_decode(q, k, v)   # well formed: only the device is wrong here


def test_key_weight_binding_refuses():
    q = torch.zeros(2, 4, 3, 64, dtype=torch.float16)
    k, _ = _cache(dt=torch.float16)
    lse = torch.zeros(2, 4, 3)
    with pytest.raises(ValueError, match="lse"):
        psa.psa_key_weight(q, k, None)
    with pytest.raises(ValueError, match="CUDA device"):
        psa.psa_key_weight(q, k, lse)
    with pytest.raises(ValueError):
        psa.psa_key_weight(q, k.bfloat16(), lse)


def test_evict_binding_refuses():
    k, v = _cache()
    score = torch.zeros(2, 2, 100)
    with pytest.raises(ValueError, match="CUDA device"):
        psa.psa_cache_evict(k, v, score, 50)
    with pytest.raises(ValueError, match="4 dimensions"):
        psa.psa_cache_evict(k[0], v, score, 50)
    with pytest.raises(ValueError, match="must be bfloat16 or float16"):
        psa.psa_cache_evict(k.float(), v.float(), score, 50)
