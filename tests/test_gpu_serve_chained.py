"""The serving calls overlap on the device (each kernel starts while the one
before it ends): a decode loop issued without a wait gives, bit for bit, what it
gives with the device idle before every call."""

import pytest
import torch

from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


def loop(B, H, G, d, budget, steps, T, wait):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    C = budget + T
    kc, vc, sc = r(B, H, C, d), r(B, H, C, d), torch.rand(B, H, C, device="cuda", generator=g)
    pos = torch.arange(C, device="cuda", dtype=torch.int32).expand(B, H, C).contiguous()
    n = torch.randint(0, budget + 1, (B,), device="cuda", generator=g).int()
    kept = torch.empty(B, H, budget, dtype=torch.int32, device="cuda")
    tokens = [(r(B, H * G, T, d), r(B, H, T, d), r(B, H, T, d)) for _ in range(steps)]
    idle = torch.cuda.synchronize if wait else lambda: None
    seen = []
    for i, (q, k, v) in enumerate(tokens):
        slot = (n.long()[:, None, None] + torch.arange(T, device="cuda")).expand(B, H, T)
        kc.scatter_(2, slot[..., None].expand(B, H, T, d), k)
        vc.scatter_(2, slot[..., None].expand(B, H, T, d), v)
        sc.scatter_(2, slot, 0.0)
        at = C + i * T + torch.arange(T, device="cuda", dtype=torch.int32)
        pos.scatter_(2, slot, at.expand(B, H, T).contiguous())
        n += T
        idle()
        out, lse = psa.psa_decode(q, kc, vc, n, want_lse=True)
        idle()
        psa.psa_key_weight(q, kc, lse, n, causal=True, score=sc, out=sc)
        idle()
        psa.psa_cache_evict(kc, vc, sc, budget, pos=pos, cache_len=n, sink=2, recent=8, out=(kc, vc, sc, pos, n, kept))
        idle()
        seen += [out, lse, kept.clone(), sc.clone(), n.clone()]
    return seen + [kc, vc, pos]


@pytest.mark.parametrize("case", [
    (1, 2, 1, 64, 20, 30, 1),       # shortest kernels
    (8, 8, 4, 64, 1000, 20, 1),     # the streaming key weights
    (2, 2, 3, 128, 500, 20, 40),    # the tensor-core ones, rows of several heads
    (3, 8, 2, 64, 200, 12, 130),    # and of one head
], ids=str)
def test_overlap_changes_nothing(case):
    want, got = loop(*case, True), loop(*case, False)
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(want, got))
