"""The serving operators as they are used together: a causal prefill
(psa_dense) leaves keys, values and lse; their accumulated weights choose what
stays; new tokens attend over what stayed, add their own weights, and the
cache is kept at its budget in place.  Each step is checked against float64 on
the state the GPU left, so that one step's rounding is not another's error.

Tolerances: as derived in test_gpu_decode.py and test_gpu_key_weight.py (same
types, and logits of the same size); the prefill's lse carries the prefill
kernel's own error (its tests: 1e-3 relative), which the weights show
relatively: 1e-3 |lse| + 3e-4."""

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O
from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def close(out, ref, spread, u=2.0 ** -8):
    assert (np.abs(f64(out) - ref) <= u * spread + u * np.abs(ref) * (1 + u) + 5e-4 * spread).all()


def test_prefill_evict_decode():
    B, H, N, d, budget, sink, recent, steps = 2, 2, 640, 64, 200, 4, 32, 6
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = r(B, H, N, d), r(B, H, N, d), r(B, H, N, d)
    _, lse = psa.psa_dense(q, k, v, causal=True, want_lse=True)
    n0 = torch.full((B,), N, dtype=torch.int32, device="cuda")
    score = psa.psa_key_weight(q, k, lse, n0, causal=True)
    _, exact_lse, _, _ = O.decode(f64(q), f64(k), f64(v), [N] * B)
    want, mass = O.key_weight(f64(q), f64(k), exact_lse, [N] * B, True)
    assert (np.abs(f64(score) - want) <= mass * (np.exp(1e-3 * np.abs(exact_lse).max() + 3e-4) - 1) + 1e-6).all()

    # the prefill's entries into a cache with room for one more token
    C = budget + 1
    new = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    kc, vc = new(B, H, C, d, dtype=k.dtype), new(B, H, C, d, dtype=k.dtype)
    sc, pos = new(B, H, C, dtype=torch.float32), new(B, H, C, dtype=torch.int32)
    n, kept = new(B, dtype=torch.int32), new(B, H, budget, dtype=torch.int32)
    ws = psa.cache_evict_workspace(B, H, N, budget)
    psa.psa_cache_evict(k, v, score, budget, cache_len=n0, sink=sink, recent=recent, ws=ws,
                        out=(kc, vc, sc, pos, n, kept))
    ref, _ = O.evict(f64(score), None, [N] * B, budget, sink, recent)
    assert np.array_equal(kept.cpu().numpy(), ref) and n.tolist() == [budget] * B
    at = torch.from_numpy(ref).cuda()
    assert torch.equal(kc[:, :, :budget], k.gather(2, at[..., None].expand(-1, -1, -1, d)))
    assert torch.equal(pos[:, :, :budget].long(), at)

    dws = psa.decode_workspace(B, H, H, 1, d, C=C)
    wws = psa.key_weight_workspace(B, H, H, 1, d, B, C)
    for step in range(steps):
        # append the token's key and value at slot n, its weight starts at zero
        tq, tk, tv = r(B, H, 1, d), r(B, H, 1, d), r(B, H, 1, d)
        slot = n.long()[:, None, None, None].expand(B, H, 1, d)
        kc.scatter_(2, slot, tk)
        vc.scatter_(2, slot, tv)
        pos.scatter_(2, slot[..., 0], torch.full((B, H, 1), N + step, dtype=torch.int32, device="cuda"))
        sc.scatter_(2, slot[..., 0], 0.0)
        n += 1
        out, l1 = psa.psa_decode(tq, kc, vc, n, ws=dws, want_lse=True)
        lens = n.tolist()
        ref, rl, spread, _ = O.decode(f64(tq), f64(kc), f64(vc), lens)
        close(out, ref, spread)
        assert np.abs(f64(l1) - rl).max() < 5e-4
        before = f64(sc)
        psa.psa_key_weight(tq, kc, l1, n, causal=True, score=sc, ws=wws, out=sc)
        want, mass = O.key_weight(f64(tq), f64(kc), f64(l1), lens, True, before)
        assert (np.abs(f64(sc) - want) <= 3e-4 * mass + 2.0 ** -23 * np.abs(want)).all()
        ref, _ = O.evict(f64(sc), pos.cpu().numpy(), lens, budget, sink, recent)
        was = [t.clone() for t in (kc, vc, sc, pos)]
        psa.psa_cache_evict(kc, vc, sc, budget, pos=pos, cache_len=n, sink=sink, recent=recent,
                            out=(kc, vc, sc, pos, n, kept))
        assert np.array_equal(kept.cpu().numpy(), ref) and n.tolist() == [budget] * B
        at = torch.from_numpy(ref).cuda()
        assert torch.equal(kc[:, :, :budget], was[0].gather(2, at[..., None].expand(-1, -1, -1, d)))
        assert torch.equal(sc[:, :, :budget], was[2].gather(2, at))
        # the sinks and the latest positions are all there
        for p in list(range(sink)) + list(range(N + step + 1 - recent, N + step + 1)):
            assert (pos[:, :, :budget] == p).any(-1).all()


def test_samples_of_one_prompt_share_its_prefix():
    """Four samples over a 1000-token prompt: the joint attention, and the
    weight they put on the prompt and on their own tokens: one in sum."""
    n, H, G, d, P, C = 4, 2, 3, 128, 1000, 40
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).half().cuda()  # noqa: E731
    q, kp, vp = r(n, H * G, 1, d), r(1, H, P, d), r(1, H, P, d)
    kc, vc = r(n, H, C, d), r(n, H, C, d)
    lens = torch.tensor([1, 17, 40, 33], dtype=torch.int32, device="cuda")
    out, lse = psa.psa_decode(q, kc, vc, lens, kp, vp, want_lse=True)
    ref, rl, spread, tiny = O.decode(f64(q), f64(kc), f64(vc), lens.tolist(), f64(kp), f64(vp), [P])
    u = 2.0 ** -11
    assert (np.abs(f64(out) - ref) <= u * spread + 2.0 ** -25 * tiny + u * np.abs(ref) * (1 + u) + 5e-4 * spread).all()
    on_prompt = psa.psa_key_weight(q, kp, lse)
    on_own = psa.psa_key_weight(q, kc, lse, lens, causal=True)
    total = on_prompt.double().sum() + on_own.double().sum()
    assert abs(float(total) / (n * H * G) - 1) < 3e-4 + 5e-4     # the weights' bound and the lse's


def test_a_nan_query_stays_in_its_row():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(8, 4, 1, 64, generator=g).bfloat16().cuda()
    kp, vp = (torch.randn(1, 2, 300, 64, generator=g).bfloat16().cuda() for _ in range(2))
    clean, l0 = psa.psa_decode(q, k_prefix=kp, v_prefix=vp, want_lse=True)
    q[3, 1, 0, 5] = float("nan")
    out, l1 = psa.psa_decode(q, k_prefix=kp, v_prefix=vp, want_lse=True)
    hit = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    hit[3, 1] = True
    assert out[hit].isnan().all() and l1[hit].isnan().all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(l1[~hit], l0[~hit])


def test_unaligned_and_strided_tensors_are_refused():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 2, 32, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        psa.psa_decode(q, k.transpose(2, 3).contiguous().transpose(2, 3), k)
    odd = torch.zeros(k.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(k)
    with pytest.raises(psa.PSAError) as e:
        psa.psa_decode(q, odd, k)
    assert e.value.status == psa.PSA_ERR_ARG


def test_offsets_past_32_bits():
    """A cache of 3.2e9 elements: the last sequence starts at element 2^31."""
    B, H, C, d = 3, 8, 1 << 20, 128
    k = torch.zeros(B, H, C, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(3)
    lens = [130, 5, 300]
    for b, n in enumerate(lens):
        k[b, :, :n] = torch.randn(H, n, d, generator=g).bfloat16().cuda()
        v[b, :, :n] = torch.randn(H, n, d, generator=g).bfloat16().cuda()
    q = torch.randn(B, H, 1, d, generator=g).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = psa.psa_decode(q, k, v, n, want_lse=True)
    small = lambda t: f64(t[:, :, :300])  # noqa: E731
    ref, rl, spread, _ = O.decode(f64(q), small(k), small(v), lens)
    close(out, ref, spread)
    score = psa.psa_key_weight(q, k, lse, n, causal=True)
    want, mass = O.key_weight(f64(q), small(k), f64(lse), lens, True)
    assert (np.abs(small(score) - want) <= 3e-4 * mass).all() and (score[:, :, 300:] == 0).all()
    # eviction at the far end: the entry at the last slot of a full cache
    score = torch.zeros(B, H, C, device="cuda")
    score[:, :, C - 1] = 2.0
    score[:, :, 7] = 1.0
    k[:, :, C - 1] = 3.0
    got = psa.psa_cache_evict(k, v, score, 2)
    assert (got[5] == torch.tensor([7, C - 1], dtype=torch.int32, device="cuda")).all()
    assert (got[0][:, :, 1] == 3.0).all() and torch.equal(got[0][:, :, 0], k[:, :, 7])


def test_a_captured_step_equals_the_eager_one():
    """Append, attend, add weights, evict: one graph, replayed as the lengths
    on the device grow to the budget and stay there."""
    B, H, G, d, budget, steps = 3, 2, 4, 128, 20, 9
    C = budget + 1
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    tokens = [(r(B, H * G, 1, d), r(B, H, 1, d), r(B, H, 1, d)) for _ in range(steps)]
    start = [r(B, H, C, d), r(B, H, C, d), torch.rand(B, H, C, generator=g).cuda(),
             torch.arange(C, dtype=torch.int32).expand(B, H, C).contiguous().cuda(),
             torch.tensor([budget, budget - 3, 0], dtype=torch.int32).cuda()]
    spaces = (psa.decode_workspace(B, H * G, H, 1, d, C=C), psa.key_weight_workspace(B, H * G, H, 1, d, B, C),
              psa.cache_evict_workspace(B, H, C, budget))

    def step(state, q, k, v, out, lse, kept):
        kc, vc, sc, pos, n = state
        slot = n.long()[:, None, None, None].expand(B, H, 1, d)
        kc.scatter_(2, slot, k)
        vc.scatter_(2, slot, v)
        sc.scatter_(2, slot[..., 0], 0.0)
        pos.scatter_(2, slot[..., 0], pos.amax(-1, keepdim=True) + 1)
        n += 1
        psa.psa_decode(q, kc, vc, n, ws=spaces[0], out=out, lse=lse)
        psa.psa_key_weight(q, kc, lse, n, causal=True, score=sc, ws=spaces[1], out=sc)
        psa.psa_cache_evict(kc, vc, sc, budget, pos=pos, cache_len=n, sink=1, recent=4, ws=spaces[2],
                            out=(kc, vc, sc, pos, n, kept))

    outs = lambda: (torch.empty_like(tokens[0][0]), torch.empty(B, H * G, 1, device="cuda"),  # noqa: E731
                    torch.empty(B, H, budget, dtype=torch.int32, device="cuda"))
    eager, want = [t.clone() for t in start], []
    for t in tokens:
        o = outs()
        step(eager, *t, *o)
        want.append([x.clone() for x in (*o, *eager)])
    state, io, o = [t.clone() for t in start], [t.clone() for t in tokens[0]], outs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(state, *io, *o)
    for t, w in zip(tokens, want):
        for x, y in zip(io, t):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip((*o, *state), w))
    assert state[-1].tolist() == [budget, budget, min(budget, steps)]
    assert all(psa.psa_read_status(w) == psa.PSA_OK for w in spaces)


def test_two_streams_with_their_own_workspaces():
    """The same calls on two streams at once, interleaved, give what they give alone."""
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g).half().cuda()  # noqa: E731
    B, H, G, T, d, C = 6, 2, 3, 40, 64, 3000
    q, k, v = r(B, H * G, T, d), r(B, H, C, d), r(B, H, C, d)
    n = torch.tensor([3000, 40, 2999, 128, 1000, 77], dtype=torch.int32, device="cuda")

    def run(stream=None):
        out, lse = psa.psa_decode(q, k, v, n, want_lse=True, stream=stream)
        score = psa.psa_key_weight(q, k, lse, n, causal=True, stream=stream)
        return (out, lse, score, *psa.psa_cache_evict(k, v, score, 1000, cache_len=n, recent=50, stream=stream))

    alone = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [[run(s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    there = alone[8] >= 0
    for pair in both:
        for got in pair:
            for i in (0, 1, 2, 7, 8):
                assert torch.equal(got[i], alone[i])
            for i in (3, 4, 5, 6):   # (slots past a length are left as they were)
                assert torch.equal(got[i][there], alone[i][there])


def test_the_native_calls_are_the_python_ones(monkeypatch):
    """_call.so makes the calls here (not the Python form), with the same results."""
    assert psa._native is not None
    psa.lib()
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    B, H, G, T, d, P, C = 4, 2, 3, 2, 64, 300, 200
    q, kp, vp, k, v = r(B, H * G, T, d), r(2, H, P, d), r(2, H, P, d), r(B, H, C, d), r(B, H, C, d)
    n = torch.tensor([200, 3, 0, 77], dtype=torch.int32, device="cuda")
    m = torch.tensor([300, 129], dtype=torch.int32, device="cuda")
    pos = torch.arange(C, dtype=torch.int32, device="cuda").expand(B, H, C).contiguous()

    def run(given):
        ws = dict(ws=psa.decode_workspace(B, H * G, H, T, d, 2, P, C)) if given else {}
        out, lse = psa.psa_decode(q, k, v, n, kp, vp, m, want_lse=True, **ws)
        a = [out, lse, psa.psa_decode(q, k, v, n), psa.psa_decode(q, k_prefix=kp, v_prefix=vp)]
        score = psa.psa_key_weight(q, k, lse, n, causal=True)
        a += [score, psa.psa_key_weight(q, kp, lse, m)]
        if given:
            out = torch.empty_like(q)
            assert psa.psa_decode(q, k, v, n, out=out) is out
            assert psa.psa_key_weight(q, k, lse, n, score=score, out=score) is score
            a += [out, score.clone()]
            bufs = (k.clone(), v.clone(), score, pos.clone(), n.clone(),
                    torch.empty(B, H, 50, dtype=torch.int32, device="cuda"))
            got = psa.psa_cache_evict(*bufs[:3], 50, pos=bufs[3], cache_len=bufs[4], sink=2, recent=9, out=bufs)
            assert all(x is y for x, y in zip(got, bufs))
        else:
            got = psa.psa_cache_evict(k, v, score, 50, cache_len=n, recent=9)
        kept = got[5] >= 0
        return a + [t[:, :, :50][kept] for t in got[:4]] + [got[4], got[5]]

    for given in (False, True):
        native = run(given)
        with monkeypatch.context() as mp:
            mp.setattr(psa, "_native", None)
            python = run(given)
        assert len(native) == len(python) and all(torch.equal(x, y) for x, y in zip(native, python))


def test_what_the_native_calls_leave_to_python_is_refused():
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(2, 2, 8, 64, generator=g).bfloat16().cuda() for _ in range(3))
    n = torch.tensor([8, 5], dtype=torch.int32, device="cuda")
    out, lse = psa.psa_decode(q, k, v, n, want_lse=True)
    score = psa.psa_key_weight(q, k, lse, n)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for bad in (dict(k_cache=k.half()), dict(cache_len=n.long()), dict(cache_len=n[:1]), dict(v_cache=v[:, :, :4]),
                dict(v_cache=v.transpose(1, 2)), dict(k_cache=k.cpu()), dict(ws=small), dict(lse=lse[:1]),
                dict(out=out.float()), dict(v_cache=None), dict(q=q.float()), dict(q=q[0]), dict(q=None),
                dict(prefix_len=n)):
        with pytest.raises((ValueError, AttributeError)):
            psa.psa_decode(**{**dict(q=q, k_cache=k, v_cache=v, cache_len=n), **bad})
    for bad in (dict(out=k), dict(out=q[:, :, :4])):
        with pytest.raises((ValueError, psa.PSAError)):
            psa.psa_decode(**{**dict(q=q, k_cache=k, v_cache=v, cache_len=n), **bad})
    for bad in (dict(lse=None), dict(lse=lse.half()), dict(key_len=n.cpu()), dict(score=score[..., :4]),
                dict(out=score.double()), dict(k=k[:1]), dict(ws=small[:10])):
        with pytest.raises((ValueError, psa.PSAError)):
            psa.psa_key_weight(**{**dict(q=q, k=k, lse=lse, key_len=n), **bad})
    for bad in (dict(budget=0), dict(budget=9), dict(sink=3, recent=2), dict(pos=n), dict(score=score.half()),
                dict(out=(k, v, score, None, n, n)), dict(out=(k, v.clone(), score, n, n, n))):
        with pytest.raises((ValueError, psa.PSAError)):
            psa.psa_cache_evict(**{**dict(k=k, v=v, score=score, budget=4, cache_len=n), **bad})
    assert torch.equal(out, psa.psa_decode(q, k, v, n))
