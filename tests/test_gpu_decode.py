"""psa_decode against the float64 restatement.

Tolerance, element by element.  u = eps / 2 of the type (2^-8 bf16, 2^-11
fp16).  Every softmax term is rounded once to the type for the tensor core:
at most u of it, or in fp16 half a step of its subnormals, 2^-25, where a
part's largest term is at least 1 (its reference never passes its maximum):
together u * sum p|v| + 2^-25 * sum|v| / sum e^(s - max).  The output is rounded
once more: u * |out|.  fp32: a logit of d products is off by at most about
(d + 2) 2^-24 sum_c |q_c k_c| / sqrt(d), below 2e-4 for these inputs
(sum_c |q_c k_c| / sqrt(d) < 25); numerator and denominator each carry it,
with the sums' own roundings: 5e-4 * sum p|v| in all, 5e-4 on lse."""

import numpy as np
import pytest
import torch

import oracle.psa_oracle_serve as O
from block_sparse_attention_psa_b200 import psa

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(B, Bp, Hq, Hkv, T, d, P, C, dtype, seed=0, clens=None, plens=None, junk=float("nan")):
    g = torch.Generator().manual_seed(seed)
    x = dict(q=torch.randn(B, Hq, T, d, generator=g).to(dtype))
    for name, n, cap, lens in (("cache", B, C, clens), ("prefix", Bp, P, plens)):
        if not cap:
            x["k_" + name] = x["v_" + name] = x[name + "_len"] = None
            continue
        if lens is None:
            lens = [cap] * n
        k = torch.randn(n, Hkv, cap, d, generator=g).to(dtype)
        v = torch.randn(n, Hkv, cap, d, generator=g).to(dtype)
        for i, m in enumerate(lens):
            k[i, :, max(m, 0):] = junk
            v[i, :, max(m, 0):] = junk
        x["k_" + name], x["v_" + name] = k, v
        x[name + "_len"] = torch.tensor(lens, dtype=torch.int32)
    return x


def on_gpu(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def check(x, out, lse):
    lens = lambda n: None if x[n] is None else x[n].tolist()  # noqa: E731
    clean = lambda n: None if x[n] is None else np.nan_to_num(f64(x[n]))  # noqa: E731
    ref, rl, spread, tiny = O.decode(f64(x["q"]), clean("k_cache"), clean("v_cache"), lens("cache_len"),
                                     clean("k_prefix"), clean("v_prefix"), lens("prefix_len"))
    u = U[x["q"].dtype]
    got, gl = f64(out), f64(lse)
    assert np.isfinite(got).all()
    tol = u * spread + 2.0 ** -25 * tiny + u * np.abs(ref) * (1 + u) + 5e-4 * spread
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    none = np.isneginf(rl)
    assert np.array_equal(none, np.isneginf(gl))
    assert np.abs(gl[~none] - rl[~none]).max(initial=0) <= 5e-4
    assert (got[none] == 0).all()


def run(x, **kw):
    y = on_gpu(x)
    ws = psa.decode_workspace(*_dims(x))
    out, lse = psa.psa_decode(y["q"], y["k_cache"], y["v_cache"], y["cache_len"], y["k_prefix"], y["v_prefix"],
                              y["prefix_len"], ws=ws, want_lse=True, **kw)
    assert psa.psa_read_status(ws) == psa.PSA_OK
    return out, lse


def _dims(x):
    B, Hq, T, d = x["q"].shape
    kc, kp = x["k_cache"], x["k_prefix"]
    Hkv = (kc if kc is not None else kp).shape[1]
    return (B, Hq, Hkv, T, d, kp.shape[0] if kp is not None else 1, kp.shape[2] if kp is not None else 0,
            kc.shape[2] if kc is not None else 0)


CASES = [
    # B, Bp, Hq, Hkv, T, d, P, C, dtype, cache lens, prefix lens
    (1, 1, 1, 1, 1, 128, 0, 1, "bf16", [1], None),
    (1, 1, 2, 2, 1, 64, 0, 64, "bf16", [64], None),
    (1, 1, 8, 2, 1, 128, 0, 1024, "bf16", [1000], None),
    (3, 1, 8, 2, 1, 128, 0, 300, "bf16", [0, 129, 300], None),                 # an empty row
    (2, 1, 4, 4, 1, 64, 0, 257, "fp16", [255, 257], None),
    (4, 1, 8, 2, 1, 128, 777, 0, "bf16", None, [777]),                         # no caches
    (4, 2, 6, 2, 1, 128, 200, 130, "bf16", [1, 63, 64, 65], [199, 0]),
    (6, 3, 12, 4, 5, 64, 1000, 100, "fp16", [5, 4, 1, 0, 100, 77], [1000, 1, 129]),   # fewer entries than tokens
    (40, 1, 16, 2, 1, 128, 2000, 40, "bf16", list(range(1, 41)), [1999]),      # several row tiles
    (33, 1, 24, 1, 2, 64, 515, 9, "bf16", [2 + i % 8 for i in range(33)], [515]),     # 48 rows per sequence
    (2, 1, 32, 1, 7, 128, 400, 333, "fp16", [333, 150], [390]),                # 224 rows per sequence
    (1, 1, 3, 1, 200, 64, 100, 500, "bf16", [450], [100]),                     # a chunk of 200 tokens
    (70, 70, 2, 1, 1, 64, 70, 70, "bf16", [i + 1 for i in range(70)], [i for i in range(70)]),  # a prefix each
    (1, 1, 5, 5, 3, 128, 5000, 130, "fp16", [130], [4999]),
    (500, 1, 2, 1, 1, 64, 0, 130, "bf16", [i % 131 for i in range(500)], None),       # more segments than threads
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:9]))
def test_against_the_definition(case):
    B, Bp, Hq, Hkv, T, d, P, C, dt, cl, pl = case
    x = make(B, Bp, Hq, Hkv, T, d, P, C, {"bf16": torch.bfloat16, "fp16": torch.float16}[dt], clens=cl, plens=pl)
    check(x, *run(x))


def test_rising_logits_move_the_reference():
    """Keys whose logits grow along the cache by far more than the lag."""
    x = make(2, 1, 4, 2, 1, 128, 900, 700, torch.bfloat16, junk=0.0)
    for n, cap in (("cache", 700), ("prefix", 900)):
        ramp = torch.linspace(0.0, 8.0, cap)[None, None, :, None]
        x["k_" + n] = (x["k_" + n].float() * 0.1 + ramp * x["q"][:1, :2, :1].float().sign()).bfloat16()
    x["q"] = (x["q"].float() * 0.3).bfloat16()   # sum_c |q_c k_c| / sqrt(d) stays below 25
    check(x, *run(x))


def test_one_key_far_above_the_rest():
    x = make(1, 1, 2, 1, 1, 64, 0, 600, torch.float16, clens=[600])
    x["k_cache"][0, 0, 431] = x["q"][0, 0, 0] * 2
    check(x, *run(x))


def test_bit_identical_on_repeats_and_after_other_shapes():
    x = make(16, 1, 32, 8, 1, 128, 3000, 200, torch.bfloat16, clens=[200 - i for i in range(16)])
    a = run(x)
    run(make(1, 1, 2, 2, 1, 128, 0, 64, torch.bfloat16))
    b = run(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_lengths_are_clamped_and_reported():
    x = make(2, 1, 2, 1, 1, 64, 100, 90, torch.bfloat16, junk=0.0)
    y = on_gpu(x)
    ws = psa.decode_workspace(*_dims(x))
    y["cache_len"] = torch.tensor([-5, 1000], dtype=torch.int32).cuda()
    out, lse = psa.psa_decode(y["q"], y["k_cache"], y["v_cache"], y["cache_len"], y["k_prefix"], y["v_prefix"],
                              None, ws=ws, want_lse=True)
    assert psa.psa_read_status(ws) == psa.PSA_ERR_LENGTH
    x["cache_len"] = torch.tensor([0, 90], dtype=torch.int32)
    check(x, out, lse)
    y["cache_len"].copy_(x["cache_len"])
    psa.psa_decode(y["q"], y["k_cache"], y["v_cache"], y["cache_len"], y["k_prefix"], y["v_prefix"], None, ws=ws)
    assert psa.psa_read_status(ws) == psa.PSA_OK


def test_captured_graph_follows_the_lengths():
    x = make(3, 1, 4, 2, 1, 128, 300, 260, torch.bfloat16, junk=0.0)
    y = on_gpu(x)
    ws = psa.decode_workspace(*_dims(x))
    out, lse = torch.empty_like(y["q"]), torch.empty(3, 4, 1, device="cuda")
    call = lambda: psa.psa_decode(y["q"], y["k_cache"], y["v_cache"], y["cache_len"], y["k_prefix"],  # noqa: E731
                                  y["v_prefix"], y["prefix_len"], ws=ws, out=out, lse=lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, plen in (([1, 130, 260], 300), ([0, 0, 7], 0), ([260, 259, 128], 257)):
        x["cache_len"], x["prefix_len"] = torch.tensor(lens, dtype=torch.int32), torch.tensor([plen],
                                                                                              dtype=torch.int32)
        y["cache_len"].copy_(x["cache_len"])
        y["prefix_len"].copy_(x["prefix_len"])
        g.replay()
        torch.cuda.synchronize()
        check(x, out, lse)


def test_other_stream_and_own_workspaces():
    xs = [make(4, 1, 8, 2, 1, 128, 900, 100, torch.bfloat16, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    ys = [on_gpu(x) for x in xs]
    torch.cuda.synchronize()
    for y, st in zip(ys, streams):
        for _ in range(3):
            r = psa.psa_decode(y["q"], y["k_cache"], y["v_cache"], y["cache_len"], y["k_prefix"], y["v_prefix"],
                               y["prefix_len"], ws=torch.empty(psa.psa_decode_workspace_size(4, 8, 2, 1, 128, 1, 900,
                                                                                             100),
                                                               dtype=torch.uint8, device="cuda"),
                               want_lse=True, stream=st)
        got.append(r)
        torch.cuda.synchronize()
    for x, r in zip(xs, got):
        check(x, *r)
