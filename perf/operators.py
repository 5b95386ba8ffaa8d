"""The serving operators measured: attention of new tokens over a shared
prefix and their own caches, accumulated attention weight per cached key, and
eviction from a cache by that weight.

``run`` computes them in plain torch operations, or, where ``own`` is true,
through the library's entry points.  ``exact`` restates each in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # -- psa_decode: new tokens over a shared prefix and their own caches
        # one conversation right after a short prompt: nothing but latency
        dict(name="decode_one_short", op="decode", B=1, Bp=1, Hq=2, Hkv=2, T=1, d=64, P=0, C=1024, dtype="bf16"),
        # a batch of unrelated conversations with ragged caches, no common prefix
        dict(name="decode_ragged_batch", op="decode", B=64, Bp=1, Hq=32, Hkv=8, T=1, d=128, P=0, C=4096, dtype="bf16"),
        # sixteen samples of one 32K prompt, the prompt's keys read once for all
        dict(name="decode_shared_32k", op="decode", B=16, Bp=1, Hq=32, Hkv=8, T=1, d=128, P=32768, C=512,
             dtype="bf16"),
        # a wide batch over one 128K document: many rows per key, the largest work
        dict(name="decode_shared_128k", op="decode", B=64, Bp=1, Hq=64, Hkv=8, T=1, d=128, P=131072, C=1024,
             dtype="bf16"),
        # five drafted tokens per sequence, three prompts of odd lengths, other type and head size
        dict(name="decode_drafts_odd", op="decode", B=21, Bp=3, Hq=24, Hkv=8, T=5, d=64, P=10007, C=777,
             dtype="fp16"),
        # -- psa_key_weight: accumulated attention weight of each key
        # every query of a causal prefill, to rank its keys
        dict(name="weight_prefill_8k", op="weight", B=1, Bk=1, Hq=32, Hkv=8, T=8192, d=128, C=8192, causal=True,
             dtype="bf16"),
        # the last 64 queries of a 128K prefill (an observation window)
        dict(name="weight_window_128k", op="weight", B=1, Bk=1, Hq=32, Hkv=8, T=64, d=128, C=131072, causal=True,
             dtype="bf16"),
        # one decoded token of a ragged batch, added to what the keys have so far
        dict(name="weight_decode_batch", op="weight", B=48, Bk=48, Hq=24, Hkv=8, T=1, d=64, C=4099, causal=True,
             dtype="fp16"),
        # -- psa_cache_evict
        # one token over the budget of a small cache: the step of a decode loop
        dict(name="evict_one_token", op="evict", B=1, Hkv=2, d=64, C=1025, budget=1024, sink=4, recent=64,
             dtype="bf16"),
        # a batch of ragged caches back to its budget
        dict(name="evict_ragged_batch", op="evict", B=32, Hkv=8, d=128, C=5001, budget=4096, sink=4, recent=512,
             dtype="bf16"),
        # a 128K prefill down to 16K entries
        dict(name="evict_prefill_128k", op="evict", B=1, Hkv=8, d=128, C=131072, budget=16384, sink=16, recent=1024,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "weight", "evict"))
    d, dtype = rng.choice((64, 128)), rng.choice(("bf16", "fp16"))
    Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    if op == "decode":
        Bp, n, T = rng.choice((1, 1, 2, 3)), _log(rng, 1, 32), rng.choice((1, 1, 2, 5, 8))
        P = _log(rng, 64, 65536) if rng.random() < 0.7 else 0
        P = min(P, (1 << 28) // (Bp * n * Hkv * G * T))
        C = _log(rng, max(T, 16), 4096)
        return dict(op=op, B=Bp * n, Bp=Bp, Hq=Hkv * G, Hkv=Hkv, T=T, d=d, P=P, C=C, dtype=dtype)
    if op == "weight":
        kind = rng.choice(("prefill", "window", "decode", "prefix"))
        if kind == "prefill":
            C = _log(rng, 64, 4096)
            return dict(op=op, B=1, Bk=1, Hq=Hkv * G, Hkv=Hkv, T=C, d=d, C=C, causal=True, dtype=dtype)
        if kind == "window":
            C = _log(rng, 256, 65536)
            return dict(op=op, B=1, Bk=1, Hq=Hkv * G, Hkv=Hkv, T=_log(rng, 8, 200), d=d, C=C, causal=True,
                        dtype=dtype)
        if kind == "decode":
            B = _log(rng, 1, 64)
            return dict(op=op, B=B, Bk=B, Hq=Hkv * G, Hkv=Hkv, T=1, d=d, C=_log(rng, 64, 8192), causal=True,
                        dtype=dtype)
        Bk, n = rng.choice((1, 2)), _log(rng, 2, 32)
        return dict(op=op, B=Bk * n, Bk=Bk, Hq=Hkv * G, Hkv=Hkv, T=1, d=d, C=_log(rng, 256, 32768), causal=False,
                    dtype=dtype)
    B, C = _log(rng, 1, 32), _log(rng, 65, 16384)
    budget = max(1, int(C * rng.uniform(0.1, 0.999)))
    return dict(op=op, B=B, Hkv=Hkv, d=d, C=C, budget=budget, sink=min(4, budget // 4), recent=budget // 8,
                dtype=dtype)


def _lens(case, count, lo, hi):
    """`count` lengths in [lo, hi], the same for every seed (they set the work)."""
    if count == 1:
        return [hi]
    # a golden-ratio sequence: spread evenly, the largest at hi
    got = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(count)]
    got[0] = hi
    return got


def _cache_lens(case):
    return _lens(case, case["B"], min(case["T"], case["C"]), case["C"])


def _prefix_lens(case):
    return _lens(case, case["Bp"], max(1, case["P"] // 2), case["P"])


def _key_lens(case):
    return _lens(case, case["Bk"], min(max(case["T"], case["C"] // 8), case["C"]), case["C"])


def _evict_lens(case):
    return _lens(case, case["B"], max(1, case["budget"] // 2), case["C"])


def _keys(shape, dtype, g):
    """Keys of which one in 64 is long (heavy hitters), the others N(0, 1)."""
    k = torch.randn(shape, device="cuda", generator=g)
    heavy = torch.rand(shape[:-1], device="cuda", generator=g) < 1 / 64
    return (k * torch.where(heavy, 3.0, 1.0)[..., None]).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, d = DTYPES[case["dtype"]], case["d"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] == "decode":
        B, Bp, Hq, Hkv, T, P, C = (case[x] for x in ("B", "Bp", "Hq", "Hkv", "T", "P", "C"))
        s["q"] = torch.randn((B, Hq, T, d), device="cuda", generator=g).to(dt)
        s["k"] = _keys((B, Hkv, C, d), dt, g)
        s["v"] = torch.randn((B, Hkv, C, d), device="cuda", generator=g).to(dt)
        s["len"] = ints(_cache_lens(case))
        if P:
            s["kp"] = _keys((Bp, Hkv, P, d), dt, g)
            s["vp"] = torch.randn((Bp, Hkv, P, d), device="cuda", generator=g).to(dt)
            s["plen"] = ints(_prefix_lens(case))
    elif case["op"] == "weight":
        B, Bk, Hq, Hkv, T, C = (case[x] for x in ("B", "Bk", "Hq", "Hkv", "T", "C"))
        s["q"] = torch.randn((B, Hq, T, d), device="cuda", generator=g).to(dt)
        s["k"] = _keys((Bk, Hkv, C, d), dt, g)
        s["len"] = ints(_key_lens(case))
        # each query's own log sum, as the attention that ran before gives it
        n, G = B // Bk, Hq // Hkv
        lse = torch.empty((B, Hq, T), device="cuda")
        slot = torch.arange(C, device="cuda")
        for b in range(B):
            last = s["len"][b // n] - (T - 1 - torch.arange(T, device="cuda")) if case["causal"] \
                else s["len"][b // n].expand(T)
            for h in range(Hkv):
                z = (s["q"][b, h * G:(h + 1) * G] @ s["k"][b // n, h].T).float() / math.sqrt(d)
                z = z.masked_fill(slot >= last[:, None], -math.inf)
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
        s["lse"] = lse
        s["score"] = torch.rand((Bk, Hkv, C), device="cuda", generator=g)
    else:
        B, Hkv, C, budget = (case[x] for x in ("B", "Hkv", "C", "budget"))
        s["k"] = _keys((B, Hkv, C, d), dt, g)
        s["v"] = torch.randn((B, Hkv, C, d), device="cuda", generator=g).to(dt)
        # accumulated weights: heavy tailed, with ties (many keys at exactly zero)
        e = torch.rand((B, Hkv, C), device="cuda", generator=g)
        s["score"] = torch.where(e < 0.05, 0.0, (e * 8 - 4).exp())
        s["pos"] = torch.arange(C, device="cuda", dtype=torch.int32).expand(B, Hkv, C).contiguous()
        s["len"] = ints(_evict_lens(case))
        # the smaller cache that takes the entries (also a user's own tensors)
        s["out"] = (torch.zeros((B, Hkv, budget, d), device="cuda", dtype=dt),
                    torch.zeros((B, Hkv, budget, d), device="cuda", dtype=dt),
                    torch.zeros((B, Hkv, budget), device="cuda"),
                    torch.zeros((B, Hkv, budget), device="cuda", dtype=torch.int32),
                    torch.zeros((B,), device="cuda", dtype=torch.int32),
                    torch.zeros((B, Hkv, budget), device="cuda", dtype=torch.int32))
    return s


def run(state):
    if own:
        return _run_own(state)
    return {"decode": _plain_decode, "weight": _plain_weight, "evict": _plain_evict}[state["case"]["op"]](state)


def _run_own(s):
    from block_sparse_attention_psa_b200 import psa

    case = s["case"]
    if case["op"] == "decode":
        if "ws" not in s:
            s["ws"] = psa.decode_workspace(case["B"], case["Hq"], case["Hkv"], case["T"], case["d"], case["Bp"],
                                           case["P"], case["C"], device=s["q"].device)
        out, lse = psa.psa_decode(s["q"], s["k"], s["v"], s["len"], s.get("kp"), s.get("vp"), s.get("plen"),
                                  ws=s["ws"], want_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "weight":
        if "ws" not in s:
            s["ws"] = psa.key_weight_workspace(case["B"], case["Hq"], case["Hkv"], case["T"], case["d"], case["Bk"],
                                               case["C"], device=s["q"].device)
        return {"score": psa.psa_key_weight(s["q"], s["k"], s["lse"], s["len"], causal=case["causal"],
                                            score=s["score"], ws=s["ws"])}
    if "ws" not in s:
        s["ws"] = psa.cache_evict_workspace(case["B"], case["Hkv"], case["C"], case["budget"], device=s["k"].device)
    k, v, score, pos, n, kept = psa.psa_cache_evict(s["k"], s["v"], s["score"], case["budget"], pos=s["pos"],
                                                    cache_len=s["len"], sink=case["sink"], recent=case["recent"],
                                                    ws=s["ws"], out=s["out"])
    return {"k": k, "v": v, "score": score, "pos": pos, "len": n, "kept": kept}


def _plain_decode(s):
    c = s["case"]
    B, Bp, Hq, Hkv, T, d, P, C = (c[x] for x in ("B", "Bp", "Hq", "Hkv", "T", "d", "P", "C"))
    n, G = B // Bp, Hq // Hkv
    q = s["q"].float().view(B, Hkv, G * T, d) / math.sqrt(d)
    seen = s["len"][:, None] - (T - 1 - torch.arange(T, device="cuda"))            # [B, T]
    hide = torch.arange(C, device="cuda") >= seen.repeat(1, G)[:, None, :, None]   # [B, 1, G T, C]
    past = torch.arange(C, device="cuda")[:, None] >= s["len"][:, None, None, None]
    z = (q @ s["k"].float().mT).masked_fill(hide, -math.inf)
    m = z.amax(-1, keepdim=True)
    if P:
        qp = q.view(Bp, n, Hkv, G * T, d).transpose(1, 2).reshape(Bp, Hkv, n * G * T, d)
        hp = torch.arange(P, device="cuda") >= s["plen"][:, None, None, None]      # [Bp, 1, 1, P]
        zp = (qp @ s["kp"].float().mT).masked_fill(hp, -math.inf)
        back = lambda x: x.view(Bp, Hkv, n, G * T, -1).transpose(1, 2).reshape(B, Hkv, G * T, -1)  # noqa: E731
        m = torch.maximum(m, back(zp.amax(-1, keepdim=True)))
    m = m.masked_fill(m == -math.inf, 0.0)
    p = (z - m).exp()
    num, den = p @ s["v"].float().masked_fill(past, 0.0), p.sum(-1, keepdim=True)
    if P:
        mp = m.view(Bp, n, Hkv, G * T, 1).transpose(1, 2).reshape(Bp, Hkv, n * G * T, 1)
        pp = (zp - mp).exp()
        num = num + back(pp @ s["vp"].float().masked_fill(hp.mT, 0.0))
        den = den + back(pp.sum(-1, keepdim=True))
    out = (num / den).masked_fill(den == 0, 0.0)
    return {"out": out.view(B, Hq, T, d).to(s["q"].dtype), "lse": (m + den.log()).view(B, Hq, T)}


def _plain_weight(s):
    c = s["case"]
    B, Bk, Hq, Hkv, T, d, C = (c[x] for x in ("B", "Bk", "Hq", "Hkv", "T", "d", "C"))
    n, G = B // Bk, Hq // Hkv
    q = s["q"].float().view(Bk, n, Hkv, G * T, d).transpose(1, 2).reshape(Bk, Hkv, n * G * T, d) / math.sqrt(d)
    lse = s["lse"].view(Bk, n, Hkv, G * T).transpose(1, 2).reshape(Bk, Hkv, n * G * T, 1)
    slot = torch.arange(C, device="cuda")
    t = torch.arange(T, device="cuda").repeat(n * G)
    seen = s["len"][:, None] - (T - 1 - t if c["causal"] else 0 * t)               # [Bk, n G T]
    w = (q @ s["k"].float().mT - lse).exp()
    w = w.masked_fill(slot >= seen[:, None, :, None], 0.0).sum(-2)
    return {"score": torch.where(slot < s["len"][:, None, None], s["score"] + w, 0.0)}


def _plain_evict(s):
    c = s["case"]
    B, Hkv, C, budget = (c[x] for x in ("B", "Hkv", "C", "budget"))
    slot = torch.arange(C, device="cuda").expand(B, Hkv, C)
    length = s["len"].long()[:, None, None]
    there = slot < length
    last = s["pos"].masked_fill(~there, -1).amax(-1, keepdim=True)
    guard = (s["pos"] < c["sink"]) | (s["pos"] > last - c["recent"])
    rank = torch.where(there, torch.where(guard, 2, 1), 0)
    score = s["score"].masked_fill(s["score"].isnan(), -math.inf)
    order = score.argsort(dim=-1, descending=True, stable=True)
    order = order.gather(-1, rank.gather(-1, order).argsort(dim=-1, descending=True, stable=True))
    nk = length.clamp(max=budget)
    keep = torch.zeros_like(there).scatter(-1, order, slot < nk)
    # holes below nk take the survivors from nk on, both in ascending order
    far = torch.where(keep & (slot >= nk), slot, C).sort(-1).values
    hole = ~keep & (slot < nk)
    src = torch.where(hole, far.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), slot)[..., :budget]
    ok = slot[..., :budget] < nk
    src = torch.where(ok, src, 0)
    k_out, v_out, score_out, pos_out = s["out"][:4]
    row = src[..., None].expand(-1, -1, -1, c["d"])
    return {"k": torch.where(ok[..., None], s["k"].gather(2, row), k_out),
            "v": torch.where(ok[..., None], s["v"].gather(2, row), v_out),
            "score": torch.where(ok, s["score"].gather(2, src), score_out),
            "pos": torch.where(ok, s["pos"].gather(2, src), pos_out),
            "len": nk.view(B).int(), "kept": torch.where(ok, src, -1).int()}


def work(case):
    d = case["d"]
    if case["op"] == "decode":
        B, Bp, Hq, Hkv, T = (case[x] for x in ("B", "Bp", "Hq", "Hkv", "T"))
        own_keys = sum(_cache_lens(case))
        prefix_keys = sum(_prefix_lens(case)) if case["P"] else 0
        rows = B * Hq * T
        return {"bytes": (own_keys + prefix_keys) * Hkv * d * 4 + rows * (d * 4 + 4),
                "flops": 4 * d * Hq * T * (own_keys + prefix_keys * (B // Bp))}
    if case["op"] == "weight":
        B, Bk, Hq, Hkv, T, C = (case[x] for x in ("B", "Bk", "Hq", "Hkv", "T", "C"))
        lens = _key_lens(case)
        pairs = sum(T * n - (T * (T - 1) // 2 if case["causal"] else 0) for n in lens) * (B // Bk)
        return {"bytes": sum(lens) * Hkv * (2 * d + 4) + Bk * Hkv * C * 4 + B * Hq * T * (2 * d + 4),
                "flops": 2 * d * Hq * pairs}
    lens = _evict_lens(case)
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": case["Hkv"] * (sum(lens) * 8 + kept * (8 * d + 12)), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "decode":
        B, Bp, Hq, Hkv, T, P, C = (case[x] for x in ("B", "Bp", "Hq", "Hkv", "T", "P", "C"))
        n, G = B // Bp, Hq // Hkv
        out = torch.zeros((B, Hq, T, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
        lens, plens = _cache_lens(case), _prefix_lens(case) if P else [0] * Bp
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            for p in range(Bp):
                seqs = range(p * n, (p + 1) * n)
                qs = s["q"][p * n:(p + 1) * n, heads].double().reshape(n * G * T, d)
                zp = vp = None
                if P:
                    zp = (qs @ s["kp"][p, h, :plens[p]].double().T / math.sqrt(d)).view(n, G, T, -1)
                    vp = s["vp"][p, h, :plens[p]].double()
                for b in seqs:
                    z = s["q"][b, heads].double() @ s["k"][b, h, :lens[b]].double().T / math.sqrt(d)
                    t, j = torch.arange(T, device="cuda")[:, None], torch.arange(lens[b], device="cuda")
                    z = torch.where(j <= lens[b] - T + t, z, -math.inf)
                    v = s["v"][b, h, :lens[b]].double()
                    if P:
                        z, v = torch.cat([zp[b - p * n], z], -1), torch.cat([vp, v])
                    total = torch.logsumexp(z, -1)
                    lse[b, heads] = total
                    out[b, heads] = torch.exp(z - total[..., None]) @ v
        return {"out": out, "lse": lse}
    if case["op"] == "weight":
        B, Bk, Hq, Hkv, T, C = (case[x] for x in ("B", "Bk", "Hq", "Hkv", "T", "C"))
        n, G, lens = B // Bk, Hq // Hkv, _key_lens(case)
        score = torch.zeros((Bk, Hkv, C), dtype=torch.float64, device="cuda")
        for b in range(Bk):
            j = torch.arange(lens[b], device="cuda")
            for h in range(Hkv):
                total = s["score"][b, h, :lens[b]].double()
                for i in range(b * n, (b + 1) * n):
                    for g in range(h * G, (h + 1) * G):
                        z = s["q"][i, g].double() @ s["k"][b, h, :lens[b]].double().T / math.sqrt(d)
                        e = torch.exp(z - s["lse"][i, g].double()[:, None])
                        if case["causal"]:
                            e = torch.where(j <= lens[b] - T + torch.arange(T, device="cuda")[:, None], e, 0.0)
                        total = total + e.sum(0)
                score[b, h, :lens[b]] = total
        return {"score": score}
    # eviction moves values: what it gives is exact, checked entry by entry
    B, Hkv, C, budget = (case[x] for x in ("B", "Hkv", "C", "budget"))
    lens = _evict_lens(case)
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int64)
    score, pos = s["score"].cpu(), s["pos"].cpu()
    for b in range(B):
        m = lens[b]
        nk = min(m, budget)
        for h in range(Hkv):
            sc, ps = score[b, h, :m].numpy(), pos[b, h, :m].numpy()
            top = int(ps.max())
            safe = (ps < case["sink"]) | (ps > top - case["recent"])
            # ascending in (not protected, -score, slot)
            key = sorted(range(m), key=lambda i: (not safe[i], -float(sc[i]), i)) if m > nk else range(m)
            stay = set(key[:nk])
            late = iter(sorted(i for i in stay if i >= nk))
            kept[b, h, :nk] = torch.tensor([i if i in stay else next(late) for i in range(nk)])
    at = kept.clamp(min=0).cuda()
    ok = (kept >= 0).cuda()
    row = at[..., None].expand(-1, -1, -1, d)
    return {"k": s["k"].gather(2, row).double() * ok[..., None], "v": s["v"].gather(2, row).double() * ok[..., None],
            "score": s["score"].gather(2, at).double() * ok, "pos": s["pos"].gather(2, at).long() * ok,
            "len": torch.tensor([min(m, budget) for m in lens]), "kept": kept}
