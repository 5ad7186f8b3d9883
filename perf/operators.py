"""Serving operators around the latent cache: their plain forms, inputs and work.

Three operators, used together when many requests are decoded over one prompt
and their caches are kept within a budget:

  shared   one decode step of a batch whose sequences share a prefix: every
           sequence attends the prefix's latent rows (stored once) and then
           its own; optionally with the weights of its own rows
  weights  one decode step that also gives each cache row's attention weight,
           summed over the heads (and added to what earlier steps gave)
  evict    the rows of a cache that stay within a budget: the first ``sink``,
           the last ``recent`` and the heaviest of the others, in order

``run`` computes them with elementary torch operations in 32 bits where
``own`` is false, and through the package's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
F16 = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def _shared(name, cache, B, H, d_h, r, prefix, lo, hi, weights=False):
    c = {"op": "shared", "cache": cache, "B": B, "H": H, "d_h": d_h, "r": r, "prefix": prefix,
         "lo": lo, "hi": hi, "weights": weights}
    return dict(c, name=name) if name else c


def _weights(name, cache, B, H, d_h, r, lo, hi, rope=False, add=False):
    c = {"op": "weights", "cache": cache, "B": B, "H": H, "d_h": d_h, "r": r, "lo": lo, "hi": hi,
         "rope": rope, "add": add}
    return dict(c, name=name) if name else c


def _evict(name, cache, B, r, lo, hi, budget, sink, recent):
    c = {"op": "evict", "cache": cache, "B": B, "r": r, "lo": lo, "hi": hi, "budget": budget,
         "sink": sink, "recent": recent}
    return dict(c, name=name) if name else c


def listed():
    return [
        # two requests on a short prompt, a few tokens in: what a call costs when there is little to do
        _shared("shared-f16-short", "f16", 2, 4, 64, 256, 77, 1, 9),
        # the 7B layer, 16 requests over one long prompt, some hundred tokens into their answers
        _shared("shared-f16-7b", "f16", 16, 32, 128, 1536, 8192, 65, 512, weights=True),
        # bf16, an odd prefix, answers about as long as half of it
        _shared("shared-bf16-odd", "bf16", 24, 32, 128, 1536, 2001, 0, 1000),
        # a bf16 layer with a quantised cache: 32 requests over a prompt of 4096 tokens
        _shared("shared-int8", "i8", 32, 32, 128, 768, 4096, 1, 256),
        # the largest batch over the longest prompt
        _shared("shared-f16-large", "f16", 64, 32, 128, 1536, 16384, 128, 1024),
        # a small ragged batch, an empty sequence among it
        _weights("weights-bf16-short", "bf16", 3, 8, 64, 256, 0, 700, add=True),
        # the 7B layer at full batch and length
        _weights("weights-f16-7b", "f16", 16, 32, 128, 1536, 8192, 8192),
        # the same layer alone, long and ragged
        _weights("weights-int8-long", "i8", 32, 32, 128, 768, 4000, 16384),
        # rotary keys, ragged
        _weights("weights-bf16-rope", "bf16", 4, 32, 128, 1536, 1000, 4096, rope=True),
        # a few short sequences, cut to 64 rows
        _evict("evict-f16-short", "f16", 4, 256, 40, 301, 64, 4, 16),
        # the 7B layer's caches cut to half
        _evict("evict-f16-7b", "f16", 16, 1536, 8192, 8192, 4096, 4, 1024),
        # one long sequence cut to an eighth
        _evict("evict-bf16-long", "bf16", 1, 1536, 60001, 60001, 7500, 4, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "weights", "evict"])
    if op == "evict":
        B, hi = _log(rng, 1, 32), _log(rng, 16, 20000)
        r = 32 * _log(rng, 4, 48)
        cache = rng.choice(["f16", "bf16", "f32"])
        hi = max(16, min(hi, (60000 if cache == "f32" else 130000) // B))
        budget = _log(rng, 8, hi)
        sink = rng.randint(0, min(4, budget))
        return _evict(None, cache, B, r, rng.randint(0, hi), hi, budget, sink,
                      rng.randint(0, (budget - sink) // 2))
    H, d_h = rng.choice([(4, 64), (8, 64), (8, 128), (16, 128), (32, 128)])
    r = 128 * rng.randint(1, min(12, H * d_h // 128))
    if op == "shared":
        B, prefix, hi = _log(rng, 1, 64), _log(rng, 1, 16000), _log(rng, 1, 1000)
        return _shared(None, rng.choice(["f16", "bf16", "i8"]), B, H, d_h, r, prefix, rng.randint(0, hi), hi,
                       weights=rng.random() < 0.5)
    rope = d_h == 128 and rng.random() < 0.3
    B, hi = _log(rng, 1, 4 if rope else 32), _log(rng, 1, 3000 if rope else 16000)
    hi = max(1, min(hi, 130000 // B))
    return _weights(None, rng.choice(["f16", "bf16"] if rope else ["f16", "bf16", "i8"]), B, H, d_h, r,
                    rng.randint(0, hi), hi, rope=rope, add=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The batch's lengths: spread evenly from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _max_len(case):
    return case["hi"] + 8   # room for the next tokens


def _weight(case):
    """The weights' and outputs' type: the cache's, bf16 beside a quantised one."""
    return "bf16" if case["cache"] == "i8" else case["cache"]


def _rows(g, n, r, cache, spectrum):
    """n latent rows with falling channel magnitudes, as the cache holds them: (rows or int8 codes, group scales)."""
    x = torch.randn(n, r, generator=g, device=DEV) * spectrum
    if cache != "i8":
        return x.to(F16[cache]), None
    v = x.view(n, r // 128, 128)
    s = (v.abs().amax(-1) / 127).to(torch.float16)
    codes = (v / s.float().unsqueeze(-1)).round().clamp(-127, 127)
    return codes.to(torch.int8).view(n, r), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    B, r, max_len = case["B"], case["r"], _max_len(case)
    spectrum = (1.0 + torch.arange(r, device=DEV)).pow(-0.4)
    spectrum = spectrum * (r / spectrum.square().sum()).sqrt()
    order = torch.randperm(B, generator=g, device=DEV)
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)[order].contiguous()
    s = {"case": dict(case), "lengths": lengths}
    cache, scales = _rows(g, B * max_len, r, case["cache"], spectrum)
    s["cache"] = cache.view(B, max_len, r)
    s["scales"] = None if scales is None else scales.view(B, max_len, r // 128)
    if case["op"] == "evict":
        # weights summed over many steps: heavy-tailed, some rows never looked at
        w = torch.exp(2.0 * torch.randn(B, max_len, generator=g, device=DEV))
        s["weights"] = torch.where(torch.rand(B, max_len, generator=g, device=DEV) < 0.05, 0.0, w)
        n = case["budget"]
        s["dst"] = {"cache": torch.zeros(B, n, r, dtype=s["cache"].dtype, device=DEV),
                    "weights": torch.zeros(B, n, device=DEV),
                    "lengths": torch.zeros(B, dtype=torch.int32, device=DEV),
                    "kept": torch.zeros(B, n, dtype=torch.int32, device=DEV)}
    else:
        H, d_h = case["H"], case["d_h"]
        E = H * d_h
        wt = F16[_weight(case)]
        # queries and keys of unit variance per channel; queries twice that, so that scores spread over some units
        up = lambda scale: (torch.randn(r, E, generator=g, device=DEV) * (scale / math.sqrt(r))).to(wt)  # noqa: E731
        s["wuq"], s["wuk"], s["wuv"] = up(2.0), up(1.0), up(1.0)
        s["qin"] = torch.randn(B, r, generator=g, device=DEV) * spectrum
        s["out"] = torch.zeros(B, E, dtype=wt, device=DEV)
        s["weights"] = torch.zeros(B, max_len, device=DEV)
        s["before"] = torch.rand(B, max_len, generator=g, device=DEV)   # weights that earlier steps gave
        if case["op"] == "shared":
            s["prefix"], s["prefix_scales"] = _rows(g, case["prefix"], r, case["cache"], spectrum)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    import rank_joint_qkv_b200 as q
    c = s["case"]
    if c["op"] == "evict":
        s["dims"] = q.make_dims(64, 1, 64, c["r"], c["B"], _max_len(c), cache=c["cache"])
        s["workspace"] = torch.empty(q.evict_workspace_bytes(s["dims"], c["budget"]), dtype=torch.uint8, device=DEV)
        return
    wt = _weight(c)
    d = s["dims"] = q.make_dims(c["H"] * c["d_h"], c["H"], c["d_h"], c["r"], c["B"], _max_len(c), cache=c["cache"],
                                weight=wt, out=wt, rope=c.get("rope", False))
    wd = torch.zeros(d.E, d.r, dtype=s["wuq"].dtype, device=DEV)   # not used by a decode step
    s["packed"] = q.qsvd_prepare_weights(d, wd, s["wuq"], s["wuk"], s["wuv"])
    n = (q.decode_shared_workspace_bytes(d, c["prefix"]) if c["op"] == "shared"
         else q.decode_weights_workspace_bytes(d))
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)


# --------------------------------------------------------------------- run

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import rank_joint_qkv_b200 as q
    c = s["case"]
    if c["op"] == "evict":
        d = s["dst"]
        q.qsvd_evict_rows(s["dims"], s["weights"], s["lengths"], c["budget"], s["cache"], s["scales"], sink=c["sink"],
                          recent=c["recent"], dst_max_len=c["budget"], dst_cache=d["cache"], dst_weights=d["weights"],
                          dst_lengths=d["lengths"], kept=d["kept"], workspace=s["workspace"])
        return d
    if c["op"] == "shared":
        q.qsvd_decode_attn_shared(s["dims"], s["packed"], s["qin"], True, s["prefix"], s["prefix_scales"], c["prefix"],
                                  s["cache"], s["scales"], s["lengths"], s["out"],
                                  weights=s["weights"] if c["weights"] else None, accumulate=False,
                                  workspace=s["workspace"])
        return {"out": s["out"], "weights": s["weights"]} if c["weights"] else {"out": s["out"]}
    if c["add"]:
        s["weights"].copy_(s["before"])
    q.qsvd_decode_attn_weights(s["dims"], s["packed"], s["qin"], True, s["cache"], s["scales"], s["lengths"], s["out"],
                               s["weights"], accumulate=c["add"], workspace=s["workspace"])
    return {"out": s["out"], "weights": s["weights"]}


def _values(rows, scales):
    """Cache rows as float32 values."""
    if scales is None:
        return rows.float()
    return (rows.float().view(*scales.shape, 128) * scales.float().unsqueeze(-1)).view(rows.shape)


def _rotate(x, cos, sin):
    """Rotary embedding of pairs (i, i + d_h / 2)."""
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "evict":
        return _plain_evict(s, c)
    B, H, d_h, r = c["B"], c["H"], c["d_h"], c["r"]
    E, L = H * d_h, s["cache"].shape[1]
    lengths = s["lengths"].long()
    rows = _values(s["cache"], s["scales"])                                # B, L, r
    q = (s["qin"] @ s["wuq"].float()).view(B, H, d_h) / math.sqrt(d_h)
    wuk = s["wuk"].float().view(r, H, d_h)
    if c.get("rope"):
        i = torch.arange(d_h // 2, device=DEV, dtype=torch.float64)
        a = torch.arange(L, device=DEV, dtype=torch.float64)[:, None] * torch.pow(10000.0, -2.0 * i / d_h)
        cos, sin = a.cos().float(), a.sin().float()                        # L, d_h / 2
        at = (lengths - 1).clamp(min=0)
        q = _rotate(q, cos[at][:, None], sin[at][:, None])
        k = (rows.view(B * L, r) @ s["wuk"].float()).view(B, L, H, d_h)
        k = _rotate(k, cos[:, None], sin[:, None])
        scores = torch.einsum("bhd,blhd->bhl", q, k)
    else:
        qt = torch.einsum("bhd,rhd->bhr", q, wuk)                          # the query in latent space
        scores = qt @ rows.transpose(1, 2)                                 # B, H, L
    live = torch.arange(L, device=DEV)[None, None] < lengths[:, None, None]
    scores = scores.masked_fill(~live, -math.inf)
    if c["op"] == "shared":
        prefix = _values(s["prefix"], s["prefix_scales"])                  # P, r
        ahead = (qt.reshape(B * H, r) @ prefix.t()).view(B, H, -1)
        top = torch.maximum(scores.amax(-1), ahead.amax(-1))[..., None]
        e, f = torch.exp(scores - top), torch.exp(ahead - top)
        total = e.sum(-1, keepdim=True) + f.sum(-1, keepdim=True)
        z = e @ _zeroed(rows, live) + (f.reshape(B * H, -1) @ prefix).view(B, H, r)
    else:
        top = scores.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)                      # an empty sequence
        e = torch.exp(scores - top)
        total = e.sum(-1, keepdim=True)
        total = torch.where(total == 0, 1.0, total)
        z = e @ _zeroed(rows, live)
    out = torch.einsum("bhr,rhd->bhd", z / total, s["wuv"].float().view(r, H, d_h)).reshape(B, E).to(s["out"].dtype)
    if c["op"] == "shared" and not c["weights"]:
        return {"out": out}
    w = (e / total).sum(1)
    return {"out": out, "weights": torch.where(live[:, 0], s["before"] + w, s["before"]) if c.get("add") else w}


def _zeroed(rows, live):
    """Rows past a length as zeros (what they hold has no bearing)."""
    return torch.where(live[:, 0, :, None], rows, 0.0)


def _plain_evict(s, c):
    L, r = s["cache"].shape[1:]
    n = s["lengths"].long()[:, None]
    t = torch.arange(L, device=DEV)[None]
    key = torch.where((t < c["sink"]) | (t >= n - c["recent"]), math.inf, s["weights"])
    key = torch.where(t < n, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["budget"]]
    kept = torch.where(order < n, order, L).sort(1).values
    there = kept < n
    at = kept.clamp(max=L - 1)
    rows = torch.gather(s["cache"], 1, at[..., None].expand(-1, -1, r))
    return {"cache": torch.where(there[..., None], rows, torch.zeros((), dtype=rows.dtype, device=DEV)),
            "weights": torch.where(there, torch.gather(s["weights"], 1, at), 0.0),
            "lengths": n.clamp(max=c["budget"])[:, 0].int(),
            "kept": torch.where(there, kept, -1).int()}


# -------------------------------------------------------------------- work

def work(case):
    r, B, n = case["r"], case["B"], sum(_lengths(case))
    row = r * {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}[case["cache"]] + (r // 128 * 2 if case["cache"] == "i8" else 0)
    if case["op"] == "evict":
        kept = sum(min(x, case["budget"]) for x in _lengths(case))
        return {"bytes": 2 * kept * row + 4 * n + 8 * kept, "flops": 0}
    H, d_h, P = case["H"], case["d_h"], case.get("prefix", 0)
    E = H * d_h
    flops = 6 * B * r * E + 4 * H * r * (n + B * P)        # three projections; scores and sums over the rows
    if case.get("rope"):
        flops = 6 * B * r * E + n * (2 * r * E + 2 * E + 2 * H * r)   # keys rebuilt for their rotation
    data = (n + P) * row + 3 * r * E * 2 + B * (4 * r + 2 * E)
    if case["op"] == "weights" or case["weights"]:
        data += 4 * n * (2 if case.get("add") else 1)
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """From the definition, in 64 bits: keys and values of every row, one sequence after another."""
    s = prepare(case, seed)
    f64 = torch.float64
    lens = s["lengths"].tolist()
    if case["op"] == "evict":
        return _exact_evict(case, s, lens)
    B, H, d_h, r = case["B"], case["H"], case["d_h"], case["r"]
    if 2e-13 * 4 * r * H * d_h * (sum(lens) + case.get("prefix", 0)) > 20:
        return None
    wq, wk, wv = (s[k].to(f64) for k in ("wuq", "wuk", "wuv"))

    def heads(rows, scales):
        c = rows.to(f64)
        if scales is not None:
            c = c * scales.to(f64).repeat_interleave(128, -1)
        return (c @ wk).view(-1, H, d_h), (c @ wv).view(-1, H, d_h)

    P = case.get("prefix", 0)
    kp, vp = heads(s["prefix"], s["prefix_scales"]) if P else (None, None)
    outs = torch.zeros(B, H * d_h, dtype=f64, device=DEV)
    add = case.get("add", False)
    weights = s["before"].to(f64) if add else torch.zeros(s["weights"].shape, dtype=f64, device=DEV)
    for b, n in enumerate(lens):
        if n + P == 0:
            continue
        k, v = heads(s["cache"][b, :n], None if s["scales"] is None else s["scales"][b, :n])
        q = (s["qin"][b].to(f64) @ wq).view(H, d_h)
        if case.get("rope"):
            turn = torch.exp(-math.log(10000.0) * 2.0 * torch.arange(d_h // 2, device=DEV, dtype=f64) / d_h)
            turn = torch.polar(torch.ones_like(turn), turn)                # unit complex numbers, one per pair
            pairs = lambda x: torch.complex(x[..., :d_h // 2], x[..., d_h // 2:])  # noqa: E731
            pos = torch.arange(n, device=DEV, dtype=f64)
            spin = torch.polar(torch.ones(n, d_h // 2, device=DEV, dtype=f64), pos[:, None] * turn.angle())
            dots = (pairs(k) * spin[:, None] * (pairs(q) * spin[n - 1]).conj()).real.sum(-1)
        else:
            if P:
                k, v = torch.cat([kp, k]), torch.cat([vp, v])
            dots = torch.einsum("thd,hd->th", k, q)
        p = torch.softmax(dots / math.sqrt(d_h), 0)
        outs[b] = torch.einsum("th,thd->hd", p, v).reshape(-1)
        weights[b, :n] += p[P:].sum(1)
    if case["op"] == "shared" and not case["weights"]:
        return {"out": outs}
    return {"out": outs, "weights": weights}


def _exact_evict(case, s, lens):
    import bisect
    budget, r = case["budget"], case["r"]
    rows = torch.zeros(case["B"], budget, r, dtype=torch.float64, device=DEV)
    weights = torch.zeros(case["B"], budget, dtype=torch.float64, device=DEV)
    kept = torch.full((case["B"], budget), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens):
        stay = list(range(n))
        if n > budget:
            w = s["weights"][b, :n].tolist()
            first, last = case["sink"], n - case["recent"]
            best = sorted(range(first, last), key=lambda t: (-w[t], t))[:budget - first - case["recent"]]
            stay = sorted(list(range(first)) + best + list(range(last, n)))
            assert bisect.bisect_left(stay, n) == budget
        at = torch.tensor(stay, dtype=torch.long, device=DEV)
        rows[b, :len(stay)] = s["cache"][b, at].to(torch.float64)
        weights[b, :len(stay)] = s["weights"][b, at].to(torch.float64)
        kept[b, :len(stay)] = at.int()
    return {"cache": rows, "weights": weights,
            "lengths": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device=DEV), "kept": kept}
