"""What serving over a paged KV cache costs: the per-head norm with the position rotation, the append to the
pages, and the attention of a chunk of new tokens over them, at the sizes this library's workloads use.

`own = False` computes each operator in its plain form (elementary torch operations in 32 bits, the angles in
64, rounded once at the end); `own = True` makes the library's calls.  `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False
dg = None   # the library's Python package, imported when `own` is true

DEV = "cuda"
THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token of one sequence through a layer's q / k norm and rotation: latency only
        dict(name="norm_rope token", op="norm_rope", T=1, Hq=4, Hkv=1, D=128, rot=128, pairs="half", offset=1.0,
             pos=4096),
        # sixteen 256-token canvases of a small model: rotation of half of each head, adjacent pairs
        dict(name="norm_rope 16 canvases", op="norm_rope", T=4096, Hq=4, Hkv=1, D=128, rot=64, pairs="adjacent",
             offset=0.0, pos=2048),
        # a long prompt at the full width, far positions: a stream of memory
        dict(name="norm_rope prompt", op="norm_rope", T=32768, Hq=16, Hkv=8, D=256, rot=256, pairs="half",
             offset=1.0, pos=229376),
        # one new token each of 32 sequences of unequal length into their pages, the queries on the way
        dict(name="append tokens", op="append", B=32, n_max=1, ragged_q=False, kv_max=4000, Hq=16, Hkv=8, D=128,
             page=16, rot=128, pairs="half", norm=True, queries=True),
        # sixteen committed 256-token blocks at the full width
        dict(name="append blocks", op="append", B=16, n_max=256, ragged_q=False, kv_max=4096, Hq=16, Hkv=8, D=256,
             page=64, rot=256, pairs="half", norm=True, queries=True),
        # prompts of unequal lengths, keys and values only, pages of 48 tokens
        dict(name="append prompts", op="append", B=13, n_max=5003, ragged_q=True, kv_max=1000, Hq=16, Hkv=8, D=128,
             page=48, rot=64, pairs="adjacent", norm=False, queries=False),
        # one token of one sequence over a short cache: latency only
        dict(name="attn token short", op="attn", B=1, n_max=1, ragged_q=False, kv_max=300, Hq=4, Hkv=1, D=128,
             page=16, causal=True, window=0, fresh=False),
        # the decode step of 64 sequences of unequal length: a stream of memory
        dict(name="attn 64 tokens", op="attn", B=64, n_max=1, ragged_q=False, kv_max=16000, Hq=16, Hkv=8, D=128,
             page=64, causal=True, window=0, fresh=False),
        # one 256-token canvas over a 4096-token cache at the full width, its own keys beside the pages, no mask
        dict(name="attn canvas", op="attn", B=1, n_max=256, ragged_q=False, kv_max=4096, Hq=16, Hkv=8, D=256,
             page=64, causal=False, window=0, fresh=True),
        # sixteen canvases over 2048-token caches of a small model
        dict(name="attn 16 canvases", op="attn", B=16, n_max=256, ragged_q=False, kv_max=2048, Hq=4, Hkv=1, D=128,
             page=128, causal=False, window=0, fresh=True),
        # committed blocks through a sliding-window layer, their keys already in the pages
        dict(name="attn window blocks", op="attn", B=5, n_max=256, ragged_q=True, kv_max=4096, Hq=16, Hkv=8, D=256,
             page=32, causal=True, window=1024, fresh=False),
        # prompt chunks of unequal lengths after long caches: arithmetic
        dict(name="attn prompt chunks", op="attn", B=4, n_max=2000, ragged_q=True, kv_max=16384, Hq=16, Hkv=8, D=128,
             page=64, causal=True, window=0, fresh=False),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(["norm_rope", "append", "attn", "attn"])
        D = rng.choice([128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        rot = rng.choice([D, D // 2, D // 4])
        pairs = rng.choice(["half", "adjacent"])
        page = rng.choice([16, 32, 48, 64, 128, 256])
        if op == "norm_rope":
            c = dict(op=op, T=_spread(rng, 1, 40000), Hq=Hq, Hkv=Hkv, D=D, rot=rot, pairs=pairs,
                     offset=rng.choice([0.0, 1.0]), pos=_spread(rng, 1, 250000))
        else:
            single = rng.random() < 0.35
            c = dict(op=op, B=_spread(rng, 1, 80), n_max=1 if single else _spread(rng, 2, 3000), ragged_q=not single,
                     kv_max=_spread(rng, 1, 20000), Hq=Hq, Hkv=Hkv, D=D, page=page)
            if op == "append":
                c.update(rot=rot, pairs=pairs, norm=rng.random() < 0.5, queries=rng.random() < 0.5)
            else:
                causal = rng.random() < 0.6
                c.update(causal=causal, window=_spread(rng, 16, 5000) if causal and rng.random() < 0.3 else 0,
                         fresh=rng.random() < 0.5)
        w = work(c)
        plain = 0 if op != "attn" else c["B"] * c["n_max"] * c["Hq"] * (c["kv_max"] + c["n_max"])
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and plain <= 6e9:
            return c


def _lengths(case):
    """(new tokens, cached tokens before them) of each sequence: a function of the case alone."""
    r = random.Random("%d %d %d" % (case["B"], case["n_max"], case["kv_max"]))
    B, n_max, kv_max = case["B"], case["n_max"], case["kv_max"]
    n = [n_max if not case["ragged_q"] else max(1, int(n_max * r.uniform(0.3, 1.0))) for _ in range(B)]
    if B == 1 or case["op"] == "attn" and not case["ragged_q"] and n_max > 1:
        kv = [kv_max] * B       # canvases in step
    else:
        kv = [int(kv_max * r.uniform(0.1, 1.0)) for _ in range(B)]
    n[0], kv[0] = n_max, kv_max
    return n, kv


def _pairs(n, total, causal, window):
    """Visible (query, key) pairs of n queries at the last n of `total` keys, and the first key any of them sees."""
    if not causal:
        return n * total, 0
    p = np.arange(total - n, total, dtype=np.int64)
    lo = np.maximum(0, p - window + 1) if window else np.zeros_like(p)
    return int(np.maximum(0, p + 1 - lo).sum()), int(lo[0])


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm_rope":
        el = case["T"] * (Hq + Hkv) * D
        return {"bytes": 4 * el + 4 * case["T"], "flops": 9 * el}
    n, kv = _lengths(case)
    T = sum(n)
    if case["op"] == "append":
        rows = 2 * Hkv + (Hq if case["queries"] else 0)
        return {"bytes": 4 * T * rows * D + 8 * T, "flops": 9 * T * (rows - Hkv) * D}
    flops = keys = 0
    for n_b, kv_b in zip(n, kv):
        pairs, first = _pairs(n_b, kv_b + n_b, case["causal"], case["window"])
        flops += 4 * D * Hq * pairs
        keys += kv_b + n_b - first
    return {"bytes": 2 * 2 * T * Hq * D + 2 * 2 * keys * Hkv * D, "flops": flops}


# ---------------------------------------------------------------- inputs
def _inv_freq(rot):
    """Radians a position, in 64 bits."""
    return THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    global dg
    if own:
        import block_diffusion_decoding_gb300 as dg
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s = dict(case=case)
    if case["op"] == "norm_rope":
        T = case["T"]
        # the rows of a joint projection: q, k and v side by side
        qkv = _bf16(gen, T, (Hq + 2 * Hkv) * D)
        s["positions"] = (case["pos"] + torch.arange(T, device=DEV)).to(torch.int32)
    else:
        n, kv = _lengths(case)
        B, T, page = case["B"], sum(n), case["page"]
        total = [a + b for a, b in zip(n, kv)]
        stored = kv if case["op"] == "attn" and case["fresh"] else total
        pages = [-(-t // page) for t in stored]
        n_pages, width = max(1, sum(pages)) + 3, max(1, max(pages))
        # pages handed out in no order; table entries past a sequence's last page are left over
        free = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
        at = 0
        for b, m in enumerate(pages):
            table[b, :m] = free[at:at + m]
            at += m
        s["k_cache"] = _bf16(gen, n_pages, page, Hkv, D)
        s["v_cache"] = _bf16(gen, n_pages, page, Hkv, D)
        s["table"] = table
        s["q_start"] = torch.tensor([0] + list(np.cumsum(n)), device=DEV, dtype=torch.int32)
        cached = kv if case["op"] == "append" else stored
        s["kv_len"] = torch.tensor(cached, device=DEV, dtype=torch.int32)
        s["n_max"], s["kv_most"] = max(n), max(cached)
        qkv = _bf16(gen, T, (Hq + 2 * Hkv) * D)
    T = qkv.shape[0]
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    s["q"], s["k"], s["v"] = q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)
    if case["op"] == "attn":
        s["q"] = s["q"] * 2         # scores of spread 2: some keys matter more than others
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    else:
        if case["op"] == "norm_rope" or case["norm"]:
            s["q_weight"] = (0.1 * torch.randn(D, generator=gen, device=DEV) + 1 - case.get("offset", 0.0)).bfloat16()
            s["k_weight"] = (0.1 * torch.randn(D, generator=gen, device=DEV) + 1 - case.get("offset", 0.0)).bfloat16()
        else:
            s["q_weight"] = s["k_weight"] = None
        s["inv_freq"] = _inv_freq(case["rot"]).to(DEV)
        s["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
        s["k_out"] = torch.empty(T, Hkv, D, device=DEV, dtype=torch.bfloat16)
        s["kv_len_out"] = torch.zeros(case.get("B", 1), device=DEV, dtype=torch.int32)
    if own:
        if case["op"] != "norm_rope":
            s["cache"] = dg.PagedCache(s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["q_start"])
            s["ws"] = dg.workspace(dg.paged_attn_workspace(T, Hq, s["cache"]) if case["op"] == "attn"
                                   else dg.paged_append_workspace(), DEV)
        if case["op"] != "attn":
            s["heads"] = dg.head_params(Hq, Hkv, D, rope_steps=dg.rope_steps(_inv_freq(case["rot"]), DEV),
                                        interleaved=case["pairs"] == "adjacent", q_weight=s["q_weight"],
                                        k_weight=s["k_weight"], eps=EPS, weight_offset=case.get("offset", 0.0))
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    return {"norm_rope": _run_norm_rope, "append": _run_append, "attn": _run_attn}[s["case"]["op"]](s)


def _norm_rope(x, weight, offset, angles, rot, pairs):
    """RMS norm over each head and the rotation of its first `rot` values, in 32 bits; angles [T, rot / 2] in 64."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (offset + weight.float())
    cos, sin = angles.cos().float()[:, None], angles.sin().float()[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    if pairs == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1).bfloat16()


def _run_norm_rope(s):
    c = s["case"]
    if own:
        dg.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["heads"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angles = s["positions"].double()[:, None] * s["inv_freq"]
    return {"q": _norm_rope(s["q"], s["q_weight"], c["offset"], angles, c["rot"], c["pairs"]),
            "k": _norm_rope(s["k"], s["k_weight"], c["offset"], angles, c["rot"], c["pairs"])}


def _places(s, T):
    """(sequence, index within its cache) of each new token of an append."""
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    return b, s["kv_len"][b] + t - s["q_start"][b]


def _run_append(s):
    c = s["case"]
    if own:
        q = s["q"] if c["queries"] else None
        dg.paged_append(s["k"], s["v"], s["cache"], s["heads"], s["ws"], q=q, q_out=s["q_out"] if c["queries"] else None,
                        kv_len_out=s["kv_len_out"])
        got = {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_len": s["kv_len_out"]}
        return {**got, "q": s["q_out"]} if c["queries"] else got
    b, at = _places(s, s["k"].shape[0])
    page, where = s["table"][b, at // c["page"]].long(), (at % c["page"]).long()
    angles = at.double()[:, None] * s["inv_freq"]
    s["k_cache"][page, where] = _norm_rope(s["k"], s["k_weight"], 0.0, angles, c["rot"], c["pairs"])
    s["v_cache"][page, where] = s["v"]
    got = {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_len": s["kv_len"] + s["q_start"].diff()}
    if c["queries"]:
        got["q"] = _norm_rope(s["q"], s["q_weight"], 0.0, angles, c["rot"], c["pairs"])
    return got


def _run_attn(s):
    c = s["case"]
    if own:
        dg.paged_attn(s["q"], s["cache"], s["out"], s["scale"], s["ws"], k_new=s["k"] if c["fresh"] else None,
                      v_new=s["v"] if c["fresh"] else None, causal=c["causal"], window=c["window"])
        return s["out"]
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, n_max = Hq // Hkv, s["n_max"]
    n, kv = s["q_start"].diff(), s["kv_len"]
    # the chunks and the cached keys, each padded to the longest
    i, j = torch.arange(n_max, device=DEV), torch.arange(s["kv_most"], device=DEV)
    row = (s["q_start"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    slot = (s["table"][:, j // page].clamp(min=0).long() * page + j % page)
    q = s["q"][row].float().view(B, n_max, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n_max * G, D)
    k, v = s["k_cache"].flatten(0, 1)[slot].float(), s["v_cache"].flatten(0, 1)[slot].float()
    seen = (j < kv[:, None])[:, None, :]
    place = kv[:, None] + i if c["fresh"] else kv[:, None] - n[:, None] + i
    if c["causal"]:
        seen = seen & (j <= place[..., None])
        if c["window"]:
            seen = seen & (j > place[..., None] - c["window"])
    seen = seen.expand(B, n_max, -1)
    if c["fresh"]:
        k, v = torch.cat([k, s["k"][row].float()], 1), torch.cat([v, s["v"][row].float()], 1)
        mine = (i < n[:, None])[:, None, :].expand(B, n_max, n_max)
        if c["causal"]:
            mine = mine & (i <= i[:, None])
            if c["window"]:
                mine = mine & (i > i[:, None] - c["window"])
        seen = torch.cat([seen, mine], 2)
    scores = q @ k.permute(0, 2, 3, 1) * s["scale"]
    hidden = ~seen[:, None, :, None, :].expand(B, 1, n_max, G, -1).reshape(B, 1, n_max * G, -1)
    scores.masked_fill_(hidden, -math.inf)
    w = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (w @ v.permute(0, 2, 1, 3)) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(B, Hkv, n_max, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_max, Hq, D)
    return o[i < n[:, None]].bfloat16()


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attn":
        return _exact_attn(s, c)
    rot, half = c["rot"], c["rot"] // 2

    def turn(x, weight, offset, at):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS) * (weight.double() + offset)
        y = x.clone()
        for m in range(half):
            a, b = (m, m + half) if c["pairs"] == "half" else (2 * m, 2 * m + 1)
            phi = (at.double() * THETA ** (-2.0 * m / rot))[:, None]
            y[..., a] = x[..., a] * torch.cos(phi) - x[..., b] * torch.sin(phi)
            y[..., b] = x[..., a] * torch.sin(phi) + x[..., b] * torch.cos(phi)
        return y

    if c["op"] == "norm_rope":
        return {"q": turn(s["q"], s["q_weight"], c["offset"], s["positions"]),
                "k": turn(s["k"], s["k_weight"], c["offset"], s["positions"])}
    n, kv = _lengths(c)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at = torch.cat([torch.arange(kv_b, kv_b + n_b, device=DEV) for n_b, kv_b in zip(n, kv)])
    k = turn(s["k"], s["k_weight"], 0.0, at)
    t = 0
    for b in range(c["B"]):
        mine = at[t:t + n[b]]
        pages = s["table"][b].long()[mine // c["page"]]
        kc[pages, mine % c["page"]] = k[t:t + n[b]]
        vc[pages, mine % c["page"]] = s["v"][t:t + n[b]].double()
        t += n[b]
    got = {"k_cache": kc, "v_cache": vc, "kv_len": None}
    if c["queries"]:
        got["q"] = turn(s["q"], s["q_weight"], 0.0, at)
    return got


def _exact_attn(s, c):
    n, kv = _lengths(c)
    if work(c)["flops"] > 4e12:
        return None
    G, page = c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(sum(n), c["Hq"], c["D"], device=DEV, dtype=torch.float64)
    t = 0
    for n_b, kv_b, pages in zip(n, kv, s["table"]):
        stored = kv_b if c["fresh"] else kv_b + n_b
        pages = pages[:-(-stored // page)].long()
        keys = s["k_cache"][pages].flatten(0, 1)[:stored]
        vals = s["v_cache"][pages].flatten(0, 1)[:stored]
        if c["fresh"]:
            keys, vals = torch.cat([keys, s["k"][t:t + n_b]]), torch.cat([vals, s["v"][t:t + n_b]])
        for at in range(0, n_b, 512):
            m = min(512, n_b - at)
            p = kv_b + at + torch.arange(m, device=DEV)[:, None]
            j = torch.arange(kv_b + n_b, device=DEV)[None]
            hide = torch.zeros(m, kv_b + n_b, device=DEV, dtype=torch.bool)
            if c["causal"]:
                hide = j > p
                if c["window"]:
                    hide = hide | (j <= p - c["window"])
            for h in range(c["Hq"]):
                w = s["q"][t + at:t + at + m, h].double() @ keys[:, h // G].double().T * s["scale"]
                w = torch.softmax(w.masked_fill(hide, -math.inf), dim=-1)
                out[t + at:t + at + m, h] = w @ vals[:, h // G].double()
        t += n_b
    return out
