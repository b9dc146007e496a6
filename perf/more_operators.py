"""What drafted trees over a paged KV cache cost: the plan of a batch of trees (who sees whom, at which positions),
the trees' attention over the pages, the draw of a token from every node's logits (temperature, top-k, top-p, min-p),
the commit of the accepted paths into the pages of every layer, and the forks of sequences that share pages.

`own = False` computes each operator in its plain form (elementary torch operations in 32 bits, weights and their sums
in 64, rounded once at the end); `own = True` makes the library's calls.  `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False
dg = None   # the library's Python package, imported when `own` is true

DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the tree of one sequence's draft: latency only
        dict(name="plan tree", op="plan", B=1, n_max=16, ragged=False, kv_max=300, window=0),
        # a large batch's trees, for sliding-window layers too
        dict(name="plan 256 trees", op="plan", B=256, n_max=64, ragged=True, kv_max=4000, window=1024),
        # one tree over a short cache, its keys already in the pages: latency only
        dict(name="attn tree", op="attn", B=1, n_max=16, ragged=False, kv_max=300, Hq=4, Hkv=1, D=128, page=16,
             window=0, fresh=False),
        # the verification step of 32 sequences of unequal length: a stream of memory
        dict(name="attn 32 trees", op="attn", B=32, n_max=32, ragged=True, kv_max=16000, Hq=16, Hkv=8, D=128, page=64,
             window=0, fresh=False),
        # trees of a few hundred nodes at the full width, their keys beside the pages, through a sliding-window layer
        dict(name="attn wide trees", op="attn", B=8, n_max=500, ragged=True, kv_max=4096, Hq=16, Hkv=8, D=256, page=32,
             window=1024, fresh=True),
        # one row of a small vocabulary: latency only
        dict(name="sample row", op="sample", R=1, V=16384, dtype="bf16", pad=0, filters="kp", masked=False),
        # a batch of rows of fp32 logits of the whole vocabulary, half of them cut by top-p and min-p, some with
        # tokens that a grammar forbids
        dict(name="sample batch", op="sample", R=64, V=262144, dtype="fp32", pad=0, filters="mixed", masked=True),
        # every node of 32 trees of 32: bf16 logits, a vocabulary of odd size in padded rows, top-k and top-p
        dict(name="sample nodes", op="sample", R=1024, V=151643, dtype="bf16", pad=293, filters="kp", masked=False),
        # one tree's accepted path, two layers: latency only
        dict(name="commit tree", op="commit", B=1, n_max=16, ragged=False, kv_max=300, Hkv=1, D=128, page=16, layers=2),
        # 64 trees' accepted paths through the pages of 16 layers
        dict(name="commit 64 trees", op="commit", B=64, n_max=32, ragged=True, kv_max=500, Hkv=8, D=128, page=64,
             layers=16),
        # one sequence continued in two ways: latency only
        dict(name="fork sequence", op="fork", B=4, n=2, kv_max=300, Hkv=1, D=128, page=16, layers=2),
        # eight prompts, sixteen continuations each: the pages are shared, the last, unfinished ones copied
        dict(name="fork 128", op="fork", B=136, n=128, kv_max=2000, Hkv=8, D=128, page=64, layers=16),
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
        op = rng.choice(["plan", "attn", "attn", "sample", "sample", "commit", "fork"])
        D, Hkv, page = rng.choice([128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 48, 64, 128])
        cost = 0
        if op == "sample":
            c = dict(op=op, R=_spread(rng, 1, 1024), V=_spread(rng, 100, 262144), dtype=rng.choice(["bf16", "fp32"]),
                     pad=rng.choice([0, 0, rng.randrange(1, 300)]), masked=rng.random() < 0.4,
                     filters=rng.choice(["none", "k", "p", "min", "kp", "mixed", "greedy"]))
        elif op == "fork":
            n = _spread(rng, 1, 128)
            c = dict(op=op, B=n + rng.randrange(1, 9), n=n, kv_max=_spread(rng, 1, 2000), Hkv=Hkv, D=D, page=page,
                     layers=rng.randrange(1, 17))
            cost = c["B"] * (c["kv_max"] + c["page"]) * c["layers"] * Hkv * D / 16
        else:
            c = dict(op=op, B=_spread(rng, 1, 256 if op == "plan" else 64), n_max=_spread(rng, 1, 600),
                     ragged=rng.random() < 0.7, kv_max=_spread(rng, 1, 16000))
            if op == "commit":
                c.update(kv_max=min(c["kv_max"], 2000), n_max=min(c["n_max"], 200), Hkv=Hkv, D=D, page=page,
                         layers=rng.randrange(1, 17))
                cost = c["B"] * (c["kv_max"] + c["n_max"] + c["page"]) * c["layers"] * Hkv * D / 16
            else:
                c["window"] = _spread(rng, 16, 5000) if rng.random() < 0.3 else 0
            if op == "attn":
                c.update(Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, D=D, page=page, fresh=rng.random() < 0.5)
                cost = c["B"] * c["n_max"] * c["Hq"] * (c["kv_max"] + c["n_max"]) / 50
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and cost <= 4e7:
            return c


def _rng(case, what):
    return random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """(nodes, cached tokens before them) of each sequence: a function of the case alone."""
    r = _rng(case, "lengths")
    B, n_max, kv_max = case["B"], case["n_max"], case["kv_max"]
    n = [max(1, int(n_max * r.uniform(0.3, 1.0))) if case["ragged"] else n_max for _ in range(B)]
    kv = [int(kv_max * r.uniform(0.1, 1.0)) for _ in range(B)]
    n[0], kv[0] = n_max, kv_max
    return n, kv


def _trees(case, n, salt=0):
    """A drafted tree for each sequence: every node's parent, the root's -1."""
    r = _rng(case, "trees %s" % salt)
    got = []
    for m in n:
        back = max(2, m // 6)
        got.append([-1] + [r.randrange(max(0, i - back), i) for i in range(1, m)])
    return got


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _paths(case, trees):
    """The nodes that are accepted of each tree, from the root on (all the way to a leaf in the first)."""
    r = _rng(case, "paths")
    got = []
    for b, parents in enumerate(trees):
        kids = {}
        for i, p in enumerate(parents):
            kids.setdefault(p, []).append(i)
        path = [0]
        while path[-1] in kids and (b == 0 or r.random() < 0.8) and len(path) < PATH_MAX:
            path.append(r.choice(kids[path[-1]]))
        got.append(path)
    return got


PATH_MAX = 16     # tokens a commit takes at most


def _forks(case):
    """Cached tokens of the sequences that are forked, and which one each fork is of."""
    r = _rng(case, "forks")
    kv = [max(1, int(case["kv_max"] * r.uniform(0.1, 1.0))) for _ in range(case["B"] - case["n"])]
    kv[0] = case["kv_max"]
    return kv, [r.randrange(len(kv)) for _ in range(case["n"])]


def work(case):
    op = case["op"]
    if op == "sample":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["R"] * (case["V"] * size + 28), "flops": 8 * case["R"] * case["V"]}
    if op == "fork":
        kv, src = _forks(case)
        row = 2 * case["layers"] * case["Hkv"] * case["D"] * 2     # a token's keys and values in bytes
        rows = sum(kv[s] % case["page"] for s in src)
        shared = sum(kv[s] // case["page"] for s in src)
        return {"bytes": 2 * rows * row + 16 * shared + 16 * case["n"], "flops": 0}
    n, kv = _lengths(case)
    T = sum(n)
    if op == "plan":
        return {"bytes": 4 * T * (2 + -(-case["n_max"] // 32)) + 8 * case["B"], "flops": 0}
    trees = _trees(case, n)
    if op == "commit":
        row = 2 * case["layers"] * case["Hkv"] * case["D"] * 2
        moved = sum(i != j for path in _paths(case, trees) for j, i in enumerate(path))
        return {"bytes": 2 * moved * row + 12 * T + 4 * case["B"] * (PATH_MAX + 4), "flops": 0}
    Hq, Hkv, D, window = case["Hq"], case["Hkv"], case["D"], case["window"]
    flops = keys = 0
    for n_b, kv_b, parents in zip(n, kv, trees):
        depth = np.array(_depths(parents), dtype=np.int64)
        seen = depth + 1 + kv_b
        if window:
            seen = np.minimum(seen, window)
        flops += 4 * D * Hq * int(seen.sum())
        keys += n_b + (min(kv_b, window - 1) if window else kv_b)
    words = -(-case["n_max"] // 32)
    return {"bytes": 2 * 2 * T * Hq * D + 2 * 2 * keys * Hkv * D + 4 * T * words, "flops": flops}


# ---------------------------------------------------------------- inputs
def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, device=DEV, dtype=torch.int32)


def _pages(gen, s, stored, page, B, spare=3):
    """A page table of B sequences of `stored` tokens whose pages are handed out in no order; the pages left over."""
    pages = [-(-t // page) for t in stored]
    n_pages, width = max(1, sum(pages)) + spare, max(1, max(pages)) + 1
    free = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = free[at:at + m]
        at += m
    s["table"] = table
    return n_pages, free[at:]


def prepare(case, seed):
    global dg
    if own:
        import block_diffusion_decoding_gb300 as dg
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case=case)
    {"plan": _prepare_plan, "attn": _prepare_attn, "sample": _prepare_sample, "commit": _prepare_commit,
     "fork": _prepare_fork}[case["op"]](s, case, gen, seed)
    return s


def _prepare_plan(s, c, gen, seed):
    n, _ = _lengths(c)
    r = random.Random(int(seed))
    kv = [r.randrange(c["kv_max"] + 1000) for _ in n]
    page = 16
    n_pages, _ = _pages(gen, s, kv, page, c["B"])
    s["parents"] = _i32([p for tree in _trees(c, n, int(seed)) for p in tree])
    s["q_start"], s["kv_len"] = _i32([0] + list(np.cumsum(n))), _i32(kv)
    s["words"] = -(-c["n_max"] // 32)
    s["mask"] = torch.zeros(sum(n), s["words"], device=DEV, dtype=torch.int32)
    s["positions"] = torch.zeros(sum(n), device=DEV, dtype=torch.int32)
    if own:
        pool = torch.zeros(n_pages, page, 1, 128, device=DEV, dtype=torch.bfloat16)
        s["cache"] = dg.PagedCache(pool, pool, s["table"], s["kv_len"], s["q_start"])
        s["ws"] = dg.workspace(dg.tree_plan_workspace(), DEV)


def _prepare_attn(s, c, gen, seed):
    n, kv = _lengths(c)
    Hq, Hkv, D, page, T = c["Hq"], c["Hkv"], c["D"], c["page"], sum(n)
    stored = kv if c["fresh"] else [a + b for a, b in zip(n, kv)]
    n_pages, _ = _pages(gen, s, stored, page, c["B"])
    s["k_cache"], s["v_cache"] = _bf16(gen, n_pages, page, Hkv, D), _bf16(gen, n_pages, page, Hkv, D)
    s["q_start"], s["kv_len"] = _i32([0] + list(np.cumsum(n))), _i32(stored)
    s["n_max"], s["kv_most"] = max(n), max(stored)
    q, k, v = _bf16(gen, T, (Hq + 2 * Hkv) * D).split([Hq * D, Hkv * D, Hkv * D], dim=1)
    s["q"] = q.reshape(T, Hq, D) * 2        # scores of spread 2: some keys matter more than others
    s["k"], s["v"] = k.view(T, Hkv, D), v.view(T, Hkv, D)
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    # the step's plan, made once for all of its layers
    words = -(-c["n_max"] // 32)
    rows, at = [], []
    for parents, kv_b in zip(_trees(c, n), kv):
        depth, bits = _depths(parents), []
        for i, p in enumerate(parents):
            own_bits, a = 1 << i, p
            while a >= 0 and not (c["window"] and depth[i] - depth[a] >= c["window"]):
                own_bits |= 1 << a
                a = parents[a]
            bits.append(own_bits)
        rows += [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in bits]
        at += [kv_b + d for d in depth]
    s["mask"] = torch.from_numpy(np.array(rows, dtype=np.uint32).view(np.int32)).to(DEV)
    s["positions"] = _i32(at)
    if own:
        s["cache"] = dg.PagedCache(s["k_cache"], s["v_cache"], s["table"], s["kv_len"], s["q_start"])
        s["ws"] = dg.workspace(dg.paged_tree_attn_workspace(T, Hq, s["cache"]), DEV)


def _prepare_sample(s, c, gen, seed):
    R, V = c["R"], c["V"]
    r = random.Random("%s %s" % (seed, c["filters"]))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    spread = torch.empty(R, 1, device=DEV).uniform_(1.0, 3.5, generator=gen)
    x = torch.randn(R, V + c["pad"], generator=gen, device=DEV) * spread
    # a model is surer of a few tokens than of all the rest
    top = torch.randint(0, V, (R, 8), generator=gen, device=DEV)
    x.scatter_add_(1, top, spread * torch.empty(R, 8, device=DEV).uniform_(2.0, 6.0, generator=gen))
    if c["masked"]:
        rows = torch.rand(R, 1, generator=gen, device=DEV) < 0.5
        x.masked_fill_(rows & (torch.rand(1, V + c["pad"], generator=gen, device=DEV) < 0.4), -math.inf)
    s["logits"] = x.to(dt)[:, :V]
    f = c["filters"]

    def rows_of(on, kind, off):
        return [kind() if on or (f == "mixed" and r.random() < 0.5) else off for _ in range(R)]

    s["temperature"] = torch.tensor([0.0 if f == "greedy" else r.uniform(0.5, 1.2) for _ in range(R)], device=DEV)
    s["top_k"] = _i32(rows_of(f in ("k", "kp"), lambda: r.choice([1, 20, 50, 64, 200, 1000]), 0))
    s["top_p"] = torch.tensor(rows_of(f in ("p", "kp"), lambda: r.uniform(0.5, 0.99), 1.0), device=DEV)
    s["min_p"] = torch.tensor(rows_of(f == "min", lambda: r.uniform(0.005, 0.2), 0.0), device=DEV)
    s["u"] = torch.rand(R, generator=gen, device=DEV)
    s["token"] = torch.empty(R, device=DEV, dtype=torch.int32)
    s["logprob"] = torch.empty(R, device=DEV)


def _prepare_commit(s, c, gen, seed):
    n, kv = _lengths(c)
    T, L, page = sum(n), c["layers"], c["page"]
    trees = _trees(c, n)
    total = [a + b for a, b in zip(n, kv)]
    n_pages, _ = _pages(gen, s, total, page, c["B"])
    s["k_cache"] = _bf16(gen, L, n_pages, page, c["Hkv"], c["D"])
    s["v_cache"] = _bf16(gen, L, n_pages, page, c["Hkv"], c["D"])
    s["q_start"], s["kv_len"] = _i32([0] + list(np.cumsum(n))), _i32(total)
    s["n_max"] = max(n)
    s["parents"] = _i32([p for tree in trees for p in tree])
    # every node's token is its own (siblings are different drafts); what is sampled at an accepted path's node is
    # the next one's token, elsewhere one that nobody drafted
    tokens = torch.randperm(262144, generator=gen, device=DEV)[:T].tolist()
    sampled = [262144 + t for t in tokens]
    at = 0
    for m, path in zip(n, _paths(c, trees)):
        for i, j in zip(path, path[1:]):
            sampled[at + i] = tokens[at + j]
        at += m
    s["tokens"], s["sampled"] = _i32(tokens), _i32(sampled)
    s["path"] = torch.zeros(c["B"], PATH_MAX, device=DEV, dtype=torch.int32)
    s["n_path"], s["next"], s["kv_out"] = (torch.zeros(c["B"], device=DEV, dtype=torch.int32) for _ in range(3))
    if own:
        s["cache"] = dg.PagedCache(s["k_cache"][0], s["v_cache"][0], s["table"], s["kv_len"], s["q_start"])
        s["ws"] = dg.workspace(dg.paged_tree_commit_workspace(), DEV)


def _prepare_fork(s, c, gen, seed):
    kv, src = _forks(c)
    B, n, L, page = c["B"], c["n"], c["layers"], c["page"]
    n_pages, free = _pages(gen, s, kv, page, B, spare=n + 5)
    s["k_cache"] = _bf16(gen, L, n_pages, page, c["Hkv"], c["D"])
    s["v_cache"] = _bf16(gen, L, n_pages, page, c["Hkv"], c["D"])
    s["kv_len"] = _i32(kv + [0] * n)
    s["src"] = _i32(src)
    s["dst"] = (torch.randperm(n, generator=gen, device=DEV) + len(kv)).to(torch.int32)
    s["refs"] = torch.ones(n_pages, device=DEV, dtype=torch.int32)
    s["refs"][free.long()] = 0
    s["free"] = torch.full((n_pages,), -1, device=DEV, dtype=torch.int32)
    s["free"][:free.numel()] = free
    s["n_free"] = _i32([free.numel()])
    s["q_start"] = torch.zeros(B + 1, device=DEV, dtype=torch.int32)
    if own:
        s["cache"] = dg.PagedCache(s["k_cache"][0], s["v_cache"][0], s["table"], s["kv_len"], s["q_start"])
        s["pool"] = dg.PagePool(s["cache"], s["free"], s["n_free"], s["refs"])
        s["ws"] = dg.workspace(dg.paged_fork_workspace(n), DEV)


# ---------------------------------------------------------------- the operators
def run(s):
    return {"plan": _run_plan, "attn": _run_attn, "sample": _run_sample, "commit": _run_commit,
            "fork": _run_fork}[s["case"]["op"]](s)


def _sequences(q_start, T):
    """Which sequence each row is of."""
    return torch.searchsorted(q_start[1:].long(), torch.arange(T, device=DEV), right=True)


def _run_plan(s):
    c = s["case"]
    if own:
        dg.tree_plan(s["parents"], s["cache"], s["mask"], s["ws"], positions=s["positions"], window=c["window"])
        return {"mask": s["mask"], "positions": s["positions"]}
    T, n_max, words = s["parents"].shape[0], c["n_max"], s["words"]
    b = _sequences(s["q_start"], T)
    i = torch.arange(T, device=DEV) - s["q_start"][b]
    # anc [B, n, n]: whether a node's ancestor at up to 2^k - 1 steps is that one; twice as many with every product
    anc = torch.zeros(c["B"], n_max, n_max, device=DEV)
    up = torch.zeros(c["B"], n_max, n_max + 1, device=DEV)
    up[b, i, s["parents"].long() % (n_max + 1)] = 1          # (a root's parent: the column that is cut off)
    up = up[..., :n_max]
    anc[b, i, i] = 1
    steps = 1
    while steps < n_max:
        anc, up, steps = anc + up @ anc, up @ up, 2 * steps
    depth = anc.sum(-1).long() - 1
    seen = anc > 0
    if c["window"]:
        seen &= depth[:, :, None] - depth[:, None, :] < c["window"]
    bits = torch.nn.functional.pad(seen, (0, 32 * words - n_max)).view(c["B"], n_max, words, 32).long()
    mask = (bits << torch.arange(32, device=DEV)).sum(-1)
    return {"mask": mask[b, i].to(torch.int32), "positions": (s["kv_len"][b] + depth[b, i]).to(torch.int32)}


def _run_attn(s):
    c = s["case"]
    if own:
        dg.paged_tree_attn(s["q"], s["cache"], s["out"], s["scale"], s["ws"], s["mask"],
                           k_new=s["k"] if c["fresh"] else None, v_new=s["v"] if c["fresh"] else None,
                           positions=s["positions"], window=c["window"])
        return s["out"]
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, n_max = Hq // Hkv, s["n_max"]
    n = s["q_start"].diff()
    base = s["kv_len"] if c["fresh"] else s["kv_len"] - n    # keys before the tree's
    i, j = torch.arange(n_max, device=DEV), torch.arange(s["kv_most"], device=DEV)
    row = (s["q_start"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    slot = s["table"][:, j // page].clamp(min=0).long() * page + j % page
    q = s["q"][row].float().view(B, n_max, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n_max * G, D)
    k, v = s["k_cache"].flatten(0, 1)[slot].float(), s["v_cache"].flatten(0, 1)[slot].float()
    bits = (s["mask"][row][..., None] >> torch.arange(32, device=DEV) & 1).flatten(2).bool()     # [B, n, 32 words]
    seen = (j < base[:, None])[:, None, :].expand(B, n_max, -1)
    if c["window"]:
        seen = seen & (j > s["positions"][row][..., None] - c["window"])
    if c["fresh"]:
        k, v = torch.cat([k, s["k"][row].float()], 1), torch.cat([v, s["v"][row].float()], 1)
        mine = (i < n[:, None])[:, None, :] & bits[..., :n_max]
        seen = torch.cat([seen, mine], 2)
    else:
        node = (j - base[:, None])[:, None, :].expand(B, n_max, -1)
        mine = (node >= 0) & (node < n[:, None, None]) & bits.gather(2, node.clamp(0, bits.shape[2] - 1))
        seen = seen | mine
    scores = q @ k.permute(0, 2, 3, 1) * s["scale"]
    hidden = ~seen[:, None, :, None, :].expand(B, 1, n_max, G, -1).reshape(B, 1, n_max * G, -1)
    scores.masked_fill_(hidden, -math.inf)
    w = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (w @ v.permute(0, 2, 1, 3)) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(B, Hkv, n_max, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_max, Hq, D)
    return o[i < n[:, None]].bfloat16()


def _run_sample(s):
    if own:
        dg.sample_logits(s["logits"], s["token"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                         top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
        return {"token": s["token"], "logprob": s["logprob"]}
    x = s["logits"].float()
    V = x.shape[1]
    rank = torch.arange(V, device=DEV)
    # tokens by logit, the lower index first among equals
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(greedy, 1.0, t))
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    w = w.masked_fill_(rank >= torch.where(greedy, 1, k), 0)
    mass = w.cumsum(1)
    p = s["top_p"].double()[:, None]
    # a token stays while the mass before it is short of its part
    out = (mass - w >= p * mass[:, -1:]) & (p < 1) | (w < s["min_p"].double()[:, None])
    out[:, 0] = False
    w = w.masked_fill_(out, 0)
    del x, mass, out
    w = torch.zeros_like(w).scatter_(1, order, w)            # back in the vocabulary's order
    del order
    mass = w.cumsum(1)
    token = (mass <= s["u"].double()[:, None] * mass[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
    got = torch.log(w.gather(1, token) / mass[:, -1:])
    return {"token": token[:, 0].to(torch.int32), "logprob": got[:, 0].float()}


def _run_commit(s):
    c = s["case"]
    if own:
        dg.paged_tree_commit(s["tokens"], s["parents"], s["sampled"], s["cache"], s["path"], s["n_path"], s["next"],
                             s["kv_out"], s["ws"], layers=(s["k_cache"], s["v_cache"]))
        return {"path": s["path"], "n_path": s["n_path"], "next": s["next"], "kv_len": s["kv_out"],
                "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    B, page, T = c["B"], c["page"], s["tokens"].shape[0]
    n, first = s["q_start"].diff(), s["q_start"][:-1].long()
    i = torch.arange(s["n_max"], device=DEV)
    row = (first[:, None] + i).clamp(max=T - 1)
    there = i < n[:, None]
    parents, tokens, sampled = s["parents"][row], s["tokens"][row], s["sampled"][row]
    cur = torch.zeros(B, 1, device=DEV, dtype=torch.long)
    path, count = torch.zeros(B, PATH_MAX, device=DEV, dtype=torch.long), torch.ones(B, 1, device=DEV, dtype=torch.long)
    on = torch.ones(B, 1, device=DEV, dtype=torch.bool)
    for at in range(1, PATH_MAX):
        fits = there & (parents == cur) & (tokens == sampled.gather(1, cur))
        on = on & fits.any(1, keepdim=True)
        cur = torch.where(on, fits.int().argmax(1, keepdim=True), cur)
        path[:, at:at + 1] = torch.where(on, cur, 0)
        count += on
    base = (s["kv_len"] - n)[:, None]
    j = torch.arange(PATH_MAX, device=DEV)
    to = torch.where(j < count, base + j, base)              # (nothing to move: the root onto itself)
    at = base + path
    table = s["table"].long()
    from_page, to_page = table.gather(1, at // page), table.gather(1, to // page)
    # (in turn, so that nothing but the moved tokens is copied)
    s["k_cache"][:, to_page, to % page] = s["k_cache"][:, from_page, at % page]
    s["v_cache"][:, to_page, to % page] = s["v_cache"][:, from_page, at % page]
    i32 = torch.int32
    return {"path": path.to(i32), "n_path": count[:, 0].to(i32), "next": sampled.gather(1, cur)[:, 0].to(i32),
            "kv_len": (base + count)[:, 0].to(i32), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_fork(s):
    """The last turn's continuations are dropped and new ones begun."""
    c = s["case"]
    got = {k: s[k] for k in ("table", "kv_len", "refs", "free", "n_free", "k_cache", "v_cache")}
    if own:
        dg.paged_release(s["pool"], s["dst"], s["ws"])
        dg.paged_fork(s["pool"], s["src"], s["dst"], s["ws"], layers=(s["k_cache"], s["v_cache"]))
        return got
    page, n_pages = c["page"], s["refs"].shape[0]
    src, dst, table = s["src"].long(), s["dst"].long(), s["table"]
    m = torch.arange(table.shape[1], device=DEV)
    # release
    gone = table[dst] >= 0
    before = s["refs"] > 0
    s["refs"].index_add_(0, table[dst].long().clamp(min=0).flatten(), -gone.flatten().int())
    freed = before & (s["refs"] == 0)
    place = torch.where(freed, s["n_free"] + freed.cumsum(0) - 1, n_pages)
    pad = torch.cat([s["free"], s["free"][:1]])
    pad[place] = torch.arange(n_pages, device=DEV, dtype=torch.int32)
    s["free"].copy_(pad[:n_pages])
    s["n_free"] += freed.sum().int()
    table[dst] = -1
    # fork
    kv = s["kv_len"][src]
    full, rest = (kv // page)[:, None], (kv % page)[:, None]
    shared = m < full
    s["refs"].index_add_(0, table[src].long().clamp(min=0).flatten(), shared.flatten().int())
    need = rest > 0
    place = s["n_free"].long() - need.cumsum(0)[:, 0]
    new = torch.where(need[:, 0], s["free"][place.clamp(min=0)], 0)
    old = table[src].gather(1, full.long())[:, 0].clamp(min=0).long()
    table[dst] = torch.where(shared, table[src], torch.where((m == full) & need, new[:, None], -1))
    s["refs"].index_add_(0, new.long(), need[:, 0].int())
    to = torch.where(need[:, 0], new.long(), old)            # (nothing to copy: a page onto itself)
    row = (torch.arange(page, device=DEV) < rest)[None, :, :, None, None]
    s["k_cache"][:, to] = torch.where(row, s["k_cache"][:, old], s["k_cache"][:, to])
    s["v_cache"][:, to] = torch.where(row, s["v_cache"][:, old], s["v_cache"][:, to])
    s["n_free"] -= need.sum().int()
    s["kv_len"][dst] = kv
    return got


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "attn":
        return _exact_attn(prepare(case, seed), c)
    if c["op"] == "sample":
        return _exact_sample(prepare(case, seed), c)
    return None      # whole numbers and copies


def _exact_attn(s, c):
    n, kv = _lengths(c)
    if work(c)["flops"] > 4e12:
        return None
    G, page = c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(sum(n), c["Hq"], c["D"], device=DEV, dtype=torch.float64)
    t = 0
    for n_b, kv_b, pages, parents in zip(n, kv, s["table"], _trees(c, n)):
        stored = kv_b if c["fresh"] else kv_b + n_b
        pages = pages[:-(-stored // page)].long()
        keys = s["k_cache"][pages].flatten(0, 1)[:stored]
        vals = s["v_cache"][pages].flatten(0, 1)[:stored]
        if c["fresh"]:
            keys, vals = torch.cat([keys, s["k"][t:t + n_b]]), torch.cat([vals, s["v"][t:t + n_b]])
        depth = _depths(parents)
        hide = np.ones((n_b, kv_b + n_b), dtype=bool)
        for i in range(n_b):
            hide[i, :kv_b] = False
            a = i
            while a >= 0:
                hide[i, kv_b + a] = False
                a = parents[a]
            if c["window"]:
                at = np.concatenate([np.arange(kv_b), kv_b + np.array(depth)])
                hide[i] |= at <= kv_b + depth[i] - c["window"]
        hide = torch.from_numpy(hide).to(DEV)
        for h in range(c["Hq"]):
            w = s["q"][t:t + n_b, h].double() @ keys[:, h // G].double().T * s["scale"]
            w = torch.softmax(w.masked_fill(hide, -math.inf), dim=-1)
            out[t:t + n_b, h] = w @ vals[:, h // G].double()
        t += n_b
    return out


def _exact_sample(s, c):
    tokens, logs = [], []
    for r in range(c["R"]):
        x = s["logits"][r].double()
        T, k, p, low, u = (float(s[name][r]) for name in ("temperature", "top_k", "top_p", "min_p", "u"))
        order = torch.argsort(x, descending=True, stable=True)
        if not T > 0:
            order = order[:1]
        if k > 0:
            order = order[:int(k)]
        w = torch.exp((x[order] - x[order[0]]) / (T if T > 0 else 1.0))
        if p < 1:
            before = torch.cat([w.new_zeros(1), w.cumsum(0)[:-1]])
            stay = before < p * w.sum()
            stay[0] = True
            order, w = order[stay], w[stay]
        stay = w >= low
        stay[0] = True
        order, at = torch.sort(order[stay])
        w = w[stay][at]
        mass = w.cumsum(0)
        i = torch.searchsorted(mass, (u * mass[-1:]), right=True).clamp(max=w.numel() - 1)
        tokens.append(order[i])
        logs.append(torch.log(w[i] / mass[-1]))
    return {"token": torch.cat(tokens).to(torch.int32), "logprob": torch.cat(logs)}
