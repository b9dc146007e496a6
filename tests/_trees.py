"""Drafted trees for the tests, and their operators' definitions on the CPU, plain loops over nodes (no library
code)."""
import random

import torch

NAN = float("nan")


def tree(n, seed, back=None, chain=False):
    """Parents of n nodes; a chain, or each one's parent among the `back` nodes before it."""
    r = random.Random(seed)
    back = max(2, n // 6) if back is None else back
    return [-1] + [i - 1 if chain else r.randrange(max(0, i - back), i) for i in range(1, n)] if n else []


def plan(trees, base, words, window=0):
    """(mask rows as lists of words, positions) of the trees, as dg_tree_plan defines them."""
    mask, positions = [], []
    for parents, at in zip(trees, base):
        depth = []
        for i, p in enumerate(parents):
            depth.append(0 if p < 0 else depth[p] + 1)
            bits, a = 0, i
            while a >= 0:
                if not window or depth[i] - depth[a] < window:
                    bits |= 1 << a
                a = parents[a]
            mask.append([bits >> 32 * w & 0xFFFFFFFF for w in range(words)])
            positions.append(at + depth[i])
    return mask, positions


def as_int32(rows):
    """Words of 32 bits as an int32 tensor."""
    t = torch.tensor(rows, dtype=torch.int64)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32)


def attention(batch, mask, positions, window, fresh, stored):
    """(out, bound) as tests/_paged.attention gives them, for trees whose rows see what their mask says."""
    out = torch.full((batch.T, batch.Hq, batch.D), NAN, dtype=torch.float64)
    bound = torch.zeros_like(out)
    G = batch.Hq // batch.Hkv
    for b, n in enumerate(batch.n):
        t0 = int(batch.q_start[b])
        keys, vals = batch.keys(b, stored[b])
        if fresh:
            keys = torch.cat([keys, batch.kn[t0:t0 + n]])
            vals = torch.cat([vals, batch.vn[t0:t0 + n]])
        base = keys.shape[0] - n
        for i in range(n):
            words = mask[t0 + i]
            seen = [j for j in range(max(0, base)) if not window or j > positions[t0 + i] - window]
            seen += [base + j for j in range(n)
                     if base + j >= 0 and j <= i and j < 32 * len(words) and words[j // 32] >> j % 32 & 1]
            for h in range(batch.Hq):
                if not seen:
                    out[t0 + i, h] = 0
                    continue
                K, V = keys[seen, h // G].double(), vals[seen, h // G].double()
                w = torch.softmax(K @ batch.q[t0 + i, h].double() * batch.scale, 0)
                out[t0 + i, h] = w @ V
                bound[t0 + i, h] = 2 ** -8 * out[t0 + i, h].abs() + (2 ** -8 + 2 ** -12) * (w @ V.abs())
    return out, bound


def walk(parents, tokens, sampled, path_max):
    """The accepted path of one tree, and what was sampled at its end."""
    if not parents:
        return [], -1
    path = [0]
    while len(path) < path_max:
        at = path[-1]
        fits = [i for i in range(at + 1, len(parents)) if parents[i] == at and tokens[i] == sampled[at]]
        if not fits:
            break
        path.append(fits[0])
    return path, sampled[path[-1]]
