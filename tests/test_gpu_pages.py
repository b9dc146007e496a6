"""GPU tests of the page pool (dg_paged_reserve, dg_paged_fork, dg_paged_release) against a pool kept in Python."""
import random

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._helpers import status_ok
from tests._paged import DEV

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16).cpu(), b.contiguous().view(torch.int16).cpu())


class Pool:
    """The pool's rules, on lists."""

    def __init__(self, B, n_pages, width, page, layers=1, Hkv=1, D=128, seed=0):
        r = random.Random(seed)
        self.B, self.page, self.width, self.n_pages = B, page, width, n_pages
        self.free = list(range(n_pages))
        r.shuffle(self.free)
        self.refs, self.held, self.kv = [0] * n_pages, [[] for _ in range(B)], [0] * B
        g = torch.Generator().manual_seed(seed)
        shape = (layers, n_pages, page, Hkv, D)
        self.k, self.v = (torch.randn(shape, generator=g).bfloat16() for _ in range(2))
        self.kd, self.vd = self.k.to(DEV), self.v.to(DEV)
        self.cache = dg.PagedCache(self.kd[0], self.vd[0], torch.full((B, width), -1, dtype=torch.int32, device=DEV),
                                   i32(self.kv), i32([0] * (B + 1)))
        self.pool = dg.PagePool(self.cache, i32(self.free), i32([n_pages]), i32(self.refs))
        self.ws = dg.workspace(dg.paged_fork_workspace(1024), DEV)

    def reserve(self, n):
        self.cache.q_start.copy_(torch.tensor([0] + [sum(n[:b + 1]) for b in range(self.B)]))
        dg.paged_reserve(self.pool, self.ws)
        short = bad = False
        for b in range(self.B):
            want = min(self.width, -(-(self.kv[b] + n[b]) // self.page))
            bad |= -(-(self.kv[b] + n[b]) // self.page) > self.width
            need = want - len(self.held[b])
            if need <= 0:
                continue
            short |= need > len(self.free)
            if short:
                continue
            for _ in range(need):
                p = self.free.pop()
                self.refs[p] = 1
                self.held[b].append(p)
        return 7 if short or bad else 0

    def grow(self, kv):
        """The lengths, as an append would leave them."""
        self.kv = list(kv)
        self.cache.kv_len.copy_(torch.tensor(kv))

    def fork(self, src, dst):
        dg.paged_fork(self.pool, i32(src), i32(dst), self.ws, layers=(self.kd, self.vd))
        kv, bad, done = list(self.kv), False, set()
        heads = {d: list(self.held[d]) for d in range(self.B)}
        copies = 0
        n_free = len(self.free)
        for s, d in zip(src, dst):
            ok = 0 <= s < self.B and 0 <= d < self.B and s != d and d not in done
            done.add(d)
            ok = ok and kv[d] == 0 and not heads[d]
            if not ok:
                bad = True
                continue
            full, rest = kv[s] // self.page, kv[s] % self.page
            if rest:
                copies += 1
                if copies > n_free:
                    bad = True
                    continue
            new = heads[s][:full]
            for p in new:
                self.refs[p] += 1
            if rest:
                p = self.free.pop()
                self.refs[p] = 1
                self.k[:, p, :rest] = self.k[:, heads[s][full], :rest]
                self.v[:, p, :rest] = self.v[:, heads[s][full], :rest]
                new = new + [p]
            self.held[d], self.kv[d] = new, kv[s]
        return 7 if bad else 0

    def release(self, seqs):
        dg.paged_release(self.pool, i32(seqs), self.ws)
        bad, done, freed = False, set(), []
        for s in seqs:
            if not 0 <= s < self.B or s in done:
                bad = True
                continue
            done.add(s)
            for p in self.held[s]:
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    freed.append(p)
            self.held[s], self.kv[s] = [], 0
        self.free += sorted(freed)
        return 7 if bad else 0

    def check(self, status=0):
        assert dg.read_device_status(self.ws, clear=True) == status
        assert self.pool.n_free.item() == len(self.free)
        assert self.pool.free_pages[:len(self.free)].tolist() == self.free
        assert self.pool.refs.tolist() == self.refs
        assert self.cache.kv_len.tolist() == self.kv
        assert self.cache.page_table.tolist() == [h + [-1] * (self.width - len(h)) for h in self.held]
        assert same_bits(self.kd, self.k) and same_bits(self.vd, self.v)


@pytest.mark.parametrize("B,n_pages,width,page,layers,Hkv,D,seed", [
    (4, 30, 8, 16, 1, 1, 128, 0), (7, 60, 12, 48, 3, 2, 128, 1), (5, 40, 9, 128, 2, 8, 256, 2), (40, 300, 20, 16, 2, 1, 128, 3)])
def test_random_turns(B, n_pages, width, page, layers, Hkv, D, seed):
    r = random.Random(seed)
    p = Pool(B, n_pages, width, page, layers, Hkv, D, seed)
    for _ in range(25):
        n = [r.choice([0, 1, page // 2, page, 3 * page]) if r.random() < 0.4 else 0 for _ in range(B)]
        n = [min(x, (width * page) - k) for x, k in zip(n, p.kv)]
        p.check(p.reserve(n))
        # an append, of which some tokens are not kept
        fits = [len(p.held[b]) * page >= p.kv[b] + n[b] for b in range(B)]
        p.grow([k + (r.randrange(m + 1) if f else 0) for k, m, f in zip(p.kv, n, fits)])
        empty = [b for b in range(B) if not p.held[b] and not p.kv[b]]
        full = [b for b in range(B) if p.kv[b]]
        if empty and full:
            m = r.randrange(1, len(empty) + 1)
            dst = r.sample(empty, m)
            p.check(p.fork([r.choice(full) for _ in dst], dst))
        held = [b for b in range(B) if p.held[b]]
        if held and r.random() < 0.6:
            p.check(p.release(r.sample(held, r.randrange(1, len(held) + 1))))
    p.check(p.release(list(range(B))))
    assert sorted(p.free) == list(range(n_pages))


def test_reserve_thousands_of_sequences_and_long_prompts():
    p = Pool(2500, 6000, 3, 16)
    p.check(p.reserve([(b * 7) % 40 for b in range(2500)]))
    p = Pool(3, 3000, 2000, 16)
    p.check(p.reserve([16 * 1500 + 1, 0, 31]))
    p.grow([16 * 1500 + 1, 0, 0])
    p.check(p.reserve([0, 100, 31]))          # the third's pages are there
    p.check(p.reserve([16 * 300, 16, 31]))


def test_pool_runs_short():
    """That sequence and the later ones get none; the status tells; what was handed out stays right."""
    p = Pool(4, 6, 10, 16)
    assert p.reserve([40, 64, 16, 0]) == 7
    p.check(7)
    p.grow([40, 0, 0, 0])
    p.check(p.reserve([0, 33, 0, 0]))
    assert p.reserve([0, 0, 0, 17]) == 7
    p.check(7)
    p.grow([40, 33, 0, 0])
    assert p.fork([0, 1], [2, 3]) == 7        # no page for a copy
    p.check(7)
    p = Pool(2, 50, 3, 16)
    assert p.reserve([100, 5]) == 7           # more than the table holds
    p.check(7)
    p = Pool(3000, 200, 3, 16)                # a later turn of sequences after one that ran short
    assert p.reserve([16] * 300 + [0] * 2000 + [16] * 700) == 7
    p.check(7)


def test_forks_that_are_not_made():
    p = Pool(8, 60, 6, 16, layers=2)
    p.check(p.reserve([20, 32, 5, 0, 0, 0, 0, 0]))
    p.grow([20, 32, 5, 0, 0, 0, 0, 0])
    for src, dst in (([0], [0]), ([0], [1]), ([-1], [3]), ([0], [8]), ([8], [3]), ([0], [-1])):
        assert p.fork(src, dst) == 7
        p.check(7)
    assert p.fork([0, 1, 2, 0], [3, 3, 4, 5]) == 7      # the same dst twice: the first
    p.check(7)
    p.check(p.fork([6], [7]))                           # an empty one
    p.check(p.fork([], []))
    assert p.release([0, 0, 9, -1]) == 7
    p.check(7)
    p.check(p.release([6, 6][:1]))
    p.check(p.release([]))


def test_more_forks_than_pages_of_the_grid():
    """1024 forks of one sequence in one call, two layers, pages of several blocks' copies."""
    p = Pool(1025, 1100, 3, 1024, layers=1, Hkv=1)
    p.check(p.reserve([1030] + [0] * 1024))
    p.grow([1030] + [0] * 1024)
    p.check(p.fork([0] * 1024, list(range(1, 1025))))
    p.check(p.release(list(range(0, 1025, 2))))


def test_corrupt_counts_are_reported():
    p = Pool(2, 20, 4, 16)
    p.check(p.reserve([20, 5]))
    p.pool.refs[p.held[0][0]] = 0             # held, and yet nobody's
    dg.paged_release(p.pool, i32([0]), p.ws)
    assert dg.read_device_status(p.ws, clear=True) == 7
    assert p.pool.refs[p.held[0][0]].item() == 0 and p.pool.n_free.item() == len(p.free) + 1
    p = Pool(2, 20, 4, 16)
    p.pool.n_free.fill_(21)
    dg.paged_reserve(p.pool, p.ws)
    assert dg.read_device_status(p.ws, clear=True) == 7
    p = Pool(2, 20, 4, 16)
    p.pool.free_pages.fill_(10 ** 6)          # ids that do not exist are not handed out
    p.cache.q_start.copy_(torch.tensor([0, 16, 16]))
    dg.paged_reserve(p.pool, p.ws)
    assert dg.read_device_status(p.ws, clear=True) == 7 and (p.cache.page_table == -1).all()
    p = Pool(2, 20, 4, 16)
    p.cache.page_table.fill_(10 ** 6)
    p.cache.kv_len.fill_(20)
    dg.paged_release(p.pool, i32([1]), p.ws)
    assert dg.read_device_status(p.ws, clear=True) == 7
    status_ok(p.ws)


def test_release_of_many():
    """More sequences, or places, than one CTA takes back; the same one twice among them."""
    r = random.Random(5)
    p = Pool(1300, 4000, 30, 16)
    p.check(p.reserve([r.choice([0, 5, 40, 60]) for _ in range(1300)]))
    p.check(p.release(r.sample(range(1300), 700)))
    p.check(p.reserve([r.choice([0, 5, 20]) for _ in range(1300)]))
    seqs = r.sample(range(1300), 1200)
    assert p.release(seqs + [seqs[3], 1300]) == 7
    p.check(7)
    p = Pool(3, 40000, 20000, 16)
    p.check(p.reserve([16 * 9000, 16 * 19999, 16]))
    p.check(p.release([1]))
    p.check(p.release([2, 0]))
