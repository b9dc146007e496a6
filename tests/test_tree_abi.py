"""The entry points of drafted trees, draws from logits and the page pool without a GPU: what they refuse before
anything is launched, the workspace queries, and the Python binding's checks of its tensors."""
import ctypes
import math

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from block_diffusion_decoding_gb300 import build as dgbuild
from tests.test_paged_abi import ALIGNMENT, BAD_CACHES, GOOD, INVALID, UNSUPPORTED, WORKSPACE, cache


@pytest.fixture(scope="module")
def lib():
    dgbuild.build()
    return dg.lib()


def plan(lib, c=None, parents=GOOD, T=5, window=0, appended=0, mask=GOOD, words=1, pos=None, ws=GOOD, n=256):
    c = cache() if c is None else c
    return lib.dg_tree_plan(parents, T, window, appended, mask, words, pos, ctypes.byref(c), ws, n, None)


def attn(lib, c=None, q=GOOD, qs=0, kn=None, ks=0, vn=None, vs=0, out=GOOD, os=0, T=5, Hq=4, scale=0.1, window=0,
         mask=GOOD, words=1, pos=None, ws=GOOD, n=1 << 30):
    c = cache() if c is None else c
    return lib.dg_paged_tree_attn(q, qs, kn, ks, vn, vs, out, os, T, Hq, scale, window, mask, words, pos, ctypes.byref(c),
                                  ws, n, None)


def commit(lib, c=None, tokens=GOOD, parents=GOOD, sampled=GOOD, T=5, layers=1, apart=0, path=GOOD, path_max=4,
           n_path=GOOD, next=GOOD, lens=GOOD, ws=GOOD, n=256):
    c = cache(kv_len=GOOD + 4096) if c is None else c
    return lib.dg_paged_tree_commit(tokens, parents, sampled, T, layers, apart, ctypes.byref(c), path, path_max, n_path,
                                    next, lens, ws, n, None)


def sample(lib, logits=GOOD, type=0, stride=0, R=3, V=100, u=GOOD, token=GOOD):
    return lib.dg_sample_logits(logits, type, stride, R, V, None, None, None, None, u, token, None, None)


def pool(**kw):
    d = dict(free_pages=GOOD, n_free=GOOD, refs=GOOD)
    d.update(kw)
    return dg.PagePoolArgs(*[d[n] for n, _ in dg.PagePoolArgs._fields_])


def reserve(lib, p=None, c=None, ws=GOOD, n=256):
    p, c = pool() if p is None else p, cache() if c is None else c
    return lib.dg_paged_reserve(ctypes.byref(p), ctypes.byref(c), ws, n, None)


def fork(lib, p=None, c=None, layers=1, apart=0, src=GOOD, dst=GOOD, k=3, ws=GOOD, n=1 << 20):
    p, c = pool() if p is None else p, cache() if c is None else c
    return lib.dg_paged_fork(ctypes.byref(p), ctypes.byref(c), layers, apart, src, dst, k, ws, n, None)


def release(lib, p=None, c=None, seqs=GOOD, k=3, ws=GOOD, n=256):
    p, c = pool() if p is None else p, cache() if c is None else c
    return lib.dg_paged_release(ctypes.byref(p), ctypes.byref(c), seqs, k, ws, n, None)


PAGE = 16 * 2 * 128      # the cache's: elements of a page
BAD_LAYERS = [(dict(layers=0), INVALID), (dict(layers=-1), INVALID), (dict(layers=2), INVALID),
              (dict(layers=2, apart=-8), INVALID), (dict(layers=2, apart=PAGE * 10 + 4), ALIGNMENT),
              (dict(layers=2, apart=PAGE * 10 - 8), INVALID), (dict(layers=3, apart=PAGE), INVALID),
              (dict(layers=1 << 17, apart=PAGE * 10), UNSUPPORTED), (dict(layers=2, apart=1 << 47), UNSUPPORTED)]


def test_plan_refuses(lib):
    for kw, code in BAD_CACHES:
        assert plan(lib, c=cache(**kw)) == code, kw
    for kw, code in ((dict(parents=None), INVALID), (dict(mask=None), INVALID), (dict(T=-1), INVALID),
                     (dict(window=-1), INVALID), (dict(appended=2), INVALID), (dict(words=0), INVALID),
                     (dict(words=129), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(ws=None), WORKSPACE),
                     (dict(n=255), WORKSPACE), (dict(ws=GOOD + 8), ALIGNMENT)):
        assert plan(lib, **kw) == code, kw
    assert plan(lib, T=0, parents=None, mask=None) == 0
    assert lib.dg_tree_plan_workspace() == 256


def test_attention_refuses(lib):
    for kw, code in BAD_CACHES:
        assert attn(lib, c=cache(**kw)) == code, kw
    for kw, code in ((dict(q=None), INVALID), (dict(out=None), INVALID), (dict(kn=GOOD), INVALID),
                     (dict(vn=GOOD), INVALID), (dict(T=-1), INVALID), (dict(Hq=3), UNSUPPORTED),
                     (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(window=-1), INVALID),
                     (dict(window=4), INVALID), (dict(mask=None), INVALID), (dict(words=0), INVALID),
                     (dict(words=129), UNSUPPORTED), (dict(qs=516), ALIGNMENT), (dict(os=8), INVALID),
                     (dict(q=GOOD + 2), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(n=1000), WORKSPACE),
                     (dict(ws=GOOD + 8), ALIGNMENT), (dict(T=1 << 29), UNSUPPORTED)):
        assert attn(lib, **kw) == code, kw
    assert attn(lib, T=0, q=None, out=None, mask=None) == 0
    c = cache()
    assert (lib.dg_paged_tree_attn_workspace(5, 4, ctypes.byref(c)) == lib.dg_paged_attn_workspace(5, 4, ctypes.byref(c))
            > 256)


def test_commit_refuses(lib):
    for kw, code in BAD_CACHES:
        assert commit(lib, c=cache(**kw)) == code, kw
    for kw, code in BAD_LAYERS:
        assert commit(lib, **kw) == code, kw
    for kw, code in ((dict(tokens=None), INVALID), (dict(parents=None), INVALID), (dict(sampled=None), INVALID),
                     (dict(path=None), INVALID), (dict(n_path=None), INVALID), (dict(next=None), INVALID),
                     (dict(lens=None), INVALID), (dict(T=-1), INVALID), (dict(path_max=0), INVALID),
                     (dict(path_max=1 << 21), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
                     (dict(lens=GOOD + 4096 + 4), INVALID), (dict(lens=GOOD + 4096), INVALID), (dict(ws=None), WORKSPACE), (dict(n=255), WORKSPACE),
                     (dict(ws=GOOD + 8), ALIGNMENT)):
        assert commit(lib, **kw) == code, kw


def test_sample_refuses(lib):
    for kw, code in ((dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(token=None), INVALID),
                     (dict(type=2), INVALID), (dict(R=-1), INVALID), (dict(V=0), INVALID), (dict(stride=99), INVALID),
                     (dict(stride=-1), INVALID), (dict(V=393217), UNSUPPORTED), (dict(R=1 << 27), UNSUPPORTED),
                     (dict(logits=GOOD + 2), ALIGNMENT)):
        assert sample(lib, **kw) == code, kw
    assert sample(lib, R=0, logits=None, u=None, token=None) == 0


def test_pool_refuses(lib):
    for call in (reserve, fork, release):
        for kw, code in BAD_CACHES:
            assert call(lib, c=cache(**kw)) == code, kw
        for kw in (dict(free_pages=None), dict(n_free=None), dict(refs=None)):
            assert call(lib, p=pool(**kw)) == INVALID, kw
        for kw, code in ((dict(ws=None), WORKSPACE), (dict(n=255), WORKSPACE), (dict(ws=GOOD + 8), ALIGNMENT)):
            assert call(lib, **kw) == code, kw
    assert lib.dg_paged_reserve(None, ctypes.byref(cache()), GOOD, 256, None) == INVALID
    for kw, code in BAD_LAYERS + [(dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(k=-1), INVALID),
                                  (dict(k=1025), UNSUPPORTED)]:
        assert fork(lib, **kw) == code, kw
    assert fork(lib, k=3, n=lib.dg_paged_fork_workspace(3) - 1) == WORKSPACE
    assert lib.dg_paged_fork_workspace(-1) == lib.dg_paged_fork_workspace(1025) == 0
    for kw, code in ((dict(seqs=None), INVALID), (dict(k=-1), INVALID), (dict(k=1 << 21), UNSUPPORTED)):
        assert release(lib, **kw) == code, kw
    assert fork(lib, k=0, src=None, dst=None) == 0 and release(lib, k=0, seqs=None) == 0
    assert lib.dg_paged_reserve_workspace() == lib.dg_paged_release_workspace() == 256


def test_binding_checks_its_tensors(lib):
    class Cache:
        pass

    c = Cache()
    c.k = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    c.v = torch.zeros_like(c.k)
    both = torch.zeros(2, 4, 3, 16, 2, 128, dtype=torch.bfloat16)
    c.k, c.v = both[0, 0], both[1, 0]
    c.first = tuple((t.data_ptr(), t.shape, t.stride()) for t in (c.k, c.v))
    assert dg._layers(None, c, "x") == (1, 0)
    assert dg._layers((both[0], both[1]), c, "x") == (4, c.k.numel())
    assert dg._layers((both[0, :1], both[1, :1]), c, "x") == (1, 0)
    for bad in ((both[0], both[1, :2]), (both[0, 1:], both[1, 1:]), (both[0].float(), both[1]),
                (both[0, :, :2], both[1, :, :2]), (both[0, 0], both[1, 0]), (both[0][:0], both[1][:0])):
        with pytest.raises(dg.DgError):
            dg._layers(bad, c, "x")
    with pytest.raises(dg.DgError):
        dg._mask(torch.zeros(3, 2), 3, "x", -1)
    with pytest.raises(dg.DgError):
        dg._mask(torch.zeros(3, 4, dtype=torch.int32)[:, :2], 3, "x", -1)
    with pytest.raises(dg.DgError):
        dg._mask(torch.zeros(4, 2, dtype=torch.int32), 3, "x", -1)
    with pytest.raises(dg.DgError):
        dg._floats(torch.zeros(3, dtype=torch.float64), 3, "x", -1)
    x = torch.zeros(2, 8)
    for bad in (x, x.half(), x[0], x.T):
        with pytest.raises(dg.DgError):
            dg.sample_logits(bad, torch.zeros(2, dtype=torch.int32), torch.zeros(2))
