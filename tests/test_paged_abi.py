"""The paged-cache entry points without a GPU: what they refuse before anything is launched, the workspace
queries, the struct layouts, the frequency conversion, and the Python binding's checks of its tensors."""
import ctypes
import math

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from block_diffusion_decoding_gb300 import build as dgbuild

GOOD = 1 << 20          # an aligned address that is never read: every call below is refused or empty
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    dgbuild.build()
    return dg.lib()


def cache(**kw):
    d = dict(k=GOOD, v=GOOD, page_table=GOOD, kv_len=GOOD, q_start=GOOD, page_stride=0, n_pages=10, page_size=16,
             max_pages=4, B=2, Hkv=2, D=128)
    d.update(kw)
    return dg.PagedCacheArgs(*[d[n] for n, _ in dg.PagedCacheArgs._fields_])


def heads(**kw):
    d = dict(Hq=4, Hkv=2, D=128, rot=128, interleaved=0, eps=1e-6, weight_offset=0.0, rope_steps=GOOD,
             q_weight=GOOD, k_weight=GOOD)
    d.update(kw)
    return dg.HeadParams(*[d[n] for n, _ in dg.HeadParams._fields_])


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_table=None), INVALID),
              (dict(kv_len=None), INVALID), (dict(q_start=None), INVALID), (dict(n_pages=0), INVALID),
              (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(B=0), INVALID),
              (dict(D=64), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(page_size=4096), UNSUPPORTED),
              (dict(max_pages=1 << 27), UNSUPPORTED), (dict(page_stride=16 * 2 * 128 - 8), INVALID),
              (dict(page_stride=16 * 2 * 128 + 4), ALIGNMENT), (dict(page_stride=-8), INVALID),
              (dict(page_stride=1 << 38), UNSUPPORTED), (dict(k=GOOD + 8), ALIGNMENT), (dict(v=GOOD + 2), ALIGNMENT)]
BAD_HEADS = [(dict(Hq=0), INVALID), (dict(D=0), INVALID), (dict(rot=-16), INVALID), (dict(interleaved=2), INVALID),
             (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(weight_offset=math.inf), INVALID),
             (dict(rope_steps=None), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
             (dict(q_weight=GOOD + 2), ALIGNMENT), (dict(k_weight=GOOD + 8), ALIGNMENT)]


def test_struct_layouts(lib):
    assert ctypes.sizeof(dg.HeadParams) == 56 and dg.HeadParams.rope_steps.offset == 32
    assert ctypes.sizeof(dg.PagedCacheArgs) == 72 and dg.PagedCacheArgs.n_pages.offset == 48


def attn(lib, c=None, q=GOOD, qs=0, kn=None, ks=0, vn=None, vs=0, out=GOOD, os=0, T=5, Hq=4, scale=0.1, causal=1,
         window=0, ws=GOOD, n=1 << 30):
    c = cache() if c is None else c
    return lib.dg_paged_attn(q, qs, kn, ks, vn, vs, out, os, T, Hq, scale, causal, window, ctypes.byref(c), ws, n, None)


def append(lib, c=None, p=None, k=GOOD, ks=0, v=GOOD, vs=0, q=None, qs=0, qo=None, qos=0, T=5, lens=None, ws=GOOD,
           n=256):
    c, p = cache() if c is None else c, heads() if p is None else p
    return lib.dg_paged_append(k, ks, v, vs, q, qs, qo, qos, None, T, ctypes.byref(p), ctypes.byref(c), lens, ws, n,
                               None)


def rope(lib, p=None, q=GOOD, qs=0, k=GOOD, ks=0, qo=GOOD, qos=0, ko=GOOD, kos=0, pos=GOOD, T=5):
    p = heads() if p is None else p
    return lib.dg_qk_norm_rope(q, qs, k, ks, qo, qos, ko, kos, pos, T, ctypes.byref(p), None)


def test_attention_refuses(lib):
    for kw, code in BAD_CACHES:
        assert attn(lib, c=cache(**kw)) == code, kw
    assert lib.dg_paged_attn(GOOD, 0, None, 0, None, 0, GOOD, 0, 5, 4, 0.1, 1, 0, None, GOOD, 1 << 30, None) == INVALID
    for kw, code in ((dict(q=None), INVALID), (dict(out=None), INVALID), (dict(kn=GOOD), INVALID),
                     (dict(vn=GOOD), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=3), UNSUPPORTED),
                     (dict(Hq=2 * 129), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
                     (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
                     (dict(causal=0, window=4), INVALID), (dict(qs=4 * 128 - 8), INVALID), (dict(qs=516), ALIGNMENT),
                     (dict(os=8), INVALID), (dict(kn=GOOD, vn=GOOD, ks=264 - 4), ALIGNMENT),
                     (dict(kn=GOOD, vn=GOOD, vs=128), INVALID), (dict(q=GOOD + 2), ALIGNMENT),
                     (dict(out=GOOD + 8), ALIGNMENT), (dict(kn=GOOD + 8, vn=GOOD), ALIGNMENT), (dict(ws=None), WORKSPACE),
                     (dict(n=1000), WORKSPACE), (dict(ws=GOOD + 8), ALIGNMENT), (dict(T=1 << 29), UNSUPPORTED)):
        assert attn(lib, **kw) == code, kw
    assert attn(lib, T=0, q=None, out=None) == 0
    c = cache()
    need = lib.dg_paged_attn_workspace(5, 4, ctypes.byref(c))
    assert attn(lib, n=need - 1) == WORKSPACE and need > 256
    assert lib.dg_paged_attn_workspace(500, 4, ctypes.byref(c)) > need
    for T, Hq, c in ((-1, 4, cache()), (5, 3, cache()), (5, 0, cache()), (5, 4, cache(D=64)), (5, 4, cache(Hkv=0))):
        assert lib.dg_paged_attn_workspace(T, Hq, ctypes.byref(c)) == 0


def test_append_refuses(lib):
    for kw, code in BAD_CACHES:
        assert append(lib, c=cache(**kw)) in (code, INVALID), kw
    for kw, code in BAD_HEADS:
        assert append(lib, p=heads(**kw)) == code, kw
    for kw, code in ((dict(p=heads(Hkv=1)), INVALID), (dict(p=heads(D=256)), INVALID), (dict(k=None), INVALID),
                     (dict(v=None), INVALID), (dict(q=GOOD), INVALID), (dict(qo=GOOD), INVALID), (dict(T=-1), INVALID),
                     (dict(ks=128), INVALID), (dict(vs=260), ALIGNMENT), (dict(q=GOOD, qo=GOOD, qs=8), INVALID),
                     (dict(k=GOOD + 4), ALIGNMENT), (dict(q=GOOD + 2, qo=GOOD), ALIGNMENT), (dict(lens=GOOD), INVALID),
                     (dict(lens=GOOD + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(n=255), WORKSPACE)):
        assert append(lib, **kw) == code, kw
    assert append(lib, T=0, k=None, v=None) == 0
    assert lib.dg_paged_append_workspace() == 256


def test_norm_rope_refuses(lib):
    for kw, code in BAD_HEADS:
        assert rope(lib, p=heads(**kw)) == code, kw
    for kw, code in ((dict(p=heads(D=264)), UNSUPPORTED), (dict(p=heads(D=120, rot=16)), UNSUPPORTED),
                     (dict(q=None, k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID),
                     (dict(pos=None), INVALID), (dict(T=-1), INVALID), (dict(qs=504), INVALID), (dict(kos=260), ALIGNMENT),
                     (dict(q=GOOD + 8), ALIGNMENT), (dict(ko=GOOD + 2), ALIGNMENT)):
        assert rope(lib, **kw) == code, kw
    assert rope(lib, T=0, q=None, k=None) == 0


def test_rope_steps(lib):
    """The steps are the turns per position to 2^-53 of themselves; position x step modulo one turn is the angle."""
    f = [10000.0 ** (-m / 64) for m in range(64)] + [0.0, 2 * math.pi, -0.25, 7.5]
    steps = dg.rope_steps(f, "cpu").tolist()
    assert steps[64] == 0 and steps[65] == 0
    for x, s in zip(f, steps):
        for pos in (1, 77, 4096, 262143):
            turns = (pos * (s % 2 ** 64) % 2 ** 64) / 2 ** 64
            want = math.fmod(pos * x, 2 * math.pi) / (2 * math.pi) % 1.0
            off = abs(turns - want)
            # the step is off by 2^-52 of itself; so is the product here, and its remainder by 2^-53 of 2^21
            assert min(off, 1 - off) < pos * (abs(x) + 1) * 2 ** -50, (x, pos)
    assert lib.dg_rope_steps(None, 3, None) == INVALID and lib.dg_rope_steps(None, 0, None) == 0
    for bad in (math.nan, math.inf):
        with pytest.raises(dg.DgError):
            dg.rope_steps([1.0, bad], "cpu")


def test_binding_checks_its_tensors(lib):
    """Wrong types, shapes and strides are refused by the Python binding, which hands the library addresses only."""
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(dg.DgError):     # not on a GPU
        dg.PagedCache(torch.zeros(4, 16, 2, 128, **bf), torch.zeros(4, 16, 2, 128, **bf),
                      torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(3, dtype=torch.int32))
    with pytest.raises(dg.DgError):
        dg.head_params(4, 2, 128, q_weight=torch.ones(64, **bf))
    with pytest.raises(dg.DgError):
        dg.head_params(4, 2, 128, q_weight=torch.ones(128))
    with pytest.raises(dg.DgError):
        dg.head_params(4, 2, 128, rope_steps=torch.zeros(64))
    p = dg.head_params(4, 2, 128, rope_steps=dg.rope_steps([1.0] * 32, "cpu"))
    assert p.rot == 64


def test_binding_refuses_rows_that_overlap_and_other_devices(lib):
    """The library takes a row stride of 0 for dense rows: an expanded tensor must not reach it.  Tensors that
    stay on the host are refused where a call would hand their addresses to a kernel."""
    x = torch.zeros(1, 4, 128, dtype=torch.bfloat16)

    def stride(t, T):
        address, s0 = dg._rows(t, (T, 4, 128), "x", -1)
        assert address == t.data_ptr()
        return s0

    assert stride(x, 1) == 0 and stride(x.repeat(3, 1, 1), 3) == 512 and stride(x[:0], 0) == 0
    assert stride(torch.zeros(3, 1024, dtype=torch.bfloat16)[:, 512:].view(3, 4, 128), 3) == 1024
    for bad in (x.expand(3, 4, 128), torch.zeros(3, 1, 128, dtype=torch.bfloat16).expand(3, 4, 128),
                torch.zeros(3 * 512, dtype=torch.bfloat16).as_strided((3, 4, 128), (256, 128, 1)),
                torch.zeros(3, 128, 4, dtype=torch.bfloat16).mT, torch.zeros(3, 4, 128), x[0], x.view(1, 8, 64), x):
        with pytest.raises(dg.DgError):
            stride(bad, 3)
    with pytest.raises(dg.DgError):
        dg._rows(x, (1, 4, 128), "x", 0)             # not on that device
    with pytest.raises(dg.DgError):
        dg._ints(torch.zeros(4, dtype=torch.int32), 4, "x", 0)
    p = dg.head_params(4, 2, 128, rope_steps=dg.rope_steps([1.0] * 32, "cpu"))
    with pytest.raises(dg.DgError):
        dg._heads_on(p, "x", 0)
    dg._heads_on(dg.head_params(4, 2, 128), "x", 0)
    with pytest.raises(dg.DgError):
        dg._scratch(torch.zeros(256, dtype=torch.uint8), "x", 0)
    with pytest.raises(dg.DgError):
        dg.qk_norm_rope(x, None, x, None, None, p)
    with pytest.raises(dg.DgError):
        dg.qk_norm_rope(None, None, None, None, None, p)
