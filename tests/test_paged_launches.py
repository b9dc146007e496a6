"""Which kernels the paged attention launches, on the host: the library's objects linked to a CUDA runtime of the
test's own, which records the launches and answers what the test tells it to."""
import ctypes
import os
import shutil
import subprocess

import pytest

import block_diffusion_decoding_gb300 as dg
from block_diffusion_decoding_gb300 import build as dgbuild

FAKE = r"""
#include <cuda_runtime_api.h>
#include <map>
#include <string>
#include <cstring>
static std::map<const void *, std::string> &names() { static std::map<const void *, std::string> m; return m; }
static std::string launched;
static int pair_regs = 168;
static std::string failing;
extern "C" {
void fake_set(int regs, const char *fail) { pair_regs = regs; failing = fail; }
const char *fake_launches() { static std::string s; s = launched; launched.clear(); return s.c_str(); }
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, void *, void *, void *, void *, int *)
{ names()[host] = name; }
static bool is(const void *f, const char *what) { return names()[f].find(what) != std::string::npos; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute, int)
{ return !failing.empty() && is(f, failing.c_str()) ? cudaErrorInvalidValue : cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *f)
{ std::memset(a, 0, sizeof *a); a->numRegs = is(f, "pair") ? pair_regs : 255; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    launched += names()[f] + " " + std::to_string(c->gridDim.x) + " " + std::to_string(c->blockDim.x) + "\n";
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) { *s = cudaStreamCaptureStatusNone; return cudaSuccess; }
static int encode() { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q)
{ *p = reinterpret_cast<void *>(&encode); *q = cudaDriverEntryPointSuccess; return cudaSuccess; }
}
"""
INC = os.path.join(os.path.dirname(os.path.dirname(dgbuild.nvcc())), "include")


def symbols(path, *flags):
    r = subprocess.run(["nm", *flags, path], capture_output=True, text=True, check=True)
    return {line.split()[-1] for line in r.stdout.splitlines() if line.strip()}


@pytest.fixture(scope="module")
def fake_lib(tmp_path_factory):
    """A maker of fresh copies of the library, each of which asks the fake runtime about its device anew."""
    dgbuild.build()
    objs = [os.path.join(dgbuild.BUILD, s[:-3] + ".o") for s in dgbuild.SOURCES]
    if not all(map(os.path.exists, objs)):
        dgbuild.build(force=True)
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.cpp").write_text(FAKE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-I", INC, "-c", str(d / "fake.cpp"), "-o", str(d / "fake.o")],
                   check=True)
    have = symbols(str(d / "fake.o"), "--defined-only")
    want = {s for o in objs for s in symbols(o, "-u") if s.startswith(("cuda", "__cuda"))} - have
    (d / "stubs.c").write_text("".join("void *%s(void) { return 0; }\n" % s for s in sorted(want)))
    subprocess.run(["gcc", "-fPIC", "-c", str(d / "stubs.c"), "-o", str(d / "stubs.o")], check=True)
    so = str(d / "libdg_fake.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", so, *objs, str(d / "fake.o"), str(d / "stubs.o"),
                    "-lpthread"], check=True)
    copies = []

    def make(regs=168, failing=""):
        path = str(d / ("copy%d.so" % len(copies)))
        shutil.copy(so, path)
        copies.append(path)
        lib = ctypes.CDLL(path)
        lib.fake_launches.restype = ctypes.c_char_p
        lib.fake_set(regs, failing.encode())
        lib.dg_paged_attn.argtypes = dg.lib().dg_paged_attn.argtypes
        lib.dg_qk_norm_rope.argtypes = dg.lib().dg_qk_norm_rope.argtypes
        return lib

    return make


GOOD = 1 << 20


def attn(lib, T, B=1, D=128, Hq=4, Hkv=2):
    c = dg.PagedCacheArgs(GOOD, GOOD, GOOD, GOOD, GOOD, 0, 100, 16, 20, B, Hkv, D)
    rc = lib.dg_paged_attn(GOOD, 0, None, 0, None, 0, GOOD, 0, T, Hq, 0.1, 1, 0, ctypes.byref(c), GOOD, 1 << 40, None)
    return rc, [line.split() for line in lib.fake_launches().decode().splitlines()]


def others(lib):
    """Calls that have nothing to do with the paged attention."""
    p = dg.HeadParams(4, 2, 128, 0, 0, 1e-6, 0.0, None, GOOD, GOOD)
    i = [ctypes.c_int() for _ in range(4)]
    rc = [lib.dg_qk_norm_rope(GOOD, 0, None, 0, GOOD, 0, None, 0, None, 5, ctypes.byref(p), None),
          lib.dg_lm_head_plan(256, 2816, 262144, *map(ctypes.byref, i))]
    assert "qk_norm_rope" in lib.fake_launches().decode()
    return rc


@pytest.mark.parametrize("D", [128, 256])
def test_kernel_by_the_rows_of_a_batch(fake_lib, D, monkeypatch):
    monkeypatch.delenv("DG_PAGED_KERNEL", raising=False)
    lib = fake_lib()
    for T, B, pair in ((64, 1, False), (65, 1, True), (128, 2, False), (2000, 3, True)):
        rc, ran = attn(lib, T, B, D)
        assert rc == 0 and ("paged_attn_pair_kernel_d%d" % D in ran[0][0]) == pair, (T, B, ran)
        assert "paged_merge_kernel" in ran[1][0] and ran[0][1] == "152"


@pytest.mark.parametrize("regs,failing", [(160, ""), (168, "paged_attn_pair_kernel")])
def test_a_pair_kernel_that_may_not_run_refuses_nothing_else(fake_lib, monkeypatch, regs, failing):
    """With fewer registers than its warps share out the pair kernel would wait for them forever.  The paged
    attention then runs on the other kernel, and no other call is the worse for it."""
    monkeypatch.setenv("DG_PAGED_KERNEL", "pair")
    lib = fake_lib(regs, failing)
    assert others(lib) == [0, 0]
    for T in (1, 3000):
        rc, ran = attn(lib, T)
        assert rc == 0 and "paged_attn_kernel_d128" in ran[0][0] and ran[0][1:] == ["152", "256"]


def test_no_paged_kernel_at_all(fake_lib):
    lib = fake_lib(168, "paged_attn")
    assert others(lib) == [0, 0]
    assert attn(lib, 5) == (5, [])


def test_a_refusal_of_the_runtime_does_not_last(fake_lib, monkeypatch):
    """What failed once (while the runtime was busy with a capture, say) is asked for again."""
    monkeypatch.delenv("DG_PAGED_KERNEL", raising=False)
    lib = fake_lib(168, "paged_attn_pair_kernel_d256")
    assert "paged_attn_kernel_d128" in attn(lib, 3000)[1][0][0]
    lib.fake_set(168, b"")
    for _ in range(2):
        assert "paged_attn_pair_kernel_d128" in attn(lib, 3000)[1][0][0]
    lib = fake_lib(168, "paged_attn")
    assert attn(lib, 3000)[0] == 5
    lib.fake_set(168, b"")
    assert attn(lib, 3000)[0] == 0
