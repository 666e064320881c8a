"""A process that uses two devices: every kernel whose shared memory passes the
default limit has the limit raised on each device before its first launch
there, and a setting that failed is tried again by the next call.

No GPU is touched.  The library's objects are linked against a small stand-in
for the CUDA runtime that keeps the limits per (device, kernel), as the runtime
does, and counts the launches that a device would refuse."""
import os
import subprocess
import sys
import textwrap

import pytest

from conftest import ROOT
from sft_trie_build_gb300 import build

RUNTIME = r"""
#include <driver_types.h>
#include <stddef.h>

static int device, failing, bad, launches, n_limits;
static cudaError_t last;
static struct { int device; const void* kernel; int bytes; } limits[4096];
static dim3 grid, block;
static size_t smem;

void fake_device(int d) { device = d; }
void fake_fail(int n) { failing = n; }
int fake_bad(void) { return bad; }
int fake_launches(void) { return launches; }

static int launch(const void* kernel, size_t bytes) {
  ++launches;
  int most = bytes < 49152 ? 49152 : 0;   /* the default, less what a kernel holds statically */
  for (int i = 0; i < n_limits; ++i)
    if (limits[i].device == device && limits[i].kernel == kernel) most = limits[i].bytes;
  if ((size_t)most < bytes) {
    ++bad;
    return last = cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* kernel, enum cudaFuncAttribute a, int v) {
  if (failing > 0) {
    --failing;
    return last = cudaErrorMemoryAllocation;
  }
  limits[n_limits].device = device;
  limits[n_limits].kernel = kernel;
  limits[n_limits++].bytes = v;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) {
  cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
const char* cudaGetErrorString(cudaError_t e) { return "refused"; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, enum cudaMemcpyKind k, cudaStream_t t) { return cudaSuccess; }
cudaError_t cudaMemcpy2DAsync(void* d, size_t dp, const void* s, size_t sp, size_t w, size_t h, enum cudaMemcpyKind k,
                              cudaStream_t t) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void* v) { *p = (void*)v; return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned f) { *s = 0; return cudaSuccess; }
cudaError_t cudaStreamCreateWithPriority(cudaStream_t* s, unsigned f, int p) { *s = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetStreamPriorityRange(int* a, int* b) { *a = *b = 0; return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned f) { return cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned f) { *e = 0; return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* kernel, void** args) {
  return launch(kernel, c->dynamicSmemBytes);
}
static int encode(void) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned v, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* r) {
  *f = (void*)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t n, struct CUstream_st* s) {
  grid = g;
  block = b;
  smem = n;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* n, void* s) {
  *g = grid;
  *b = block;
  *n = smem;
  *(void**)s = 0;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) { *k = (cudaKernel_t)f; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3 b, void** args, size_t n, cudaStream_t s) {
  return launch((const void*)k, n);
}
void** __cudaRegisterFatBinary(void* p) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void** h) {}
void __cudaUnregisterFatBinary(void** h) {}
void __cudaRegisterFunction(void** h, const char* f, char* d, const char* n, int t, void* a, void* b, void* c, void* e,
                            int* w) {}
void __cudaRegisterVar(void** h, char* v, char* d, const char* n, int e, size_t s, int c, int g) {}
"""

CALLS = """
import ctypes, sys
import numpy as np
sys.path.insert(0, sys.argv[2])
from sft_trie_build_gb300 import stp
stp.LIB_PATH = sys.argv[1]
fake = ctypes.CDLL(sys.argv[1])
A = 1 << 20
B, F = stp.STP_BF16, stp.STP_FP32

def stats(dt, n):
    d = stp.stats_desc(n, 40000, 5, dt)
    stp.stp_token_stats_fwd(d, *[A] * 8, stream=0)
    stp.stp_token_stats_bwd(d, *[A] * 7, stream=0)

def distill(dt, n):
    d = stp.distill_desc(n, 40000, 5, dt)
    stp.stp_distill_fwd(d, *[A] * 7, stream=0)
    stp.stp_distill_bwd(d, *[A] * 7, stream=0)
    stp.stp_distill_step(d, *[A] * 9, stream=0)

def qk(dt, d):
    desc = stp.qk_desc(9, 3, 1, d, d, False, dt)
    f = np.ones(d // 2)
    stp.stp_qk_norm_rope_fwd(desc, A, A, A, A, f, A, A, A, stream=0)
    stp.stp_qk_norm_rope_bwd(desc, A, A, A, A, f, *[A] * 8, stream=0)

def attn(dt, hq):
    d = stp.Desc(1, 256, hq, 1, 128, dt)
    stp.stp_attn_fwd(d, *[A] * 8, stream=0)
    stp.stp_attn_bwd(d, *[A] * 12, stream=0)
    stp.stp_attn_window_fwd(d, 9, 0, *[A] * 9, stream=0)
    stp.stp_attn_window_bwd(d, 9, 0, *[A] * 13, stream=0)

def index():
    stp.stp_index_topk(stp.index_desc(1, 256, 4, 128, 8), *[A] * 8, stream=0)

def logprob():
    stp.stp_logprob_gather(stp.logprob_desc(1, 128, 128, 1000), *[A] * 6, stream=0)

def gdn():
    d = stp.gdn_desc(1, 256, 2)
    plan = stp.stp_gdn_plan(d, np.full((1, 256), 255, np.int32))
    stp.stp_gdn_fwd(d, plan, *[A] * 7, stream=0)
    stp.stp_gdn_bwd(d, plan, *[A] * 11, stream=0)

calls = [lambda dt=dt, n=n, f=f: f(dt, n) for f in (stats, distill) for dt in (B, F) for n in (2, 700)]
calls += [lambda dt=dt, d=d: qk(dt, d) for dt in (B, F) for d in (16, 32, 64, 128, 256, 512)]
calls += [lambda dt=dt, h=h: attn(dt, h) for dt in (B, F) for h in (1, 4)] + [index, logprob, gdn]
for device in (0, 1, 5, 0):
    fake.fake_device(device)
    for call in calls:
        call()
assert fake.fake_launches() > 4 * len(calls)
assert fake.fake_bad() == 0, f"{fake.fake_bad()} of {fake.fake_launches()} launches refused"
# a setting that fails once is an error of that call alone
fake.fake_device(7)
for call in calls:
    fake.fake_fail(1)
    try:
        call()
    except stp.StpError as e:
        assert e.status == stp.STP_ECUDA
    fake.fake_fail(0)
    call()
print("done")
"""


@pytest.fixture(scope="module")
def fake_lib(stp_lib, tmp_path_factory):
    at = tmp_path_factory.mktemp("runtime")
    cu, cpp = build.sources()
    objects = [os.path.join(build.BUILD, f + ".o") for f in cu + cpp]
    if not all(os.path.exists(o) for o in objects):
        build.build()
    src, lib = at / "runtime.c", at / "libstp_fake.so"
    src.write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    subprocess.check_call(["gcc", "-fPIC", "-w", "-I", include, "-c", str(src), "-o", str(at / "runtime.o")])
    subprocess.check_call(["g++", "-shared", "-Wl,-Bsymbolic", "-Wl,-z,lazy", "-o", str(lib), *objects,
                           str(at / "runtime.o"), "-lpthread"])
    return str(lib)


def test_limits_are_raised_on_every_device(fake_lib):
    p = subprocess.run([sys.executable, "-c", textwrap.dedent(CALLS), fake_lib, ROOT], capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and "done" in p.stdout, p.stdout + p.stderr
