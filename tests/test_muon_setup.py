"""The kernels of orthogonalised updates are set up by the first call that needs them: where their clusters of thread blocks do not fit
on a device (a part of a GPU, say), that refuses these calls and no others. On the CPU, against a stand-in for the CUDA runtime
that has an sm_103 device, launches nothing and knows kernels by the names they are registered under."""
import os
import shutil
import subprocess
import sys

import pytest

from hybrid_upcycling_gb300 import build

FAKE = r"""
#define _GNU_SOURCE
#include <cuda_runtime_api.h>
#include <dlfcn.h>
#include <stdlib.h>
#include <string.h>

static const void* of_muon[64];
static int known, asked;
static int is_muon(const void* f) {
  for (int i = 0; i < known; ++i) if (of_muon[i] == f) return 1;
  return 0;
}
int fake_asked(void) { return asked; }

void __cudaRegisterFunction(void** h, const char* host, char* dev, const char* name, int limit, void* a, void* b, void* c, void* d, int* w) {
  static void (*real)(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*);
  if (!real) *(void**)&real = dlsym(RTLD_NEXT, "__cudaRegisterFunction");
  if (strstr(name, "muon_pipe_kernel")) of_muon[known++] = host;
  real(h, host, dev, name, limit, a, b, c, d, w);
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* cfg) {
  (void)cfg;
  *n = 76;
  if (is_muon(f)) {
    ++asked;
    if (!getenv("FAKE_MUON_FITS")) *n = 0;
  }
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) { (void)d; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)d;
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) { (void)f, (void)a, (void)v; return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void* s) { static int word; (void)s; *p = &word; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int t, size_t s) { (void)f, (void)t, (void)s; *n = 1; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int t, size_t s, unsigned g) {
  (void)f, (void)t, (void)s, (void)g;
  *n = 1;
  return cudaSuccess;
}
static int encode(void) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** f, unsigned v, unsigned long long g, enum cudaDriverEntryPointQueryResult* q) {
  (void)s, (void)v, (void)g;
  *f = (void*)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t s, enum cudaStreamCaptureStatus* c) { (void)s; *c = cudaStreamCaptureStatusNone; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** a) { (void)c, (void)f, (void)a; return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) { (void)f; *k = 0; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3 b, void** a, size_t m, cudaStream_t s) {
  (void)k, (void)g, (void)b, (void)a, (void)m, (void)s;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
"""

CALLS = r"""
import ctypes, struct
from hybrid_upcycling_gb300 import _lib
lib, fake = _lib.load(), ctypes.CDLL(None)
at = lambda i: 0x10000000 * (i + 1)
k = (ctypes.c_double * 3)(3.4445, -4.775, 2.0315)

def norm():
    return lib.hylo_norm(at(0), None, 1, 4, 64, 64, 0, None, None, 1, 1, 1e-6, None, at(1), None, None)

def orthogonalize():
    table = struct.pack("=" + _lib.ORTH_MATRIX, at(0), at(1), 64, 64, 64)
    return lib.hylo_orthogonalize(table, 1, 0, 1, 1, k, 1e-7, at(8), 1 << 26, None)

def muon():
    table = struct.pack("=" + _lib.MUON_TENSOR, at(0), at(1), 0, at(2), 64, 64, 0.1, 0.0, 1.0)
    return lib.hylo_muon_step(table, 1, 0, 0, 0.9, 1, 1, k, 1e-7, 1.0, None, 1.0, 0, at(8), 1 << 26, None)

def error():
    return lib.hylo_kl_last_error().decode()
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    build.build()
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.c").write_text(FAKE)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-I", include, "-o", str(d / "fake.so"), str(d / "fake.c"), "-ldl"], check=True)

    def run(code, **env):
        r = subprocess.run([sys.executable, "-c", CALLS + code], cwd=build.ROOT, capture_output=True, text=True, timeout=300,
                           env={**os.environ, "LD_PRELOAD": str(d / "fake.so"), **env})
        assert r.returncode == 0, r.stderr[-2000:]
    return run


def test_other_calls_run_where_the_clusters_do_not_fit(fake):
    fake("""
assert norm() == 0, error()
for call in (orthogonalize, muon):
    assert call() == -6 and "cluster" in error(), error()
    assert norm() == 0, error()
""")


def test_set_up_once_by_the_first_call_that_needs_it(fake):
    fake("""
assert norm() == 0 and fake.fake_asked() == 0, (error(), fake.fake_asked())
assert orthogonalize() == 0, error()
n = fake.fake_asked()
assert n > 0 and muon() == 0 and orthogonalize() == 0 and fake.fake_asked() == n, error()
""", FAKE_MUON_FITS="1")
