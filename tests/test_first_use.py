"""What the first call of a family configures, with the kernels and the CUDA runtime
replaced: the host side of the library is linked against counters (no GPU)."""
import ctypes
import os
import subprocess

import pytest

from speculative_decoding_verification_26_gb300 import build

# the runtime's calls as the host side uses them, without its headers
RUNTIME = r"""
int minor_version = 3;
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int a, int dev) {
  *v = a == 75 ? 10 : a == 76 ? minor_version : 152;       /* cudaDevAttrComputeCapabilityMajor, Minor */
  return 0;
}
int cudaEventRecord(void* e, void* s) { return 0; }
int cudaGetSymbolAddress(void** p, const void* symbol) { return 999; }
int cudaMemsetAsync(void* p, int v, unsigned long n, void* s) { return 0; }
void** __cudaRegisterFatBinary(void* f) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void** h) {}
void __cudaUnregisterFatBinary(void** h) {}
char __cudaInitModule(void** h) { return 1; }
void __cudaRegisterVar(void** h, char* a, char* b, const char* c, int d, unsigned long e, int f, int g) {}
"""
KERNELS = r"""
#include "common.cuh"
extern "C" {
int configured[4], launched[4], failing[4];
}
namespace sv {
static cudaError_t used(int f) { ++configured[f]; return failing[f] ? cudaErrorUnknown : cudaSuccess; }
static cudaError_t ran(int f) { ++launched[f]; return cudaSuccess; }
cudaError_t configure_kernels() { return used(0); }
cudaError_t configure_record(int) { return used(1); }
cudaError_t configure_distill(int) { return used(2); }
cudaError_t configure_linear_ce() { return used(3); }
cudaError_t verify_blocks_per_sm(int* n) { *n = 1; return cudaSuccess; }
cudaError_t launch_plan(const Params&, cudaStream_t) { return ran(0); }
cudaError_t launch_verify(const Params&, int, cudaStream_t, bool) { return ran(0); }
cudaError_t launch_filter(const FiltParams&, int, cudaStream_t) { return ran(0); }
cudaError_t launch_divergence(const DivParams&, int, cudaStream_t) { return ran(0); }
cudaError_t launch_gamma_select(const float*, const float*, const float*, int, int32_t*, float*, cudaStream_t) { return ran(0); }
cudaError_t launch_record(const RecordParams&, int, int, cudaStream_t) { return ran(1); }
cudaError_t launch_distill(const DistillParams&, int, int, cudaStream_t) { return ran(2); }
size_t ce_layout(CeParams&, bool, void*) { return 256; }
cudaError_t launch_ce_forward(const CeParams&, int, cudaStream_t, int* n) { *n = 3; return ran(3); }
cudaError_t launch_ce_backward(const CeParams&, int, cudaStream_t, int* n) { *n = 4; return ran(3); }
}
"""


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    d = tmp_path_factory.mktemp("first_use")
    (d / "kernels.cu").write_text(KERNELS)
    (d / "runtime.c").write_text(RUNTIME)
    r = subprocess.run(["gcc", "-fPIC", "-c", str(d / "runtime.c"), "-o", str(d / "runtime.o")], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    jobs = [subprocess.Popen([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
                              "-I", build.CSRC, "-c", src, "-o", str(d / obj)],
                             stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            for src, obj in ((os.path.join(build.CSRC, "api.cu"), "api.o"), (str(d / "kernels.cu"), "kernels.o"))]
    for j in jobs:
        out = j.communicate()[0]
        assert j.returncode == 0, out
    return d


class Host:
    """A copy of the library's host side with its state new."""

    def __init__(self, objects, name):
        so = objects / f"{name}.so"
        # nothing is resolved outside: a second runtime must not be found in the process
        r = subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), str(objects / "api.o"),
                            str(objects / "kernels.o"), str(objects / "runtime.o")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        self.L = ctypes.CDLL(str(so))
        for k in ("configured", "launched", "failing"):
            setattr(self, k, (ctypes.c_int * 4).in_dll(self.L, k))
        self.minor = ctypes.c_int.in_dll(self.L, "minor_version")

    def call(self, family):
        P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        f = P(0x7f0000000000)              # never dereferenced
        w, g = P(0x7a0000000000), P(0x7b0000000000)
        one = I(1)
        if family == 0:
            return self.L.spec_verify_greedy(f, one, I(4), I(3), I(1000), f, f, f, f, f, f, Z(1 << 30), P(None))
        if family == 1:
            return self.L.spec_topk_logits(f, one, I(4), I(1000), I(8), P(None), f, f, f, P(None), P(None))
        if family == 2:
            return self.L.spec_distill_topk(f, one, I(4), I(1000), I(8), f, f, P(None), P(None), P(None), P(None),
                                            F(1), F(0), F(0), f, P(None), P(None), P(None), P(None))
        if family == 3:
            return self.L.spec_linear_ce_forward(f, w, one, I(4), I(64), I(1000), f, f, f, P(None), f, Z(1 << 30),
                                                 P(None))
        return self.L.spec_linear_ce_backward(f, w, one, I(4), I(64), I(1000), f, f, P(None), f, g, f, Z(1 << 30),
                                              P(None))


@pytest.mark.parametrize("family", range(4))
def test_a_call_configures_its_own_kernels_once(objects, family):
    h = Host(objects, f"own{family}")
    assert [h.call(family) for _ in range(3)] == [0, 0, 0]
    assert list(h.configured) == [int(k == family) for k in range(4)]
    assert h.launched[family] >= 3


@pytest.mark.parametrize("broken", range(4))
def test_what_fails_for_one_family_leaves_the_others(objects, broken):
    h = Host(objects, f"broken{broken}")
    h.failing[broken] = 1
    for family in (0, 1, 2, 3, 4):
        assert h.call(family) == (3 if min(family, 3) == broken else 0), family
    assert h.launched[broken] == 0
    h.failing[broken] = 0                  # it is tried again
    assert h.call(broken) == 0


def test_another_device_is_refused_by_every_family(objects):
    h = Host(objects, "other")
    h.minor.value = 0
    assert [h.call(f) for f in range(5)] == [4] * 5
    assert not any(h.configured) and not any(h.launched)
