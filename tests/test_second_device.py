"""A first call on a second device beside calls on the first: what host threads share of
the calls that copy by tensor maps, with the CUDA runtime replaced and every access of
the host code checked for races (no GPU)."""
import os
import subprocess

import pytest

from speculative_decoding_verification_26_gb300 import build

RUNTIME = r"""
#include <atomic>
#include <cuda.h>
std::atomic<int> lookups{0}, encoded{0}, failing{0};
static CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  ++encoded;
  return CUDA_SUCCESS;
}
extern "C" {
int cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, int* found) {
  ++lookups;
  if (failing) return 999;
  *f = reinterpret_cast<void*>(&fake_encode);
  *found = 0;                                /* cudaDriverEntryPointSuccess */
  return 0;
}
int cudaFuncSetAttribute(const void*, int, int) { return 0; }
int cudaLaunchKernelExC(const void*, const void*, void**) { return 0; }
int cudaGetLastError() { return 0; }
int __cudaGetKernel(void**, const void*) { return 0; }
int __cudaLaunchKernel(void*, ...) { return 0; }
unsigned __cudaPushCallConfiguration(...) { return 0; }
int __cudaPopCallConfiguration(void*, void*, void*, void*) { return 0; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
}
"""
PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <cstring>
#include <thread>
#include "serve.cuh"
extern std::atomic<int> lookups, encoded, failing;
int main(int, char** argv) {
  const bool w4 = !strcmp(argv[1], "w4");
  const auto configure = [&] { return (int)(w4 ? sv::configure_w4() : sv::configure_linear_ce()); };
  const auto call = [&] {
    static char memory[1 << 12];
    int n = 0;
    if (w4) {
      sv::W4Params P{};
      P.n = 1; P.H = 256; P.V = 128; P.group = 128; P.groups = 2;
      return (int)sv::launch_w4_linear(P, 152, nullptr);
    }
    sv::CeParams P{};
    P.n = 8; P.H = 64; P.V = 100;
    sv::ce_layout(P, false, memory);         // addresses alone
    return (int)sv::launch_ce_forward(P, 152, nullptr, &n);
  };
  failing = 1;
  if (configure() == 0) return 3;            // and it is tried again
  failing = 0;
  if (configure() != 0 || call() != 0) return 4;
  int a = 0, b = 0;
  std::thread second([&] { for (int i = 0; i < 100; ++i) a |= configure(); });
  std::thread first([&] { for (int i = 0; i < 100; ++i) b |= call(); });
  second.join();
  first.join();
  printf("%d %d %d %d\n", a, b, lookups.load(), encoded.load());
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("second_device")
    (d / "runtime.cpp").write_text(RUNTIME)
    (d / "main.cu").write_text(PROGRAM)
    checked = ["-Xcompiler", "-fsanitize=thread,-fPIE,-O1,-g"]
    cmd = [build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", *checked, "-Xptxas", "-O0", "-I", build.CSRC, "-c"]
    sources = [os.path.join(build.CSRC, "w4_linear.cu"), os.path.join(build.CSRC, "linear_ce.cu"), str(d / "main.cu"), str(d / "runtime.cpp")]
    jobs = [subprocess.Popen([*cmd, src, "-o", str(d / f"{k}.o")], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            for k, src in enumerate(sources)]
    for j in jobs:
        out = j.communicate()[0]
        assert j.returncode == 0, out
    r = subprocess.run(["g++", "-fsanitize=thread", "-pie", "-o", str(d / "program"), *(str(d / f"{k}.o") for k in range(4))],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "program")


@pytest.mark.parametrize("family", ["w4", "ce"])
def test_the_encoder_is_shared_without_a_race(program, family):
    """Looked up until it is found (once in vain, once more here), not again for another device."""
    r = subprocess.run([program, family], capture_output=True, text=True, timeout=120)
    if "unexpected memory mapping" in r.stderr:          # the sanitizer wants addresses less random
        r = subprocess.run(["setarch", "-R", program, family], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[:3000]
    a, b, lookups, encoded = map(int, r.stdout.split())
    assert (a, b, lookups) == (0, 0, 2) and encoded == 202
