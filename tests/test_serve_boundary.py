"""4-bit weights and adjusted logits: host checks (no GPU, nothing is launched),
the plain implementations by hand, and what a first call configures."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import serve_plain as SP

P = ctypes.c_void_p
FAKE = P(0x7f0000000000)           # never dereferenced: the host checks fail first
ODD = P(0x7f0000000001)
W, S, Z, Y, T = 0x7a0000000000, 0x7b0000000000, 0x7c0000000000, 0x7d0000000000, 0x7e0000000000


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verification_26_gb300 import build
    import speculative_decoding_verification_26_gb300 as sv
    build.build()
    return sv.lib()


def args(base, **change):
    a = dict(base)
    a.update(change)
    return list(a.values())


QUANT = dict(weight=FAKE, dtype=1, V=100, H=256, group=128, packed=P(W), scale=P(S), zero=P(Z), status=P(T), stream=None)
WEIGHTS = [{"V": 0}, {"V": 1 << 28}, {"H": 0}, {"H": 48}, {"H": 65568}, {"group": 16}, {"group": 256}, {"group": 0},
           {"packed": None}, {"scale": None}, {"packed": P(W + 8)}, {"scale": ODD}]


@pytest.mark.parametrize("change", WEIGHTS + [
    {"weight": None}, {"weight": P(0x7f0000000008)}, {"dtype": 2}, {"status": ODD}, {"packed": FAKE}, {"scale": FAKE},
    {"zero": FAKE}, {"scale": P(W + 100 * 128 - 2)}, {"zero": P(S + 100 * 2 * 2 - 1)}, {"zero": P(W)}, {"status": P(W)},
    {"status": P(0x7f0000000000 + 100 * 256 * 2 - 4)}])
def test_quantize_refusals(L, change):
    assert L.spec_w4_quantize(*args(QUANT, **change)) == 1


DEQUANT = dict(packed=P(W), scale=P(S), zero=None, V=100, H=256, group=128, weight=FAKE, dtype=1, stream=None)


@pytest.mark.parametrize("change", WEIGHTS + [
    {"weight": None}, {"weight": P(0x7f0000000008)}, {"dtype": 2}, {"weight": P(W + 100 * 128 - 16)}, {"weight": P(S)},
    {"weight": P(Z), "zero": P(Z + 16)}])
def test_dequantize_refusals(L, change):
    assert L.spec_w4_dequantize(*args(DEQUANT, **change)) == 1


LINEAR = dict(hidden=FAKE, dtype=1, n=4, packed=P(W), scale=P(S), zero=None, V=100, H=256, group=128, logits=P(Y),
              logits_dtype=0, stream=None)


@pytest.mark.parametrize("change", WEIGHTS + [
    {"hidden": None}, {"hidden": P(0x7f0000000008)}, {"dtype": 0}, {"n": 0}, {"n": (1 << 20) + 1},
    {"n": 1 << 20, "V": (1 << 28) - 1}, {"logits": None}, {"logits_dtype": 2}, {"logits": P(Y + 2)},
    {"logits": ODD, "logits_dtype": 1}, {"logits": FAKE}, {"logits": P(W)}, {"logits": P(S - 4)},
    {"logits": P(Z), "zero": P(Z + 4 * 4 * 100 - 1)}])
def test_linear_refusals(L, change):
    assert L.spec_linear_w4(*args(LINEAR, **change)) == 1


ADJUST = dict(logits=FAKE, out=FAKE, dtype=1, B=4, R=3, V=1000, history=P(W), L=64, history_len=None, prompt_len=None,
              draft=P(S), D=2, gamma=None, rep=None, freq=None, pres=None, bias_index=None, bias_value=None, biases=0,
              mask=P(Z), status=P(T), stream=None)


@pytest.mark.parametrize("change", [
    {"logits": None}, {"out": None}, {"logits": ODD, "out": ODD}, {"dtype": 2}, {"B": 0}, {"B": 65536}, {"R": 0}, {"R": 33},
    {"V": 1}, {"V": 1 << 28}, {"L": -1}, {"L": (1 << 28) + 1}, {"history": None}, {"history": ODD}, {"D": -1}, {"D": 33},
    {"D": 1}, {"draft": None}, {"draft": ODD}, {"biases": -1}, {"biases": 4097}, {"biases": 1}, {"history_len": ODD},
    {"prompt_len": ODD}, {"gamma": ODD}, {"rep": ODD}, {"freq": ODD}, {"pres": ODD}, {"mask": ODD}, {"status": ODD},
    {"biases": 2, "bias_index": P(Y)}, {"biases": 2, "bias_index": P(Y), "bias_value": ODD},
    {"out": P(0x7f0000000002)}, {"out": P(0x7f0000000000 - 2 * 4 * 3 * 1000 + 2)}, {"out": P(W)}, {"out": P(Z)},
    {"out": P(T)}, {"status": FAKE, "out": P(Y)}, {"status": P(W)}, {"status": P(Z + 4 * 4 * 3 * 32 - 4)}])
def test_adjust_refusals(L, change):
    assert L.spec_adjust_logits(*args(ADJUST, **change)) == 1


def test_new_status_strings(L):
    assert b"penalty" in L.spec_request_status_string(256) and b"length" in L.spec_request_status_string(512)


def test_wrappers_refuse():
    import speculative_decoding_verification_26_gb300 as sv
    w, u = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(4, 1, dtype=torch.bfloat16)
    for call in (lambda: sv.quantize_w4(w), lambda: sv.quantize_w4(w[0]), lambda: sv.quantize_w4(w, 100),
                 lambda: sv.dequantize_w4(u, s), lambda: sv.linear_w4(w.bfloat16(), u, s),
                 lambda: sv.adjust_logits(w), lambda: sv.adjust_logits(w[None]),
                 lambda: sv.linear_w4(w.bfloat16(), u, s, group=7)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ plain forms

def test_plain_pack_by_hand():
    q = torch.tensor([[1, 2, 3, 4, 5, 6, 7, 8]])
    # nibbles 0 .. 7 hold weights 0, 2, 4, 6, 1, 3, 5, 7: the word 0x86427531
    assert SP.pack(q).tolist() == [[0x31, 0x75, 0x42, 0x86]]
    q = torch.randint(0, 16, (3, 64), generator=torch.Generator().manual_seed(1))
    assert torch.equal(SP.unpack(SP.pack(q)), q)


def test_plain_quantize_by_hand():
    w = torch.tensor([[7.0, -7.0, 0.5, 1.5, 2.5, -0.5, -1.5, 0.0] + [0.0] * 24])
    q, s, z = SP.quantize(w, 32, False)
    assert s.item() == 1.0 and z.item() == 8
    assert q[0, :8].tolist() == [15, 1, 8, 10, 10, 8, 6, 8]             # halves to even
    w = torch.tensor([[0.0, 15.0, 3.0, 2.5] + [0.0] * 28])
    q, s, z = SP.quantize(w, 32, True)
    assert s.item() == 1.0 and z.item() == 0 and q[0, :4].tolist() == [0, 15, 3, 2]
    w = torch.tensor([[-5.0, 10.0] + [1.0] * 30])
    q, s, z = SP.quantize(w, 32, True)
    assert z.item() == 5 and q[0, :3].tolist() == [0, 15, 6]
    assert torch.equal(SP.weights(q, s, z, 32), w.double())


def test_plain_adjust_by_hand():
    x = torch.tensor([[[2.0, -2.0, 1.0, 0.0]] * 3])
    y, _, touched = SP.adjust(x, torch.tensor([[0, 1, 2, 2, -1]], dtype=torch.int32), torch.tensor([4]),
                              torch.tensor([1]), torch.tensor([[2, 3]]), None, torch.tensor([2.0]), torch.tensor([0.25]),
                              torch.tensor([0.5]))
    # prompt {0}, outputs {1, 2, 2}; rows see 2 once more, then 3
    assert y[0, 0].tolist() == [1.0, -4.0 - 0.75, 0.5 - 1.0, 0.0]
    assert y[0, 1].tolist() == [1.0, -4.75, 0.5 - 1.25, 0.0]
    assert y[0, 2].tolist() == [1.0, -4.75, -0.75, -0.75]
    assert not touched[0, 1, 3] and touched[0, 2, 3]
    y, _, _ = SP.adjust(x, bias_index=torch.tensor([[3, 3, -1]]), bias_value=torch.tensor([[1.0, 2.0, 9.0]]),
                        mask=torch.tensor([[[15], [9], [0]]], dtype=torch.int32))
    assert y[0, 0].tolist() == [2.0, -2.0, 1.0, 3.0]
    assert y[0, 1].tolist() == [2.0, -math.inf, -math.inf, 3.0]
    assert y[0, 2].tolist() == [-math.inf] * 4


# ------------------------------------------------- the host side, with counters

KERNELS = r"""
#include "serve.cuh"
extern "C" {
int configured[2], launched[4], failing[2];
}
namespace sv {
cudaError_t configure_kernels() { return cudaSuccess; }
cudaError_t configure_record(int) { return cudaSuccess; }
cudaError_t configure_distill(int) { return cudaSuccess; }
cudaError_t configure_linear_ce() { return cudaSuccess; }
cudaError_t verify_blocks_per_sm(int* n) { *n = 1; return cudaSuccess; }
cudaError_t launch_plan(const Params&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_verify(const Params&, int, cudaStream_t, bool) { return cudaSuccess; }
cudaError_t launch_filter(const FiltParams&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_divergence(const DivParams&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_gamma_select(const float*, const float*, const float*, int, int32_t*, float*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_record(const RecordParams&, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_distill(const DistillParams&, int, int, cudaStream_t) { return cudaSuccess; }
size_t ce_layout(CeParams&, bool, void*) { return 256; }
cudaError_t launch_ce_forward(const CeParams&, int, cudaStream_t, int* n) { *n = 3; return cudaSuccess; }
cudaError_t launch_ce_backward(const CeParams&, int, cudaStream_t, int* n) { *n = 4; return cudaSuccess; }
static cudaError_t used(int f) { ++configured[f]; return failing[f] ? cudaErrorUnknown : cudaSuccess; }
static cudaError_t ran(int f) { ++launched[f]; return cudaSuccess; }
cudaError_t configure_w4() { return used(0); }
cudaError_t configure_adjust() { return used(1); }
cudaError_t launch_w4_quantize(const W4Params&, int, cudaStream_t) { return ran(0); }
cudaError_t launch_w4_dequantize(const W4Params&, int, cudaStream_t) { return ran(1); }
cudaError_t launch_w4_linear(const W4Params&, int, cudaStream_t) { return ran(2); }
cudaError_t launch_adjust(const AdjustParams&, int, cudaStream_t) { return ran(3); }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from speculative_decoding_verification_26_gb300 import build
    import test_first_use as F
    d = tmp_path_factory.mktemp("serve_first_use")
    (d / "kernels.cu").write_text(KERNELS)
    (d / "runtime.c").write_text(F.RUNTIME)
    r = subprocess.run(["gcc", "-fPIC", "-c", str(d / "runtime.c"), "-o", str(d / "runtime.o")], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    sources = [os.path.join(build.CSRC, "api.cu"), os.path.join(build.CSRC, "api_serve.cu"), str(d / "kernels.cu")]
    jobs = [subprocess.Popen([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
                              "-I", build.CSRC, "-c", src, "-o", str(d / f"{k}.o")],
                             stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for k, src in enumerate(sources)]
    for j in jobs:
        out = j.communicate()[0]
        assert j.returncode == 0, out

    def load(name):
        so = d / f"{name}.so"
        r = subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), *(str(d / f"{k}.o") for k in range(3)),
                            str(d / "runtime.o")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return ctypes.CDLL(str(so))
    return load


def typed(base):
    """The argument list with sizes as int: ctypes passes them so by default."""
    return [ctypes.c_int(a) if isinstance(a, int) else P(None) if a is None else a for a in base.values()]


CALLS = [("spec_w4_quantize", QUANT, 0), ("spec_w4_dequantize", DEQUANT, 0), ("spec_linear_w4", LINEAR, 0),
         ("spec_adjust_logits", ADJUST, 1)]


def test_a_call_configures_its_own_kernels_once(host):
    h = host("own")
    count = {k: (ctypes.c_int * n).in_dll(h, k) for k, n in (("configured", 2), ("launched", 4), ("failing", 2))}
    before = h.spec_launch_count()
    count["failing"][0] = 1
    assert [getattr(h, f)(*typed(a)) for f, a, _ in CALLS] == [3, 3, 3, 0]
    count["failing"][0] = 0
    for _ in range(2):
        assert [getattr(h, f)(*typed(a)) for f, a, _ in CALLS] == [0] * 4
    assert list(count["configured"]) == [4, 1] and list(count["launched"]) == [2, 2, 2, 3]
    assert h.spec_launch_count() - before == 9


def test_another_device_is_refused(host):
    h = host("other")
    ctypes.c_int.in_dll(h, "minor_version").value = 0
    assert [getattr(h, f)(*typed(a)) for f, a, _ in CALLS] == [4] * 4
    assert not any((ctypes.c_int * 2).in_dll(h, "configured"))
