"""The drafter-training calls: host checks (no GPU, nothing is launched), the
workspace sizes, and the plain implementations against differences."""
import ctypes
import threading
import time
import types

import pytest
import torch

import train_plain as TP

P = ctypes.c_void_p
FAKE = P(0x7f0000000000)           # never dereferenced: the host checks fail first
ODD = P(0x7f0000000001)


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verification_26_gb300 import build
    import speculative_decoding_verification_26_gb300 as sv
    build.build()
    return sv.lib()


def bad(base, **change):
    a = dict(base)
    a.update(change)
    return list(a.values())


RECORD = dict(logits=FAKE, dtype=1, n=4, V=1024, K=8, temperature=None, top=FAKE, idx=FAKE, tail=FAKE, status=None,
              stream=None)


@pytest.mark.parametrize("change", [
    {"logits": None}, {"logits": ODD}, {"dtype": 2}, {"n": 0}, {"n": (1 << 30) + 1}, {"V": 1}, {"V": 1 << 28}, {"K": 0}, {"K": 257},
    {"V": 7}, {"top": None}, {"idx": None}, {"tail": None}, {"tail": ODD}, {"temperature": ODD}, {"status": ODD}])
def test_record_refusals(L, change):
    assert L.spec_topk_logits(*bad(RECORD, **change)) == 1


DISTILL = dict(logits=FAKE, dtype=1, n=4, V=1024, K=8, top=FAKE, idx=FAKE, tail=None, label=None, w=None, T=None,
               kl=1.0, tv=0.0, ce=0.0, loss=FAKE, parts=None, grad=None, status=None, stream=None)


@pytest.mark.parametrize("change", [
    {"logits": None}, {"logits": ODD}, {"dtype": 2}, {"n": 0}, {"n": (1 << 30) + 1}, {"V": 1}, {"V": (1 << 20) + 1}, {"K": 0}, {"K": 257},
    {"top": None}, {"idx": None}, {"loss": None}, {"label": ODD}, {"parts": ODD}, {"grad": ODD},
    {"kl": float("nan")}, {"tv": float("inf")}, {"ce": float("nan")},
    {"grad": P(0x7f0000000000 + 2 * 1024)}, {"grad": P(0x7f0000000000 - 2)}])
def test_distill_refusals(L, change):
    assert L.spec_distill_topk(*bad(DISTILL, **change)) == 1


FWD = dict(hidden=FAKE, weight=FAKE, dtype=1, n=4, H=64, V=1000, label=FAKE, loss=FAKE, lse=FAKE, status=None,
           ws=FAKE, size=1 << 30, stream=None)
W, GW = 0x7a0000000000, 0x7b0000000000        # apart from FAKE, and from one another
BWD = dict(hidden=FAKE, weight=P(W), dtype=1, n=4, H=64, V=1000, label=FAKE, lse=FAKE, g=None, gh=FAKE, gw=P(GW),
           ws=FAKE, size=1 << 30, stream=None)
EITHER = [({"hidden": None}, 1), ({"weight": None}, 1), ({"dtype": 0}, 1), ({"n": 0}, 1), ({"n": (1 << 20) + 1}, 1),
          ({"n": 1 << 20, "V": (1 << 28) - 1}, 1),
          ({"H": 0}, 1), ({"H": 65544}, 1), ({"H": 60}, 1), ({"V": 1}, 1), ({"V": 1 << 28}, 1), ({"label": None}, 1),
          ({"lse": None}, 1), ({"hidden": P(0x7f0000000008)}, 1), ({"weight": P(0x7f0000000008)}, 1),
          ({"ws": None}, 2), ({"size": 1024}, 2), ({"ws": P(0x7f0000000010)}, 1)]


@pytest.mark.parametrize("change,code", EITHER + [({"loss": None}, 1), ({"status": ODD}, 1)])
def test_ce_forward_refusals(L, change, code):
    assert L.spec_linear_ce_forward(*bad(FWD, **change)) == code


@pytest.mark.parametrize("change,code", EITHER + [({"gh": None, "gw": None}, 1), ({"gw": P(0x7f0000000008)}, 1),
                                                  ({"g": ODD}, 1), ({"gw": P(W)}, 1),
                                                  ({"gw": P(W + 2 * 64 * 1000 - 16)}, 1), ({"gw": FAKE, "gh": None}, 1),
                                                  ({"gh": P(W)}, 1), ({"gh": P(GW + 256)}, 1),
                                                  ({"gh": P(0x7f0000000010)}, 1)])
def test_ce_backward_refusals(L, change, code):
    assert L.spec_linear_ce_backward(*bad(BWD, **change)) == code


def test_ce_workspace_bytes(L):
    f = L.spec_linear_ce_workspace_bytes
    assert f(0, 64, 1000, 0) == 0 and f(4, 60, 1000, 0) == 0 and f(4, 64, 1, 1) == 0
    for args in ((1, 8, 2), (4096, 2048, 151936), (1 << 20, 65536, 1000)):
        for backward in (0, 1):
            b = f(*args, backward)
            assert b > 0 and b % 256 == 0
            size = dict(n=args[0], H=args[1], V=args[2], size=b - 1)
            if max(args) * max(args[1:]) > 1 << 34:
                continue                   # its operands would overlap at these addresses
            call, base = (L.spec_linear_ce_backward, BWD) if backward else (L.spec_linear_ce_forward, FWD)
            assert call(*bad(base, **size)) == 2
    # the logits of this batch would take 2.5 GB; neither pass keeps them
    assert f(4096, 2048, 151936, 0) < 128 << 20
    assert f(4096, 2048, 151936, 1) < 768 << 20


def test_wrappers_refuse_cpu_tensors():
    import speculative_decoding_verification_26_gb300 as sv
    x = torch.zeros(2, 16)
    with pytest.raises(ValueError):
        sv.topk_logits(x, 4)
    with pytest.raises(ValueError):
        sv.distill_topk(x, torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.linear_ce_forward(x.bfloat16(), x.bfloat16(), torch.zeros(2, dtype=torch.int32))


def test_plain_gradients_against_differences():
    """The 64-bit formulas themselves: central differences of the losses."""
    g = torch.Generator().manual_seed(3)
    n, V, K = 3, 13, 4
    x = torch.randn(n, V, generator=g, dtype=torch.double) * 2
    z = x + torch.randn(n, V, generator=g, dtype=torch.double)
    T, w = torch.tensor([1.0, 0.7, 1.3]), torch.tensor([1.0, 0.5, 2.0])
    top, idx, tail = TP.record(x, K, T)
    label = torch.tensor([int(idx[0, 1]), -1, 5])
    for tl in (tail, None):
        args = (top, idx, tl, label, w, T, 0.7, 1.1, 0.3)
        grad = TP.distill(z, *args)[2]
        for v in range(V):
            d = torch.zeros(n, V, dtype=torch.double)
            d[:, v] = 1e-6
            diff = (TP.distill(z + d, *args)[0] - TP.distill(z - d, *args)[0]) / 2e-6
            assert torch.allclose(diff, grad[:, v], atol=1e-7)
    h = torch.randn(4, 5, generator=g, dtype=torch.double)
    wt = torch.randn(7, 5, generator=g, dtype=torch.double)
    lab, gl = torch.tensor([2, -1, 6, 0]), torch.tensor([0.5, 1.0, 2.0, 0.0], dtype=torch.double)
    gh, gw = TP.ce_backward(h, wt, lab, gl)[:2]
    total = lambda a, b: (TP.ce_forward(a, b, lab)[0] * gl).sum()   # noqa: E731
    for t, gt, f in ((h, gh, lambda a: total(a, wt)), (wt, gw, lambda b: total(h, b))):
        for k in range(t.numel()):
            d = torch.zeros_like(t).view(-1)
            d[k] = 1e-6
            d = d.view_as(t)
            assert abs((f(t + d) - f(t - d)) / 2e-6 - gt.view(-1)[k]) < 1e-7


def test_threads_take_turns_on_a_cached_workspace(monkeypatch):
    """Host threads on one stream, with the library's calls replaced: no two of them
    are in a call with the same workspace, and a thread on another stream has its own."""
    from speculative_decoding_verification_26_gb300 import _lib as lib
    stream = threading.local()
    busy, wrong, seen = set(), [], set()

    def entry(*args):
        ws = args[-3]
        if ws in busy:
            wrong.append(ws)
        busy.add(ws)
        seen.add((stream.id, ws))
        time.sleep(0.002)                  # as ctypes does, without the interpreter's lock
        busy.discard(ws)
        return 0

    entry.__name__ = "entry"
    cuda = types.SimpleNamespace(is_current_stream_capturing=lambda: False)
    h = types.SimpleNamespace(
        torch=types.SimpleNamespace(uint8=torch.uint8, device=torch.device, cuda=cuda), empty=torch.empty,
        f32=torch.float32, i32=torch.int32, bf16=torch.bfloat16, device=lambda: None, stream=lambda i: stream.id,
        ce_forward=entry, ce_backward=entry)
    monkeypatch.setattr(lib, "_hot", lambda: h)
    monkeypatch.setattr(lib, "_check", lambda *a, **k: None)
    monkeypatch.setattr(lib, "_ce_ws_cache", {})
    monkeypatch.setattr(lib, "linear_ce_workspace_bytes", lambda n, H, V, b: 256 * (2 if b else 1) * n)
    x, label = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)

    def work(k):
        stream.id = 7 if k < 4 else 8
        for n in (2, 4, 3):
            lse = lib.linear_ce_forward(x[:n], x, label[:n])["lse"]
            lib.linear_ce_backward(x[:n], x, label[:n], lse)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert {s for s, _ in seen} == {7, 8}
