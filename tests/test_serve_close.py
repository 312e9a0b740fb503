"""The comparisons of serve_close.py see what is wrong where an infinity is expected
(no GPU: what a call would give is computed here, and spoilt)."""
import math

import pytest
import torch

import serve_close as SC
import serve_plain as SP
from test_gpu_serve import BF, F32, request as make, weights_of

INF, NAN = math.inf, math.nan


def test_close_by_hand():
    want = torch.tensor([1.0, INF, -INF, NAN, 2.0, -INF, INF, -INF, NAN, 3.0]).double()
    got = torch.tensor([1.1, INF, -INF, NAN, 9.0, 5.0, -INF, NAN, 1.0, INF]).double()
    assert SC.close(got, want, torch.full((10,), INF).double()).tolist() == [True] * 5 + [False] * 5
    assert SC.close(got, want, torch.full((10,), 0.2).double()).tolist() == [True] * 4 + [False] * 6


def plain(logits, out=None, spoil=None, **a):
    """adjust_logits by the plain implementation; `spoil` changes the rows before they are stored."""
    y, _, _ = SP.adjust(logits, **{k: v for k, v in a.items() if k != spoil})
    y = y.to(logits.dtype)
    if callable(spoil):
        spoil(y)
    to = logits if out is None else out["logits"]
    for b in range(y.shape[0]):
        rows = int(a["gamma"][b]) + 1 if "gamma" in a else y.shape[1]
        to[b, :rows] = y[b, :rows]
    return {"logits": to, "status": torch.zeros(y.shape[0], dtype=torch.int32)}


def request(dtype, **more):
    x, a = make(2, 3, 700, 60, 5, biases=12, allowed=0.7, dtype=dtype, **more)
    a["bias_value"][:, 3] = -INF
    return x, {**a, "gamma": torch.tensor([2, 1], dtype=torch.int32)}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_adjusted_rows_that_are_right(dtype):
    x, a = request(dtype)
    SC.check_adjusted(plain, x, a, lay=torch.clone, lay_out=torch.clone)


def put(value):
    """Gives the first removed logit that value."""
    def spoil(y):
        y[tuple(torch.isinf(y[:, :2]).nonzero()[0].tolist())] = value
    return spoil


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spoil", ["mask", put(0.5), put(INF), put(NAN), put(-3e38)])
def test_removed_logits_that_are_not(dtype, spoil):
    x, a = request(dtype)
    with pytest.raises(AssertionError):
        SC.check_adjusted(lambda *p, **k: plain(*p, spoil=spoil, **k), x, a, lay=torch.clone, lay_out=torch.clone)
    only = {"mask": a["mask"]}                        # the mask alone, too
    with pytest.raises(AssertionError):
        SC.check_adjusted(lambda *p, **k: plain(*p, spoil=spoil, **k), x, only, lay=torch.clone, lay_out=torch.clone)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_with_infinities_that_are_wrong(dtype):
    q, scale, z = weights_of(60, 160, 32, True, 3)
    x = torch.randn(4, 160).to(BF)
    x[2, 40], scale[5, 1], scale[6, 4] = INF, INF, -INF
    want, tol = SC.product(x, q, scale, z, 32, dtype)
    right = want.to(dtype).double()
    SC.all_close(right, want, tol)
    assert torch.isinf(want[2]).any() and torch.isinf(want[0, 5]) and torch.isinf(want[0, 6])
    for at in ((2, int(torch.isinf(want[2]).nonzero()[0])), (0, 5), (3, 6)):
        for value in (0.0, -float(right[at]), NAN):
            wrong = right.clone()
            wrong[at] = value
            with pytest.raises(AssertionError):
                SC.all_close(wrong, want, tol)
    # a finite product is what the matrix of weights gives
    w = SP.weights(q, scale, z, 32)
    fine = torch.isfinite(want)
    assert torch.allclose(want[fine], (x.double() @ w.t())[fine], rtol=1e-12, atol=1e-12)
