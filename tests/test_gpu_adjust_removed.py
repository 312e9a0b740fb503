"""What a mask or a ban removes, on the GPU: equal to what the 64-bit plain implementation
gives (tolerances: serve_close.py)."""
import math

import pytest
import torch

import serve_close as SC
from test_gpu_serve import BF, F32, guarded, request, sv          # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def check_adjusted(sv, x, a, refused=(), in_elems=0, out_elems=0):       # noqa: F811
    guards = []

    def lay(elems):
        def to(y):
            t, guard = guarded(y.shape, y.dtype, elems)
            guards.append(guard)
            return t.copy_(y)
        return to

    def call(logits, out=None, **k):
        return sv.adjust_logits(logits, **{n: v.cuda() for n, v in k.items()}, out=out)
    SC.check_adjusted(call, x, a, refused, lay(in_elems), lay(out_elems))
    for guard in guards:
        guard()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("keep", [("mask",), ("mask", "gamma"), ("bias_index", "bias_value"),
                                  ("history", "history_len", "repetition", "mask"),
                                  ("draft_tokens", "gamma", "presence", "bias_index", "bias_value", "mask"), None])
def test_removed_logits(sv, keep, dtype):             # noqa: F811
    for allowed in (0.02, 0.5, 0.98):
        x, a = request(3, 4, 6001, 200, 11, biases=40, allowed=allowed, dtype=dtype, D=4 if keep is None or "draft_tokens" in keep else 3)
        a["bias_value"][:, ::7] = -INF
        check_adjusted(sv, x, a if keep is None else {k: v for k, v in a.items() if k in keep})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_elems,out_elems", [(0, 0), (1, 1), (3, 3), (0, 1), (5, 2)])
@pytest.mark.parametrize("V", [2, 31, 33, 1000, 2048, 4100, 8200, 5003])
def test_removed_logits_of_unaligned_rows(sv, V, in_elems, out_elems, dtype):          # noqa: F811
    x, a = request(2, 3, V, 300, 13, biases=12, allowed=0.8, dtype=dtype)
    check_adjusted(sv, x, a, in_elems=in_elems, out_elems=out_elems)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 8192, 40000])
def test_rows_that_a_mask_empties(sv, V, dtype):      # noqa: F811
    """Rows without an allowed token, with one, with all; infinities, NaN and the lowest value under the mask or not."""
    x, a = request(2, 5, V, 50, 19, biases=20, allowed=0.5, dtype=dtype)
    a["mask"][:, :2] = 0
    a["mask"][:, 1, 0] = 1 << 7
    a["mask"][:, 2] = -1
    a["mask"][:, 3, ::2] = 0
    x[:, :, 3], x[:, :, 64], x[:, :, 50], x[:, :, V - 2] = NAN, INF, -INF, torch.finfo(dtype).min
    a["history"][:, :3] = torch.tensor([3, 64, 50])
    check_adjusted(sv, x, {k: v for k, v in a.items() if k != "gamma"})
