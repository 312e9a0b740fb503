"""Infinities of hidden states and scales in products with 4-bit weights on the GPU: equal to
what the formula gives in 64 bits (tolerances: serve_close.py)."""
import math

import pytest
import torch

import serve_close as SC
import serve_plain as SP
from test_gpu_serve import BF, F32, cuda, gen, guarded, sv, weights_of          # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


@pytest.mark.parametrize("n", [1, 4, 24, 70, 130])
@pytest.mark.parametrize("V,H,group", [(300, 160, 32), (129, 416, 128), (130, 4096, 64), (70, 8192, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_with_infinities(sv, n, V, H, group, dtype):            # noqa: F811
    """Of hidden states and of scales, of either sign, alone and where they meet; the last two sizes split
    their k over CTAs."""
    q, scale, z = weights_of(V, H, group, n % 2 == 0, V + H)
    x = torch.randn(n, H, generator=gen(n)).to(BF)
    G = scale.shape[1]
    scale[5, 0], scale[6, G - 1], scale[7, G // 2], scale[V - 1, 0] = INF, -INF, NAN, INF
    scale[8, 0], scale[8, G - 1] = INF, -INF
    if n > 1:
        x[1, 40] = INF
        x[n - 1, H - 1], x[n - 1, 0] = -INF, -INF
    if n > 4:
        x[3, 3] = NAN
    want, tol = SC.product(x, q, scale, z, group, dtype)
    assert torch.isinf(want[:, 5]).any() and torch.isfinite(want[0]).sum() == V - 5
    out, guard = guarded((n, V), dtype)
    sv.linear_w4(x.cuda(), SP.pack(q).cuda(), scale.cuda(), cuda(z), group=group, dtype=dtype, out={"logits": out})
    guard()
    SC.all_close(out.cpu().double(), want, tol)
