"""Waits of a product with 4-bit weights that do run out."""
import pytest
import torch

import serve_plain as SP
from test_gpu_serve import BF, F32, gen, sv, weights_of          # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,V,H", [(1, 500, 1024), (8, 30000, 1024), (100, 30000, 1024), (5, 700, 8192), (60, 300, 4096)])
def test_waits_of_a_product_do_run_out(sv, n, V, H):  # noqa: F811
    """A first copy takes more than a cycle, so with a limit of one some wait runs out and its logits are NaN
    (the last two sizes split their k over a cluster)."""
    q, scale, _ = weights_of(V, H, 128, False, 9)
    packed, sc, x = SP.pack(q).cuda(), scale.cuda(), torch.randn(n, H, generator=gen(2)).to(BF).cuda()
    want = sv.linear_w4(x, packed, sc, dtype=F32)["logits"]
    assert torch.isfinite(want).all()
    try:
        sv.set_wait_limit(1)
        got = sv.linear_w4(x, packed, sc, dtype=F32)["logits"]
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    late = torch.isnan(got)
    assert late.any(), "a limit of one cycle timed nothing out"
    assert (late | (got == want)).all()
    assert torch.equal(sv.linear_w4(x, packed, sc, dtype=F32)["logits"], want)
