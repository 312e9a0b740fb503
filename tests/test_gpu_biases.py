"""Biases of a token that is listed several times.

A token's biases are added in the order of their list, each sum rounded to the 24 bits
of fp32 but not bounded by its largest value, and the last one to the logit, rounded once
to fp32 and once to the type.  The same roundings are made here, so without penalties
the logits are equal, not close.  (A sum of two numbers of 24 bits in 64 bits, rounded
to 24, is the sum rounded to 24: 53 >= 2 24 + 2.)
"""
import math

import pytest
import torch

from test_gpu_serve import BF, F32, gen, sv           # noqa: F401

pytestmark = pytest.mark.gpu

INF = math.inf
BIG = 3e38                                            # two of them are past the largest fp32


def rounded(s):
    """To 24 bits, in 64; the values here are no subnormal numbers."""
    if not math.isfinite(s):
        return s
    m, e = math.frexp(s)
    return math.ldexp(round(m * (1 << 24)), e - 24)        # halves to even


def expected(x, index, value):
    """Rows with the biases alone."""
    y = x.clone()
    for b in range(x.shape[0]):
        sums = {}
        for v, a in zip(index[b].tolist(), value[b].tolist()):
            if v >= 0:
                sums[v] = rounded(sums.get(v, 0.0) + a)
        for v, s in sums.items():
            y[b, :, v] = (x[b, :, v].double() + s).float().to(x.dtype)
    return y


def check(sv, x, index, value, **more):               # noqa: F811
    want = expected(x, index, value)
    dev = dict(bias_index=index.cuda(), bias_value=value.cuda(), **more)
    for place in ("out", "in"):
        src = x.cuda()
        r = sv.adjust_logits(src, **dev, out={"logits": torch.full_like(src, 9)} if place == "out" else None)
        assert r["status"].eq(0).all()
        got = r["logits"].cpu()
        ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
        assert ok.all(), (place, (~ok).nonzero()[:5], got[~ok][:5], want[~ok][:5])
    return want


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sums_past_the_largest_value(sv, dtype):      # noqa: F811
    """Finite biases whose sum is past fp32's range: the logit is what is left of them."""
    x = torch.zeros(1, 2, 3001, dtype=dtype)
    x[:, 1] = -BIG
    index = torch.tensor([[7, 7, 2500, 2500, 2500, 40, 9, 9]]).int()
    value = torch.tensor([[BIG, BIG, BIG, BIG, -BIG, 1.0, -BIG, -BIG]])
    want = check(sv, x, index, value)
    assert want[0, 0, 7] == INF and want[0, 1, 7].isfinite() and want[0, 1, 7] > 2.9e38
    assert want[0, 0, 2500] > 2.9e38 and want[0, 1, 2500].abs() < 1e37
    assert want[0, 0, 9] == -INF and want[0, 1, 9] == -INF


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (2, 0, 1)])
def test_a_ban_beside_large_biases(sv, dtype, order):  # noqa: F811
    """-inf among biases whose other sum is past fp32's range bans the token; next to each other in the
    list, and more than 32 entries apart."""
    three = [(BIG, BIG, -INF)[k] for k in order]
    for gap in (0, 40):
        x = (torch.randn(2, 3, 5003, generator=gen(3)) * 3).to(dtype)
        n = 3 + 2 * gap
        index = (torch.arange(n) + 100).int().repeat(2, 1)
        value = torch.randn(2, n, generator=gen(4))
        for k in range(3):
            index[:, k * (gap + 1)] = 4321
            value[:, k * (gap + 1)] = three[k]
        want = check(sv, x, index, value)
        assert want[:, :, 4321].eq(-INF).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,N,few", [(5, 1, 5), (2, 3, 2), (1000, 31, 4), (1000, 33, 1000), (40001, 300, 30), (40001, 4096, 40001),
                                     (2048, 4096, 2048), (151936, 4095, 9), (30011, 4096, 3)])
def test_lists(sv, V, N, few, dtype):                  # noqa: F811
    """One entry to the most; more tokens than a CTA has threads, every token of its range, a few
    tokens over and over; padding in between."""
    B, R = 3, 2
    g = gen(V + N)
    x = (torch.randn(B, R, V, generator=g) * 3).to(dtype)
    index = torch.randint(0, few, (B, N), generator=g).int() * (V // few)
    value = torch.randn(B, N, generator=g) * 4
    pad = torch.rand(B, N, generator=g) < 0.1
    index[pad], value[pad] = -1, math.nan
    value[:, ::17] *= 1e30
    check(sv, x, index, value)


def test_lists_with_histories(sv):                    # noqa: F811
    """Biased tokens that the history or a draft names too, and the same bits again; without effect
    on the penalties: a repetition of 1 leaves what the biases give."""
    B, R, V, L, N = 4, 3, 20011, 700, 600
    g = gen(41)
    x = torch.randn(B, R, V, generator=g) * 3
    index = torch.randint(0, 500, (B, N), generator=g).int()
    value = torch.randn(B, N, generator=g)
    history = torch.randint(0, 500, (B, L), generator=g).int().cuda()
    drafts = torch.randint(0, 500, (B, R), generator=g).int().cuda()
    check(sv, x, index, value, history=history, draft_tokens=drafts)
    rep = torch.full((B,), 1.3).cuda()
    dev = dict(bias_index=index.cuda(), bias_value=value.cuda(), history=history, draft_tokens=drafts, repetition=rep)
    first = sv.adjust_logits(x.cuda(), **dev)["logits"]
    for _ in range(5):
        assert torch.equal(sv.adjust_logits(x.cuda(), **dev)["logits"], first)
