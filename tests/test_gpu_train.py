"""The drafter-training calls on the GPU against 64-bit plain implementations.

Tolerances.  A weight 2^{(x - m) c} carries about 1e-6 for exponents that
matter (an fma's half step at |a| <= 32, c to 2^-24, ex2.approx), and a thread
adds at most a few hundred of them one after another: a sum of V terms is off
by at most 2e-5 relative, its logarithm by 2e-5 absolute (TOL).  Losses are sums
of p (ln p - ln q) with two such logarithms; gradients are held, element by
element, to 1e-4 of the sum of their terms' magnitudes, and half a step of the
output type.  The projection's logits are fp32 sums of H exact products:
(8 + sqrt H) 2^-23 of the sum of magnitudes; G is rounded to bf16 once, so
its products are off by 2^-8 of the sum of their terms' magnitudes.
"""
import math

import pytest
import torch

import train_plain as TP

pytestmark = pytest.mark.gpu

TOL = 2e-5
INF, NAN = math.inf, math.nan
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_26_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(n, V, dtype, seed, scale=3.0):
    g = gen(seed)
    bias = -1.1 * torch.log1p(torch.randperm(V, generator=g).float())
    return (torch.randn(n, V, generator=g) * scale + bias).to(dtype)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def offset(t, elems):
    """The same tensor on the GPU, `elems` elements past an aligned start."""
    buf = torch.zeros(t.numel() + elems, dtype=t.dtype, device="cuda")
    v = buf[elems:].view(t.shape)
    v.copy_(t)
    return v


# ---------------------------------------------------------------------- records

def check_record(sv, x, K, T, dev_x=None):
    r = sv.topk_logits(x.cuda() if dev_x is None else dev_x, K, None if T is None else T.cuda())
    T = torch.ones(x.shape[0]) if T is None else T
    top, idx, tail = TP.record(x, K, T)
    assert r["status"].cpu().eq(0).all()
    assert torch.equal(r["top_index"].cpu().long(), idx.long())
    assert torch.equal(r["top_logits"].cpu().double(), top)
    got = r["tail_lse"].cpu().double()
    # a weight beside the row's largest logit below 2^-126 is 0 in fp32 (e^-87.3 = 2^-126): a
    # rest whose whole mass is below that has none, and its tail is -inf
    tail = torch.where(tail - top[:, 0] / T.double() < -87.3, -INF, tail)
    fin = torch.isfinite(tail)
    assert torch.equal(torch.isfinite(got), fin) and torch.equal(got[~fin], tail[~fin])
    assert ((got - tail)[fin].abs() <= TOL + 3e-7 * tail[fin].abs()).all(), (got - tail)[fin].abs().max()
    return r


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K", [(1, 2, 1), (1, 2, 2), (3, 7, 7), (5, 100, 100), (2, 256, 256), (4, 1001, 256),
                                   (9, 4093, 33), (3, 8191, 256), (2, 65537, 1), (2, 151936, 64), (40, 20000, 5),
                                   (160, 5000, 16), (320, 5003, 8), (700, 1000, 3)])
def test_record(sv, n, V, K, dtype):
    T = torch.rand(n, generator=gen(V)) * 1.5 + 0.3
    check_record(sv, rows(n, V, dtype, n + V + K), K, T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_record_ties_and_filtered_rows(sv, dtype):
    V, K = 30011, 48
    x = rows(9, V, dtype, 5)
    x[0] = 1.5                                        # all equal
    x[1] = torch.round(x[1].float()).to(dtype)        # few values
    x[2, :20000] = 40.0                               # a tie past any candidate list
    x[3] = torch.where(x[3] < x[3].float().topk(10).values[-1], torch.tensor(-INF, dtype=dtype), x[3])
    x[4] = -INF
    x[4, V - 1] = -2.0                                # one token
    x[5, ::2] = 0.0
    x[5, 1::2] = -0.0                                 # equal zeros
    x[6] = -INF
    x[6, 1000:1000 + K] = 3.0                         # exactly K equal logits, nothing else
    x[7, V - 3:] = 50.0
    x[8] = torch.arange(V, dtype=torch.float32).to(dtype) * 0.001
    x[5] = torch.clamp(x[5].float(), max=0.0).to(dtype)
    check_record(sv, x, K, torch.linspace(0.5, 2.0, 9))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(3, 4000), (2, 70001), (350, 9000)])
def test_record_masks_of_finite_values(sv, n, V, dtype):
    """Rows masked with the type's lowest value, with zeros, or by clamping; large
    values in one period of positions; sorted rows."""
    K = 40
    x = rows(n, V, dtype, 31)
    low = torch.finfo(dtype).min
    g = gen(4)
    x[0] = torch.where(torch.rand(V, generator=g) < 20.0 / V, x[0], torch.tensor(low, dtype=dtype))
    x[1] = torch.where(torch.rand(V, generator=g) < 0.001, x[1].abs(), torch.tensor(0.0, dtype=dtype))
    if n > 2:
        x[2] = low
        x[2, V - 1] = 1.0
    if n > 8:
        x[3] = x[3].clamp(max=-2.0)
        x[4] = x[4].sort().values
        x[5] = x[5].sort(descending=True).values
        x[6] = (torch.arange(V) % 2048 < 8).to(dtype) * 9 + x[6] * 0.01
        x[7] = (torch.arange(V) % 1000 < 300).to(dtype) * 9 + x[7] * 0.1
        x[8] = -(torch.arange(V) % 3).to(dtype)
        x[9] = torch.where(torch.rand(V, generator=g) < 20.0 / V, x[9], torch.tensor(-1e9, dtype=dtype))
        x[10] = torch.where(torch.rand(V, generator=g) < 20.0 / V, x[10], torch.tensor(-1e-9, dtype=dtype))
    check_record(sv, x, K, torch.rand(n, generator=g) + 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(2, 2500003), (20, 600000)])
def test_record_of_long_rows(sv, n, V, dtype):
    """Several stages to a group, and records of the largest size."""
    check_record(sv, rows(n, V, dtype, 41), 256, torch.rand(n, generator=gen(6)) + 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K", [(4, 283111, 142), (3, 1 << 20, 64), (320, 70000, 256)])
def test_record_of_clustered_rows(sv, n, V, K, dtype):
    """The large logits in few threads' vectors, more of them than are listed: the K-th largest
    by counting, and a tail of all the others."""
    x = torch.randn(n, V, generator=gen(43))
    x[:, torch.arange(V) % 2048 < 8] += 20
    check_record(sv, x.to(dtype), K, torch.rand(n, generator=gen(7)) + 1.0)


@pytest.mark.parametrize("shift", [1, 3, 5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_record_of_rows_off_alignment(sv, dtype, shift):
    x = rows(3, 10007, dtype, 8)
    check_record(sv, x, 20, None, dev_x=offset(x, shift))


def test_record_row_errors(sv):
    x = rows(6, 3001, torch.float32, 2)
    x[0, 3000] = NAN
    x[1, 0] = INF
    x[2] = -INF
    T = torch.tensor([1.0, 1.0, 1.0, 0.0, NAN, 1.0])
    r = sv.topk_logits(x.cuda(), 9, T.cuda())
    assert r["status"].cpu().tolist() == [1, 1, 1, 64, 64, 0]
    assert (r["top_index"][:5] == -1).all() and r["top_logits"][:5].isnan().all() and r["tail_lse"][:5].isnan().all()
    ok = TP.record(x[5:], 9, T[5:])
    assert torch.equal(r["top_index"][5:].cpu().long(), ok[1])


@pytest.mark.parametrize("V,K", [(2, 1), (9, 4), (1200, 200)])
def test_record_refused_rows_among_short_ones(sv, V, K):
    """Refused rows between others, and runs of them, many to a CTA: each row gets its
    own result."""
    n = 6000
    x = rows(n, V, torch.float32, V)
    T = torch.rand(n, generator=gen(19)) + 0.5
    g = gen(20)
    bad = torch.rand(n, generator=g) < 0.5
    bad[2000:3500] = True
    hot = bad & (torch.rand(n, generator=g) < 0.5)
    x[hot, 1] = NAN
    T[bad & ~hot] = 0.0
    xd, Td = cuda(x, T)
    first = sv.topk_logits(xd, K, Td)
    good = ~bad
    top, idx, tail = TP.record(x[good], K, T[good])
    st = torch.where(hot, 1, torch.where(bad, 64, 0)).to(torch.int32)
    assert torch.equal(first["status"].cpu(), st)
    assert torch.equal(first["top_index"].cpu()[good].long(), idx)
    assert torch.equal(first["top_logits"].cpu()[good].double(), top)
    assert ((first["tail_lse"].cpu()[good].double() - tail).abs() <= TOL + 3e-7 * tail.abs()).all()
    assert (first["top_index"].cpu()[bad] == -1).all() and first["tail_lse"].cpu()[bad].isnan().all()
    for _ in range(5):
        r = sv.topk_logits(xd, K, Td)
        assert all(torch.equal(r[k][good.cuda()], first[k][good.cuda()]) for k in r)


def test_record_tail_does_not_cancel(sv):
    """Nearly all of the mass in the record: the tail keeps its precision."""
    x = torch.full((2, 5000), -30.0) + torch.rand(2, 5000, generator=gen(1))
    x[:, :4] = 20.0
    check_record(sv, x, 4, None)


# ------------------------------------------------------------------ distillation

def make_distill(n, V, K, dtype, seed, tail=True):
    g = gen(seed)
    T = torch.rand(n, generator=g) * 0.8 + 0.5
    x = rows(n, V, dtype, seed + 1)
    z = (x.float() + 1.5 * torch.randn(n, V, generator=g)).to(dtype)
    top, idx, tl = TP.record(x, K, T)
    label = torch.randint(0, V, (n,), generator=g)
    if n > 1:
        label[1] = idx[1, 0]
        label[n - 1] = -1
    w = torch.rand(n, generator=g) + 0.2
    return dict(z=z, top=top.float(), idx=idx.to(torch.int32), tail=tl.float() if tail else None,
                label=label.to(torch.int32), w=w, T=T)


def check_distill(sv, d, kl, tv, ce, grad=True, z_dev=None, out=None, ref=None, kl_finite=True):
    z = d["z"]
    loss, parts, g64, size = ref or TP.distill(z, d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"], kl, tv, ce)
    top, idx, tail, label, w, T = cuda(d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"])
    r = sv.distill_topk(z.cuda() if z_dev is None else z_dev, top, idx, tail, label=label, row_weight=w,
                        temperature=T, kl=kl, tv=tv, ce=ce, grad=grad, out=out)
    assert r["status"].cpu().eq(0).all(), r["status"]
    gl, gp = r["loss"].cpu().double(), r["parts"].cpu().double()
    if not kl_finite:                                 # of the order of 1e38: fp32 has no such logarithms
        parts, gp = parts[:, 1:], gp[:, 1:]
    tol_parts = 3 * TOL + 2e-6 * torch.where(torch.isfinite(parts), parts.abs(), 0.0)
    for a, b, t in ((gp, parts, tol_parts),
                    (gl, loss, d["w"].double().abs() * (abs(kl) + abs(tv) + abs(ce)) * 3 * TOL + 4e-6 * torch.where(
                        torch.isfinite(loss), loss.abs(), 0.0))):
        fin = torch.isfinite(b)
        assert torch.equal(torch.isfinite(a), fin) and torch.equal(a[~fin], b[~fin])
        assert ((a - b).abs() <= t)[fin].all(), (a - b)[fin].abs().max()
    if grad:
        e = (r["grad"].cpu().double() - g64).abs()
        lim = 1e-4 * size + HALF[z.dtype] * g64.abs() + 1e-37
        assert (e <= lim).all(), (e - lim).max()
    return r


@pytest.mark.parametrize("kl,tv,ce", [(1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.7, 1.0, 0.1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K,tail", [(1, 2, 1, True), (2, 9, 9, True), (5, 100, 7, False), (3, 1001, 256, True),
                                        (4, 8191, 64, True), (3, 8191, 64, False), (2, 40001, 1, True)])
def test_distill(sv, n, V, K, tail, dtype, kl, tv, ce):
    check_distill(sv, make_distill(n, V, K, dtype, n + V + K, tail), kl, tv, ce)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K", [(1, 151936, 64), (20, 50021, 16), (48, 20011, 16), (100, 7000, 16), (400, 3001, 5)])
def test_distill_batches(sv, n, V, K, dtype):
    """Few rows and many: every split of a row over CTAs."""
    d = make_distill(n, V, K, dtype, 7)
    d["w"][::7] = 0
    check_distill(sv, d, 0.7, 1.0, 0.1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V", [(2, 1 << 20), (3, (1 << 20) - 3), (6, 400001)])
def test_distill_long_rows(sv, n, V, dtype):
    """Up to the largest vocabulary: shares that do not stay in shared memory."""
    check_distill(sv, make_distill(n, V, 200, dtype, 8), 0.7, 1.0, 0.1)
    check_distill(sv, make_distill(n, V, 40, dtype, 8), 1.0, 0.0, 0.1, grad=False)


def test_distill_more_entries_than_tokens(sv):
    """K past V: the record ends with entries that are left out."""
    d = make_distill(3, 7, 7, torch.float32, 14)
    for k, v in (("idx", -1), ("top", NAN)):
        t = torch.full((3, 100), v, dtype=d[k].dtype)
        t[:, 50:57] = d[k]
        d[k] = t
    check_distill(sv, d, 1.0, 1.0, 1.0)


def test_distill_loss_alone_is_the_same(sv):
    d = make_distill(4, 5003, 20, torch.bfloat16, 3)
    a = check_distill(sv, d, 1.0, 1.0, 0.5)
    b = check_distill(sv, d, 1.0, 1.0, 0.5, grad=False)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["parts"], b["parts"]) and "grad" not in b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_in_place_and_off_alignment(sv, dtype):
    d = make_distill(3, 10007, 20, dtype, 4)
    a = check_distill(sv, d, 1.0, 1.0, 0.5)
    z = d["z"].cuda()
    b = check_distill(sv, d, 1.0, 1.0, 0.5, z_dev=z, out={"grad": z})
    assert b["grad"].data_ptr() == z.data_ptr() and torch.equal(a["grad"], b["grad"])
    for zs, gs in ((1, 1), (3, 0), (0, 5)):
        c = check_distill(sv, d, 1.0, 1.0, 0.5, z_dev=offset(d["z"], zs), out={"grad": offset(d["z"], gs)})
        # another split into vectors and single elements: other orders of the sums
        assert torch.allclose(a["loss"], c["loss"], rtol=1e-5, atol=1e-5)


def test_distill_masked_rows_and_entries(sv):
    """Weight 0: NaN rows, bad tokens and bad temperatures do not matter.  Index
    -1: the entry's logit does not matter.  -inf logits of the student."""
    d = make_distill(6, 3001, 12, torch.float32, 9)
    d["w"][2] = 0
    d["z"][2] = NAN
    d["idx"][2] = 99999
    d["T"][2] = 1.0
    d["idx"][3, 5:] = -1
    d["top"][3, 5:] = NAN
    d["z"][4, ::3] = -INF
    keep = d["idx"][4].long()
    d["z"][4, keep] = 1.0
    d["label"][4] = 1
    d["z"][4, 1] = 0.5
    zero = d["idx"][2].clone()
    ref = dict(d)
    ref["idx"] = d["idx"].clone()
    ref["idx"][2] = 0
    r64 = TP.distill(ref["z"], d["top"], ref["idx"], d["tail"], d["label"], d["w"], d["T"], 1.0, 1.0, 0.5)
    r = check_distill(sv, d, 1.0, 1.0, 0.5, ref=r64)
    assert (r["grad"][2] == 0).all() and r["loss"][2] == 0 and zero[0] == 99999


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("K", [5, 256])
def test_distill_runs_of_padded_rows(sv, K, grad):
    """Many more rows than are at work at once, and runs of padded ones among them, at
    the start too: the record of a padded row never takes the place of the next one's."""
    n, V = 2500, 601
    d = make_distill(n, V, K, torch.bfloat16, 17)
    g = gen(18)
    pad = torch.rand(n, generator=g) < 0.7
    pad[:900] = True
    pad[1400:1500] = False
    d["w"][pad] = 0
    # what a padded row holds would be a valid record for its neighbours
    d["idx"][pad] = torch.arange(K, dtype=torch.int32)
    d["top"][pad] = torch.linspace(9, -9, K)
    a = check_distill(sv, d, 0.7, 1.0, 0.1, grad=grad)
    assert (a["loss"].cpu()[pad] == 0).all() and (a["parts"].cpu()[pad] == 0).all()
    for _ in range(5):
        b = sv.distill_topk(*cuda(d["z"], d["top"], d["idx"], d["tail"]), label=d["label"].cuda(),
                            row_weight=d["w"].cuda(), temperature=d["T"].cuda(), kl=0.7, tv=1.0, ce=0.1, grad=grad)
        assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_masks_of_the_lowest_value(sv, dtype):
    """Student rows masked with the type's lowest value: runs of it before the first
    other logit, at recorded tokens, at every token but one, and everywhere."""
    low = torch.finfo(dtype).min
    d = make_distill(5, 20011, 12, dtype, 33)
    g = gen(5)
    d["z"][0, :15000] = low
    d["z"][0, d["idx"][0].long()] = 1.5
    d["z"][1] = torch.where(torch.rand(20011, generator=g) < 0.5, d["z"][1], torch.tensor(low, dtype=dtype))
    d["z"][1, d["idx"][1].long()] = 2.0
    d["z"][1, int(d["label"][1])] = 0.5
    d["z"][2] = low
    d["z"][2, d["idx"][2].long()[:1]] = 0.25
    d["z"][3] = low                                   # a uniform student
    d["T"][3] = 1.0
    d["label"][:] = d["idx"][:, 0]
    # KL with q = e^{-1e38}: far past fp32, left out of rows 2 and so of all
    check_distill(sv, d, 0.0, 1.0, 1.0, kl_finite=False)
    sub = {k: (v[3:] if v is not None else None) for k, v in d.items()}
    check_distill(sv, sub, 1.0, 1.0, 0.5)


def test_distill_infinite_losses(sv):
    """q = 0 under teacher mass: the loss is +inf, the gradient finite."""
    d = make_distill(3, 501, 6, torch.float32, 10)
    d["z"][0, int(d["idx"][0, 2])] = -INF             # KL = inf
    d["label"][1] = int(d["idx"][1, 0])
    d["z"][1, int(d["idx"][1, 0])] = -INF             # CE = inf and KL = inf
    d["z"][2] = -INF
    d["z"][2, d["idx"][2].long()] = 2.0               # q_rest = 0 < p_rest
    d["label"][2] = -1
    top, idx, tail, label, w, T = cuda(d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"])
    r = sv.distill_topk(d["z"].cuda(), top, idx, tail, label=label, row_weight=w, temperature=T, kl=1.0, tv=1.0,
                        ce=0.5, grad=True)
    assert torch.isinf(r["loss"]).all() and r["status"].eq(0).all() and torch.isfinite(r["grad"]).all()
    # the terms that are infinite are left out at coefficient 0
    r = sv.distill_topk(d["z"].cuda(), top, idx, tail, label=label, row_weight=w, temperature=T, kl=0.0, tv=1.0,
                        ce=0.0)
    assert torch.isfinite(r["loss"]).all()


def confident(n, V, K, dtype, seed, p_rest, gap, T):
    """Students whose logits outside the record lie `gap` temperatures or more below all
    inside it (gap < 0: inside below the largest outside), teachers with a mass of p_rest
    outside; temperatures of T to 2 T."""
    d = make_distill(n, V, K, dtype, seed)
    d["T"] = torch.rand(n, generator=gen(seed + 2)) * T + T
    lse = torch.logsumexp(d["top"].double() / d["T"].double()[:, None], 1)
    d["tail"] = (lse + math.log(p_rest / (1 - p_rest))).float()
    z = d["z"].float()
    inside = torch.zeros(n, V, dtype=torch.bool).scatter_(1, d["idx"].long(), True)
    top = torch.where(inside, -INF, z).max(1, keepdim=True).values
    if gap < 0:
        low = torch.where(inside, z, -INF).max(1, keepdim=True).values
    else:
        low = torch.where(inside, z, INF).min(1, keepdim=True).values
    d["z"] = torch.where(inside, z - low + top + gap * d["T"][:, None], z).to(dtype)
    return d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K", [(3, 5003, 16), (40, 20011, 200), (400, 3001, 5)])
@pytest.mark.parametrize("gap,T,p_rest", [(95, 0.2, 0.1), (300, 0.05, 0.1), (90, 1.0, 0.9), (-300, 0.05, 0.9),
                                          (-95, 0.3, 0.1), (-20000, 0.001, 0.99999)])
def test_distill_rest_far_from_the_record(sv, n, V, K, dtype, gap, T, p_rest):
    """One of the two has no weight beside the other in 32 bits (e^-87.3 = 2^-126): KL is
    finite all the same, its logarithms are."""
    check_distill(sv, confident(n, V, K, dtype, 50, p_rest, gap, T), 1.0, 0.5, 0.1, grad=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 65536.0, -65536.0, 1e-4])
@pytest.mark.parametrize("n,V,K", [(3, 5003, 16), (400, 3001, 5), (2, 600011, 30)])
@pytest.mark.parametrize("gap,p_rest", [(80, 0.2), (86, 0.2), (95, 0.2), (200, 0.9), (-200, 0.2)])
def test_distill_gradient_of_a_rest_far_from_the_record(sv, n, V, K, dtype, scale, gap, p_rest):
    """The pull towards the rest is there whatever q_rest is, and it is finite under a loss
    scale: |gradient| <= 2 (kl + tv + ce) w / T."""
    d = confident(n, V, K, dtype, 51, p_rest, gap, 0.2)
    d["w"] *= scale
    kl, tv, ce = 5.0, 0.5, 0.1
    top, idx, tail, label, w, T = cuda(d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"])
    r = sv.distill_topk(d["z"].cuda(), top, idx, tail, label=label, row_weight=w, temperature=T, kl=kl, tv=tv, ce=ce,
                        grad=True)
    loss, _, g64, size = TP.distill(d["z"], d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"], kl, tv, ce)
    assert (r["status"] == 0).all()
    lim = d["w"].double().abs() * (kl + tv + ce) * 3 * TOL + 4e-6 * loss.abs()
    assert ((r["loss"].cpu().double() - loss).abs() <= lim).all()
    # weights below 2^-126 are 0, of q beside the row's largest logit and of the teacher's share
    # beside the rest's: up to 2^-126 of the terms' coefficients, twice; and an output that is
    # itself below 2^-126 is rounded to steps of 2^-126 eps (2^-133 in bf16, 2^-149 in fp32)
    flush = (d["w"].abs() / d["T"]).double()[:, None] * 2 * (kl + tv + ce) * 2.0 ** -126 + 2.0 ** -126 * HALF[dtype]
    e = (r["grad"].cpu().double() - g64).abs()
    assert (e <= 1e-4 * size + HALF[dtype] * g64.abs() + flush).all()


def test_distill_rest_by_hand(sv):
    """V = 3, K = 1, T = 0.1, teacher (8, 0, 0), student (10, 0, 0): p_rest = 2 e^-80, q_rest =
    2 e^-100, KL = 40 e^-80 - (p_rest - q_rest) = 7e-34."""
    r = sv.distill_topk(torch.tensor([[10.0, 0.0, 0.0]], device="cuda"), torch.tensor([[8.0]], device="cuda"),
                        torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([math.log(2)], device="cuda"),
                        temperature=torch.tensor([0.1], device="cuda"))
    assert r["status"].item() == 0 and abs(r["loss"].item()) <= 1e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,V,K", [(5, 1001, 9), (3, 70001, 256), (400, 5000, 40)])
def test_low_temperatures(sv, n, V, K, dtype):
    T = torch.rand(n, generator=gen(V)) * 0.2 + 0.01
    x = rows(n, V, dtype, 53)
    top, idx, tail = TP.record(x, K, T)
    r = sv.topk_logits(x.cuda(), K, T.cuda())
    assert (r["status"] == 0).all() and torch.equal(r["top_index"].cpu().long(), idx)
    assert torch.equal(r["top_logits"].cpu().double(), top)
    # A weight below 2^-126 of the row's largest is 0: up to V of them are missing from the tail,
    # V 2^-126 of its mass beside that weight, so ln(1 - share) of the tail; half of it or more
    # may be missing near the limit, all of it below.
    got, share = r["tail_lse"].cpu().double(), V * 2.0 ** -126 / torch.exp(tail - top[:, 0] / T.double())
    lim = TOL + 3e-7 * tail.abs()
    assert (got <= tail + lim).all() and (got >= tail - lim - 2 * share)[share < 0.5].all() and (share < 1e-6).any()
    d = make_distill(n, V, K, dtype, 52)
    d["T"] = T
    d.update(top=top.float(), idx=idx.to(torch.int32), tail=tail.float())
    check_distill(sv, d, 1.0, 1.0, 0.5, grad=False)


def test_distill_row_errors(sv):
    d = make_distill(9, 701, 5, torch.float32, 11)
    d["z"][0, 700] = NAN
    d["z"][1] = -INF
    d["label"][2] = 701
    d["idx"][3, 4] = 701
    d["idx"][4, 1] = d["idx"][4, 0]                   # recorded twice
    d["T"][5] = -1
    d["idx"][6] = -1
    d["tail"][6] = -INF                               # no mass
    d["tail"][7] = NAN
    top, idx, tail, label, w, T = cuda(d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"])
    r = sv.distill_topk(d["z"].cuda(), top, idx, tail, label=label, row_weight=w, temperature=T, ce=1.0, tv=1.0,
                        grad=True)
    assert r["status"].cpu().tolist() == [1, 1, 2, 2, 2, 64, 1, 1, 0]
    assert r["loss"][:8].isnan().all() and r["parts"][:8].isnan().all() and (r["grad"][:8] == 0).all()
    sub = {k: (v[8:] if v is not None else None) for k, v in d.items()}
    a = check_distill(sv, sub, 1.0, 1.0, 1.0)
    assert torch.equal(a["loss"], r["loss"][8:]) and torch.equal(a["grad"], r["grad"][8:])


def test_distill_gradient_against_differences(sv):
    """The returned gradient against central differences of the returned losses:
    fp32 losses to ~1e-6 over steps of 0.02 leave 1e-4, the third order 1e-4."""
    d = make_distill(3, 40, 6, torch.float32, 12)
    top, idx, tail, label, w, T = cuda(d["top"], d["idx"], d["tail"], d["label"], d["w"], d["T"])
    f = lambda z, grad=False: sv.distill_topk(z, top, idx, tail, label=label, row_weight=w, temperature=T,   # noqa
                                              kl=1.0, tv=0.0, ce=0.5, grad=grad)
    z = d["z"].cuda()
    g = f(z, True)["grad"]
    for v in range(40):
        e = torch.zeros_like(z)
        e[:, v] = 0.02
        diff = (f(z + e)["loss"] - f(z - e)["loss"]) / 0.04
        assert torch.allclose(diff, g[:, v], atol=5e-4), (v, diff, g[:, v])


# ----------------------------------------------------------- linear cross entropy

def make_ce(n, H, V, seed):
    g = gen(seed)
    w = (torch.randn(V, H, generator=g) * (2.0 / math.sqrt(H))).to(torch.bfloat16)
    label = torch.randint(0, V, (n,), generator=g)
    h = torch.randn(n, H, generator=g) + torch.rand(n, 1, generator=g) * 4 * w[label].float()
    return h.to(torch.bfloat16), w, label.to(torch.int32)


def ce_tol(h, w):
    H = h.shape[1]
    h = torch.nan_to_num(h.double())
    size = (h.abs() @ w.double().abs().t()).max(1).values
    return (8 + math.sqrt(H)) * 2.0 ** -23 * size + 2 * TOL


def check_ce_forward(sv, h, w, label, **kw):
    r = sv.linear_ce_forward(*cuda(h, w, label), **kw)
    safe = h.clone()
    safe[label < 0] = 0
    loss, lse = TP.ce_forward(safe, w, label)
    tol = ce_tol(safe, w)
    assert r["status"].cpu().eq(0).all()
    for k, b in (("loss", loss), ("lse", lse)):
        e = (r[k].cpu().double() - b).abs()
        assert (e <= 2 * tol + 2e-7 * b.abs()).all(), (k, (e - tol).max())
    return r


def check_ce_grads(r, want):
    for k, b, lim in (("grad_hidden", want[0], want[2]), ("grad_weight", want[1], want[3])):
        if k in r:
            e = (r[k].cpu().double() - b).abs()
            assert (e <= lim).all(), (k, (e / lim).max())


def check_ce_backward(sv, h, w, label, g, **kw):
    hd, wd, ld = cuda(h, w, label)
    f = sv.linear_ce_forward(hd, wd, ld)
    r = sv.linear_ce_backward(hd, wd, ld, f["lse"], None if g is None else g.cuda(), **kw)
    gr = torch.ones(h.shape[0]) if g is None else g
    safe = h.clone()
    safe[(label < 0) | (gr == 0)] = 0
    delta = 4 * float(ce_tol(safe, w).max())             # the logits' and lse's
    check_ce_grads(r, TP.ce_backward(safe, w, label, gr, delta))
    return r


CE_SIZES = [(1, 8, 2), (2, 8, 300), (1, 64, 1000), (7, 72, 257), (64, 128, 513), (130, 200, 1023), (257, 64, 2000),
            (300, 264, 5000), (513, 512, 3001), (40, 1024, 777)]


@pytest.mark.parametrize("n,H,V", CE_SIZES)
def test_ce_forward(sv, n, H, V):
    check_ce_forward(sv, *make_ce(n, H, V, n + H + V))


@pytest.mark.parametrize("n,H,V", CE_SIZES)
def test_ce_backward(sv, n, H, V):
    h, w, label = make_ce(n, H, V, n + H + V)
    check_ce_backward(sv, h, w, label, torch.rand(n, generator=gen(1)) / n)


@pytest.mark.parametrize("n,H,V", [(7, 1032, 300), (70, 2048, 513), (300, 2056, 1023), (33, 2560, 777), (5, 4104, 257),
                                   (129, 8192, 300)])
def test_ce_wide_hidden_states(sv, n, H, V):
    """Sums of several parts of 1024 of H, whole and ragged ones, some rows without a label."""
    h, w, label = make_ce(n, H, V, H + V)
    label[1::5] = -1
    check_ce_forward(sv, h, w, label)
    check_ce_backward(sv, h, w, label, torch.rand(n, generator=gen(1)) / n)


@pytest.mark.parametrize("n,H,V", [(4097, 24, 600), (9001, 16, 300), (32769, 8, 300), (70003, 8, 257)])
def test_ce_many_rows(sv, n, H, V):
    """More than one group of row tiles (4096 rows), and CTAs that gather 64 rows (32768)."""
    h, w, label = make_ce(n, H, V, H + V)
    label[1::5] = -1
    label[4000:4300] = -1
    check_ce_forward(sv, h, w, label)
    check_ce_backward(sv, h, w, label, torch.rand(n, generator=gen(1)) / n)


@pytest.mark.parametrize("H", [1024, 2048, 2560])
def test_ce_small_losses(sv, H):
    """The label has nearly all of the mass: the loss ln(1 + sum e^{l_v - z}) keeps its precision.
    It is off by what l_v and z are: others of up to 5 in size, 64 additions of a part cut off by
    2^-24 of them on average, 1.9e-5, over up to 2.5 parts of which most is chance; z of up to
    24 from 64 chains joined in nearest, 3e-6; ex2 and the sums, 2e-6."""
    n, V = 64, 3001
    _, w, label = make_ce(n, H, V, 77)
    h = (torch.linspace(2.5, 5.6, n)[:, None] * w[label.long()].float()).to(torch.bfloat16)
    f = sv.linear_ce_forward(*cuda(h, w, label))
    l = h.double() @ w.double().t()
    z = l.gather(1, label.long()[:, None])
    hot = torch.zeros_like(l).scatter_(1, label.long()[:, None], 1.0)
    loss = torch.log1p((torch.exp(l - z) * (1 - hot)).sum(1))
    assert loss.min() < 1e-5 and loss.max() > 1e-2
    assert ((f["loss"].cpu().double() - loss).abs() <= 4e-5 * loss).all()


def test_ce_large_vocabulary_in_several_pieces(sv):
    """A small batch whose G does not fit one piece (checked on a few rows)."""
    n, H, V = 1024, 64, 151936
    assert sv.linear_ce_workspace_bytes(n, H, V, True) < 2 * n * V + (64 << 20)
    h, w, label = make_ce(n, H, V, 4)
    g = torch.rand(n, generator=gen(2)) / n
    hd, wd, ld, gd = cuda(h, w, label, g)
    f = sv.linear_ce_forward(hd, wd, ld)
    r = sv.linear_ce_backward(hd, wd, ld, f["lse"], gd)
    W = wd.double()
    l = hd.double() @ W.t()
    lse = torch.logsumexp(l, 1)
    assert ((f["lse"].double() - lse).abs() <= 1e-4).all()
    p = torch.exp(l - lse[:, None]) * gd.double()[:, None]
    G = p.clone()
    G[torch.arange(n, device="cuda"), ld.long()] -= gd.double()
    off = 2.0 ** -8 * G.abs() + 2e-4 * p                 # see train_plain.ce_backward
    for got, want, lim in ((r["grad_hidden"], G @ W, off @ W.abs()),
                           (r["grad_weight"], G.t() @ hd.double(), off.t() @ hd.double().abs())):
        e = (got.double() - want).abs()
        assert (e <= lim + 2.0 ** -8 * want.abs() + 1e-37).all(), (e / lim).max()


@pytest.mark.parametrize("n,H,V", [(300, 64, 700), (5, 16, 40)])
def test_ce_masked_rows(sv, n, H, V):
    """Rows without a label and of weight 0 hold NaN and infinities."""
    h, w, label = make_ce(n, H, V, 6)
    g = torch.rand(n, generator=gen(3)) + 0.1
    label[::3] = -1
    h[::3] = NAN
    check_ce_forward(sv, h, w, label)
    g[1::3] = 0
    h2 = h.clone()
    h2[1::3] = INF
    f = sv.linear_ce_forward(*cuda(h2, w, label))
    assert f["status"][1].item() == 1 and f["lse"][1].isnan() and f["loss"][0] == 0
    lse = sv.linear_ce_forward(*cuda(torch.nan_to_num(h, nan=0.0), w, label))["lse"]
    r = sv.linear_ce_backward(*cuda(h2, w, label), lse, g.cuda())
    safe = h2.clone()
    safe[::3] = 0
    safe[1::3] = 0
    check_ce_grads(r, TP.ce_backward(safe, w, label, g, 4 * float(ce_tol(safe, w).max())))
    assert (r["grad_hidden"][::3] == 0).all() and (r["grad_hidden"][1::3] == 0).all()


def test_ce_no_row_takes_part(sv):
    h, w, label = make_ce(3, 32, 100, 1)
    label[:] = -1
    f = sv.linear_ce_forward(*cuda(h, w, label))
    assert (f["loss"] == 0).all() and (f["lse"] == 0).all() and (f["status"] == 0).all()
    out = {"grad_hidden": torch.full((3, 32), 7.0, dtype=torch.bfloat16, device="cuda"),
           "grad_weight": torch.full((100, 32), 7.0, dtype=torch.bfloat16, device="cuda")}
    sv.linear_ce_backward(*cuda(h, w, label), f["lse"], out=out)
    assert (out["grad_hidden"] == 0).all() and (out["grad_weight"] == 0).all()


def test_ce_row_errors(sv):
    h, w, label = make_ce(6, 32, 100, 2)
    label[1], label[2] = 100, -2
    h[3, 5] = NAN
    f = sv.linear_ce_forward(*cuda(h, w, label))
    assert f["status"].cpu().tolist() == [0, 2, 2, 1, 0, 0]
    assert f["loss"][1:4].isnan().all() and f["lse"][1:4].isnan().all()
    r = sv.linear_ce_backward(*cuda(h, w, label), f["lse"])
    keep = torch.tensor([0, 4, 5])
    want = TP.ce_backward(h[keep], w, label[keep], torch.ones(3), 4 * float(ce_tol(h[keep], w).max()))
    check_ce_grads({"grad_weight": r["grad_weight"], "grad_hidden": r["grad_hidden"][keep.cuda()]}, want)
    assert (r["grad_hidden"][1:4] == 0).all()


@pytest.mark.parametrize("n", [1 << 15, 1 << 17, 1 << 20])
def test_ce_weight_gradient_of_many_rows(sv, n):
    """Sums of one sign over up to the most rows.  With W = 0 and V = 256, G is -255/256 at the
    label and 1/256 elsewhere, exact in bf16, so that only the sums of h and the output's
    rounding are left.  The tensor cores add 16 rows at a time and cut off less than a step of
    2^-23 of the sum so far; of a sum that grows evenly that is half of it on average, over at
    most 2048 additions in a row: 2^-13."""
    H, V = 64, 256
    g = gen(5)
    h = ((torch.rand(n, H, generator=g) + 1) * 2 ** (torch.arange(H) / H)).to(torch.bfloat16)
    hd, wd, ld = cuda(h, torch.zeros(V, H, dtype=torch.bfloat16), torch.full((n,), 3, dtype=torch.int32))
    lse = sv.linear_ce_forward(hd, wd, ld)["lse"]
    r = sv.linear_ce_backward(hd, wd, ld, lse)
    G = torch.full((V, 1), 1 / 256, dtype=torch.double)
    G[3] = -255 / 256
    want = G * h.double().sum(0)
    e = (r["grad_weight"].cpu().double() - want).abs()
    step = 2.0 ** (torch.floor(torch.log2(want.abs())) - 7)
    assert (e <= step / 2 + 2.0 ** -13 * want.abs()).all(), ((e - step / 2) / want.abs()).max()
    assert (r["grad_hidden"] == 0).all()


def test_ce_hidden_gradient_over_a_large_vocabulary(sv):
    """grad_hidden's sum over a piece joined from parts (checked on the GPU)."""
    n, H, V = 2000, 1288, 65700
    h, w, label = make_ce(n, H, V, 24)
    w = w.abs()
    g = torch.rand(n, generator=gen(10)) / n
    hd, wd, ld, gd = cuda(h * 0.1, w, label, g)
    f = sv.linear_ce_forward(hd, wd, ld)
    r = sv.linear_ce_backward(hd, wd, ld, f["lse"], gd)
    W = wd.double()
    p = torch.softmax(hd.double() @ W.t(), 1) * gd.double()[:, None]
    G = p.clone()
    G[torch.arange(n, device="cuda"), ld.long()] -= gd.double()
    off = 2.0 ** -8 * G.abs() + 2e-4 * p                 # see train_plain.ce_backward
    for got, want, lim in ((r["grad_hidden"], G @ W, off @ W.abs()),
                           (r["grad_weight"], G.t() @ hd.double(), off.t() @ hd.double().abs())):
        e = (got.double() - want).abs()
        assert (e <= lim + 2.0 ** -8 * want.abs() + 1e-37).all(), (e / lim).max()


@pytest.mark.parametrize("H,offset", [(1024, 100), (2048, 100), (2056, 100), (8192, 300), (65536, 1000)])
def test_ce_logits_that_share_an_offset(sv, H, offset):
    """Logits of one sign, all about `offset`: the backward call's match the lse that they are
    taken beside.  A column of ones in the weights makes grad_hidden the sum of a row of G, 0 by
    the formula.  G is rounded to bf16, off by 2^-8 of itself at most and not all one way, so its
    row sums to that of the rounded G of the formula, within what moves a rounding: the logits'
    own error.  At most 128 additions in a row, of sums that grow evenly, cut off 128 / 2 steps of
    2^-23 (whole sums at H <= 2048); the parts' own additions are 2^-24 offset each, in lse and
    in the logits; and ex2's 2e-6."""
    n, V = 8, 1000
    g = gen(6)
    w = (torch.rand(V, H, generator=g) * 0.2 + 0.9) * offset / H / 1.5
    w[:, 0] = 1.0
    w = w.to(torch.bfloat16)
    h = (torch.rand(n, H, generator=g) + 1).to(torch.bfloat16)
    label = torch.arange(n, dtype=torch.int32)
    hd, wd, ld = cuda(h, w, label)
    f = sv.linear_ce_forward(hd, wd, ld)
    got = sv.linear_ce_backward(hd, wd, ld, f["lse"])["grad_hidden"][:, 0].double()
    l = hd.double() @ wd.double().t()
    G = torch.softmax(l, 1)
    G[torch.arange(n), label.long()] -= 1
    rounded = G.to(torch.bfloat16).double().sum(1)
    parts = max(1, H // 1024)
    slip = (64 * 2.0 ** -23 + 2 * parts * 2.0 ** -24) * offset * 1.1 + 2e-6
    # e^slip of all weights, of which sums to 1; and a rounding that goes the other way moves a
    # weight by a step: those within slip of a border, twice slip of them, by 2^-7 at most
    assert ((got - rounded).abs() <= slip + 2 * slip + 2.0 ** -8 * rounded.abs()).all(), (got - rounded).abs().max()


def test_ce_one_gradient_alone(sv):
    h, w, label = make_ce(70, 72, 900, 3)
    g = torch.rand(70, generator=gen(5))
    both = check_ce_backward(sv, h, w, label, g)
    a = check_ce_backward(sv, h, w, label, g, need_weight=False)
    b = check_ce_backward(sv, h, w, label, g, need_hidden=False)
    assert list(a) == ["grad_hidden"] and list(b) == ["grad_weight"]
    assert torch.equal(a["grad_hidden"], both["grad_hidden"]) and torch.equal(b["grad_weight"], both["grad_weight"])
    check_ce_backward(sv, h, w, label, None)


def test_ce_gradient_over_its_hidden_states(sv):
    h, w, label = make_ce(40, 64, 500, 15)
    g = torch.rand(40, generator=gen(8))
    a = check_ce_backward(sv, h, w, label, g)
    hd, wd, ld, gd = cuda(h, w, label, g)
    lse = sv.linear_ce_forward(hd, wd, ld)["lse"]
    b = sv.linear_ce_backward(hd, wd, ld, lse, gd, out={"grad_hidden": hd})
    assert b["grad_hidden"].data_ptr() == hd.data_ptr()
    assert torch.equal(a["grad_hidden"], hd) and torch.equal(a["grad_weight"], b["grad_weight"])
    with pytest.raises(sv.SpecVerifyError):
        sv.linear_ce_backward(h.cuda(), wd, ld, lse, gd, out={"grad_weight": wd})


@pytest.mark.parametrize("V", [257, 513, 8449])
def test_ce_label_alone_in_the_last_tile(sv, V):
    """The last tile of the vocabulary holds one entry, the label."""
    h, w, label = make_ce(5, 64, V, 21)
    label[:4] = V - 1
    check_ce_forward(sv, h, w, label)
    check_ce_backward(sv, h, w, label, torch.rand(5, generator=gen(9)))


@pytest.mark.parametrize("V,lo,hi", [(1000, 0, 300), (9000, 0, 8700), (9000, 300, 9000), (9000, 0, 256),
                                     (9000, 8448, 8704)])
def test_ce_vocabulary_masked_by_minus_infinity(sv, V, lo, hi):
    """Logits of -inf over whole tiles weigh nothing; of NaN they are an error."""
    h, w, label = make_ce(4, 64, V, 22)
    h[:, 0] = 1
    keep = torch.cat([torch.arange(lo), torch.arange(hi, V)])
    at = label.long() % len(keep)
    wd = w.clone()
    wd[lo:hi, 0] = -INF
    f = sv.linear_ce_forward(*cuda(h, wd, keep[at].to(torch.int32)))
    cut = sv.linear_ce_forward(*cuda(h, w[keep], at.to(torch.int32)))
    assert (f["status"] == 0).all()
    lim = ce_tol(h, w[keep]).cuda()
    for k in ("loss", "lse"):                            # both within check_ce_forward's bound of the formula
        assert ((f[k] - cut[k]).abs() <= 4 * lim + 4e-7 * cut[k].abs()).all()
    wd[lo:hi, 0] = NAN
    f = sv.linear_ce_forward(*cuda(h, wd, keep[at].to(torch.int32)))
    assert (f["status"] == 1).all() and f["loss"].isnan().all() and f["lse"].isnan().all()


LOWEST = torch.finfo(torch.bfloat16).min


@pytest.mark.parametrize("V,lo,hi", [(1000, 0, 300), (9000, 0, 8700), (9000, 300, 9000), (9000, 0, 256),
                                     (9000, 8448, 8704), (300, 0, 128)])
def test_ce_vocabulary_masked_by_the_lowest_value(sv, V, lo, hi):
    """The same with the type's lowest value, in whole half tiles and tiles: no weight, and
    no gradient."""
    h, w, label = make_ce(4, 64, V, 22)
    h[:, 0] = 1
    keep = torch.cat([torch.arange(lo), torch.arange(hi, V)])
    at = label.long() % len(keep)
    wd = w.clone()
    wd[lo:hi, 0] = LOWEST
    y = keep[at].to(torch.int32)
    f = sv.linear_ce_forward(*cuda(h, wd, y))
    cut = sv.linear_ce_forward(*cuda(h, w[keep], at.to(torch.int32)))
    assert (f["status"] == 0).all()
    lim = ce_tol(h, w[keep]).cuda()
    for k in ("loss", "lse"):
        assert ((f[k] - cut[k]).abs() <= 4 * lim + 4e-7 * cut[k].abs()).all()
    b = sv.linear_ce_backward(*cuda(h, wd, y), f["lse"])
    c = TP.ce_backward(h, w[keep], at, torch.ones(4), 4 * float(ce_tol(h, w[keep]).max()))
    check_ce_grads({"grad_weight": b["grad_weight"][keep.cuda()]}, c)
    assert (b["grad_weight"][lo:hi] == 0).all()
    check_ce_grads({"grad_hidden": b["grad_hidden"]}, c)


def test_ce_every_logit_of_the_lowest_value(sv):
    """A uniform row so far below 0 that ln V is less than half a step of lse: the loss is ln V,
    and the gradient is the one of the lse that was given, e^{l - lse} = 1 for each token."""
    V = 700
    h, w, label = make_ce(3, 64, V, 23)
    h[:, 0] = 1
    w[:, 0] = LOWEST
    f = sv.linear_ce_forward(*cuda(h, w, label))
    assert (f["status"] == 0).all() and (f["lse"] == LOWEST).all()
    assert torch.allclose(f["loss"], torch.full((3,), math.log(V), device="cuda"), rtol=1e-5)
    b = sv.linear_ce_backward(*cuda(h, w, label), f["lse"], need_hidden=False)["grad_weight"].cpu().double()
    G = torch.ones(3, V, dtype=torch.double)
    G[torch.arange(3), label.long()] = 0
    want = G.t() @ h.double()
    assert ((b - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()


def test_ce_shared_labels(sv):
    """Every row has the same label: its weight row gathers all of them."""
    h, w, label = make_ce(200, 64, 300, 8)
    label[:] = 17
    check_ce_forward(sv, h, w, label)
    check_ce_backward(sv, h, w, label, torch.rand(200, generator=gen(6)))


def test_ce_stale_workspace(sv):
    """Nothing of the workspace's old contents reaches the results."""
    h, w, label = make_ce(300, 72, 3001, 12)
    label[::5] = -1
    g = torch.rand(300, generator=gen(7))
    ws = torch.full((sv.linear_ce_workspace_bytes(300, 72, 3001, True),), 0xFF, dtype=torch.uint8, device="cuda")
    check_ce_forward(sv, h, w, label, ws=ws)
    ws.fill_(0xFF)
    check_ce_backward(sv, h, w, label, g, ws=ws)


# ------------------------------------------------------------- calls around them

def all_calls(sv, x, z, T, label, w, h, wt, cl, gl, ws):
    """The four calls as a training step makes them."""
    r = sv.topk_logits(x, 16, T)
    d = sv.distill_topk(z, r["top_logits"], r["top_index"], r["tail_lse"], label=label, row_weight=w, temperature=T,
                        kl=1.0, tv=1.0, ce=0.1, grad=True)
    f = sv.linear_ce_forward(h, wt, cl, ws=ws[0])
    b = sv.linear_ce_backward(h, wt, cl, f["lse"], gl, ws=ws[1])
    return [r["top_logits"], r["top_index"], r["tail_lse"], d["loss"], d["parts"], d["grad"], f["loss"], f["lse"],
            b["grad_hidden"], b["grad_weight"]]


def step_inputs(seed, n=37, V=9001, H=136):
    g = gen(seed)
    x, z = rows(n, V, torch.bfloat16, seed), rows(n, V, torch.bfloat16, seed + 50)
    label = torch.randint(0, V, (n,), generator=g).to(torch.int32)
    label[3] = -1
    h, wt, cl = make_ce(n, H, V, seed)
    cl[5] = -1
    return cuda(x, z, torch.rand(n, generator=g) + 0.4, label, torch.rand(n, generator=g), h, wt, cl,
                torch.rand(n, generator=g))


def step_ws(sv, n=37, V=9001, H=136):
    return [torch.empty(sv.linear_ce_workspace_bytes(n, H, V, b), dtype=torch.uint8, device="cuda") for b in (0, 1)]


def test_waits_that_run_out(sv):
    """With the wait limit at one cycle every row is either right or void with
    SPEC_ST_TIMEOUT, and the calls return; with the default limit on the same
    workspaces every row is right again."""
    ins = step_inputs(3)
    ws = step_ws(sv)
    want = [t.clone() for t in all_calls(sv, *ins, ws)]
    x, z, T, label, w, h, wt, cl, gl = ins
    # the projection's weights are larger than what a stage or two holds: waits are real
    big = cuda(*make_ce(700, 512, 9001, 4))
    more = [rows(n, V, torch.bfloat16, 8).cuda() for n, V in ((600, 40000), (8, 151936))]      # a CTA, and clusters, a row
    rec = [sv.topk_logits(m, 16) for m in more]

    def losses():
        return [sv.distill_topk(m.flip(0), r["top_logits"], r["top_index"], r["tail_lse"], kl=1.0, tv=1.0, grad=True)
                for m, r in zip(more, rec)]
    loss = losses()
    f = sv.linear_ce_forward(*big)
    b = sv.linear_ce_backward(*big, f["lse"])
    torch.cuda.synchronize()
    sv.set_wait_limit(1)
    try:
        few = sv.topk_logits(x, 16, T)
        rec1 = [sv.topk_logits(m, 16) for m in more]
        loss1 = losses()
        f1 = sv.linear_ce_forward(*big)
        b1 = sv.linear_ce_backward(*big, f["lse"])
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    late = 0
    record_keys, loss_keys = ("top_logits", "top_index", "tail_lse"), ("loss", "parts", "grad")
    for r, full, keys in ([(few, dict(zip(record_keys, want)), record_keys), (f1, f, ("loss", "lse"))] +
                          [(a, c, record_keys) for a, c in zip(rec1, rec)] + [(a, c, loss_keys) for a, c in zip(loss1, loss)]):
        st = r["status"]
        to = st == sv._lib.ST_TIMEOUT
        late += int(to.sum())
        assert ((st == 0) | to).all()
        for k in keys:
            assert torch.equal(r[k][~to], full[k][~to]), k
            if k == "top_index":
                assert (r[k][to] == -1).all()
            elif k != "grad":
                assert r[k][to].isnan().all(), k
    for k in b:
        assert torch.equal(b1[k], b[k]) or b1[k].isnan().all(), k
    assert late > 0, "a one-cycle wait limit timed nothing out"
    for p, q in zip(want, all_calls(sv, *ins, ws)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n,H,V", [(300, 2568, 3001), (40000, 64, 1500)])
def test_waits_that_run_out_between_parts(sv, n, H, V):
    """The same for sums joined from parts: of wide hidden states, and of many rows."""
    big = cuda(*make_ce(n, H, V, 4))
    f = sv.linear_ce_forward(*big)
    b = sv.linear_ce_backward(*big, f["lse"])
    torch.cuda.synchronize()
    sv.set_wait_limit(1)
    try:
        f1 = sv.linear_ce_forward(*big)
        b1 = sv.linear_ce_backward(*big, f["lse"])
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    to = f1["status"] == sv._lib.ST_TIMEOUT
    assert ((f1["status"] == 0) | to).all()
    for k in ("loss", "lse"):
        assert torch.equal(f1[k][~to], f[k][~to]) and f1[k][to].isnan().all()
    for k in b:
        assert torch.equal(b1[k], b[k]) or b1[k].isnan().all(), k
    f2 = sv.linear_ce_forward(*big)
    b2 = sv.linear_ce_backward(*big, f2["lse"])
    assert all(torch.equal(f[k], f2[k]) for k in f) and all(torch.equal(b[k], b2[k]) for k in b)


def test_repeated_captured_and_on_two_streams(sv):
    """The same bits from a second call, from a replayed graph on new inputs, and
    from two streams at once with a workspace each."""
    A, B = step_inputs(1), step_inputs(2)
    want_a = [t.clone() for t in all_calls(sv, *A, step_ws(sv))]
    want_b = [t.clone() for t in all_calls(sv, *B, step_ws(sv))]
    for p, q in zip(want_a, all_calls(sv, *A, step_ws(sv))):
        assert torch.equal(p, q)
    torch.cuda.synchronize()
    # two streams, interleaved
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws1, ws2 = step_ws(sv), step_ws(sv)
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            got.append((want_a, all_calls(sv, *A, ws1)))
        with torch.cuda.stream(s2):
            got.append((want_b, all_calls(sv, *B, ws2)))
    torch.cuda.synchronize()
    for want, g in got:
        for p, q in zip(want, g):
            assert torch.equal(p, q)
    # a graph, replayed on other inputs
    ins = [t.clone() for t in A]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = all_calls(sv, *ins, ws1)
    for src, want in ((A, want_a), (B, want_b), (A, want_a)):
        for d, t in zip(ins, src):
            d.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, outs):
            assert torch.equal(p, q)


FIRST_CAPTURED = """
import sys
import torch
sys.path.insert(0, "tests")
import speculative_decoding_verification_26_gb300 as sv
import test_gpu_train as T
ins = T.step_inputs(1)
ws = T.step_ws(sv)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = T.all_calls(sv, *ins, ws)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
assert all(torch.equal(a, b) for a, b in zip(got, T.all_calls(sv, *ins, ws)))
print("same")
"""


def test_first_calls_of_a_process_are_captured(sv):
    """Kernels are configured on the first call that needs them, in a capture too."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURED], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_captured_call_has_its_own_workspace(sv):
    h, w, label = cuda(*make_ce(50, 64, 700, 5))
    eager = sv.linear_ce_forward(h, w, label)["loss"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sv.linear_ce_forward(h, w, label)
    other = sv.linear_ce_forward(h * 2, w, label)["loss"].clone()   # the eager workspace in between
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["loss"], eager) and not torch.equal(other, eager)


def test_threads_on_one_stream(sv):
    """Host threads that call on the default stream with its cached workspace."""
    import threading
    sets = [cuda(*make_ce(n, 72, V, 30 + n)) for n, V in ((300, 3001), (40, 9000), (5, 700))]
    want = []
    for h, w, y in sets:
        f = sv.linear_ce_forward(h, w, y)
        want.append((f["loss"], f["lse"], *sv.linear_ce_backward(h, w, y, f["lse"]).values()))
    torch.cuda.synchronize()
    got = [[] for _ in sets]

    def work(k):
        h, w, y = sets[k]
        for _ in range(60):
            f = sv.linear_ce_forward(h, w, y)
            got[k] = [f["loss"], f["lse"], *sv.linear_ce_backward(h, w, y, f["lse"]).values()]
            wrong.extend(k for a, b in zip(want[k], got[k]) if not torch.equal(a, b))

    wrong = []
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and all(got)


def test_rows_behind_the_last_stay(sv):
    """Outputs are views into larger buffers: what lies behind them stays."""
    d = make_distill(3, 1003, 6, torch.bfloat16, 21)
    buf = torch.full((5, 1003), 3.0, dtype=torch.bfloat16, device="cuda")
    check_distill(sv, d, 1.0, 1.0, 0.1, out={"grad": buf[1:4]})
    assert (buf[0] == 3).all() and (buf[4] == 3).all()
    h, w, label = make_ce(3, 64, 303, 3)
    gh = torch.full((5, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full((305, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    check_ce_backward(sv, h, w, label, torch.ones(3), out={"grad_hidden": gh[1:4], "grad_weight": gw[1:304]})
    assert (gh[0] == 3).all() and (gh[4] == 3).all() and (gw[0] == 3).all() and (gw[304] == 3).all()


def test_verified_chains_are_distilled(sv):
    """As used together: chains are verified, their target rows filtered and
    recorded, and the draft rows trained on the records; the loss's parts agree
    with the divergence statistics of the same rows, and CE on the committed
    tokens through the projection agrees with CE on its logits."""
    import numpy as np

    import parity as PT
    from speculative_decoding_verification_26_gb300 import workloads as W
    import oracle as O
    wl = PT.make_workload(O.load(), "c3", 0)
    wl_t, wl_d = PT.logits_dev(wl, "target", "cuda"), PT.logits_dev(wl, "draft", "cuda")
    B, G, V = wl_d.shape
    toks, gam, T, u = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in
                       (wl.draft_tokens, wl.gamma, wl.temperature, wl.uniforms))
    ver = sv.verify_sample(wl_t, wl_d, toks, gam, T, u)
    rows_t = wl_t[:, :G].reshape(B * G, V).contiguous()
    T_rows = T.repeat_interleave(G)
    rec = sv.topk_logits(rows_t, 256, T_rows)
    committed = ver["tokens"][:, :G].reshape(-1).contiguous()       # -1 past the drawn token
    d = sv.distill_topk(wl_d, rec["top_logits"], rec["top_index"], rec["tail_lse"], label=committed,
                        temperature=T_rows, kl=1.0, tv=1.0, ce=0.1, grad=True)
    assert (d["status"] == 0).all()
    st = sv.divergence_stats(wl_t, wl_d, gam, T)["stats"].view(-1, 5)
    # a bucket for the rest can only lower KL and TV (data processing)
    assert (d["parts"][:, 0] <= st[:, 2] * math.log(2) + 1e-4).all()
    assert (d["parts"][:, 1] <= st[:, 1] / 2 + 1e-4).all() and (d["parts"][:, 1] > 0).all()
    # with the whole row filtered to the record, the record is the row: KL, TV and 1 - A agree
    sv.filter_top_k_top_p(rows_t, torch.full((B * G,), 50, dtype=torch.int32, device="cuda"))
    rec = sv.topk_logits(rows_t, 256, T_rows)
    assert torch.isinf(rec["tail_lse"]).any()
    tf = torch.cat([rows_t.view(B, G, V), wl_t[:, G:]], 1).contiguous()
    d = sv.distill_topk(wl_d, rec["top_logits"], rec["top_index"], rec["tail_lse"], temperature=T_rows, tv=1.0)
    st = sv.divergence_stats(tf, wl_d, gam, T)["stats"].view(-1, 5)
    whole = torch.isinf(rec["tail_lse"])
    assert torch.allclose(d["parts"][whole, 0], st[whole, 2] * math.log(2), rtol=2e-5, atol=2e-5)
    assert torch.allclose(d["parts"][whole, 1], 1 - st[whole, 0], rtol=2e-5, atol=2e-5)
    assert torch.allclose(d["parts"][whole, 1], st[whole, 1] / 2, rtol=2e-5, atol=2e-5)
    # the projection: its losses are those of its logits, row by row
    h, w, _ = cuda(*make_ce(B * G, 64, V, 3))
    f = sv.linear_ce_forward(h, w, committed)
    logits = (h.double() @ w.double().t()).float()
    idx0 = torch.full((B * G, 1), -1, dtype=torch.int32, device="cuda")
    c = sv.distill_topk(logits, torch.zeros(B * G, 1, device="cuda"), idx0, torch.zeros(B * G, device="cuda"),
                        label=committed, kl=0.0, ce=1.0)
    assert torch.allclose(f["loss"], c["loss"], atol=1e-4)
