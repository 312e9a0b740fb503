"""4-bit weights, products with them, and adjusted logits on the GPU against
64-bit plain implementations.

Tolerances.  Quantising and reading back are exact.  A product with 4-bit weights
sums, for each group, exact products of bf16 and whole numbers in fp32, and the
groups' sums times their scales in fp32: as for the vocabulary projection of the
linear cross entropy, (8 + sqrt H) 2^-23 of the sum of the magnitudes of all terms,
and half a step of the output type.  An adjusted logit has a quotient or product, a
product with a sum, a difference and a sum, each off by half a step (2^-24) of what
it is made of: 4 2^-24 of the sum of those magnitudes; n biases of a token are off
by n 2^-24 of the sum of theirs; and half a step of the output type.
"""
import math

import pytest
import torch

import serve_plain as SP

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_26_gb300 as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cuda(t):
    return None if t is None else t.cuda()


def guarded(shape, dtype, elems=0):
    """A tensor `elems` elements past an aligned start with 64 bytes of 0x5A before
    and after it, and a check that those stayed."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = math.prod(shape) * size
    buf = torch.full((64 + elems * size + n + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    at = 64 + elems * size
    t = buf[at:at + n].view(dtype).view(shape)

    def check():
        assert buf[:at].eq(0x5A).all() and buf[at + n:].eq(0x5A).all()
    return t, check


# ---------------------------------------------------------------------- weights

def check_quantize(sv, w, group, zero):
    q, scale, z = SP.quantize(w, group, zero)
    V, H = w.shape
    G = -(-H // group)
    out, checks = {}, []
    for k, shape, dt in (("packed", (V, H // 2), torch.uint8), ("scale", (V, G), BF), ("zero", (V, G), torch.uint8)):
        out[k], c = guarded(shape, dt)
        checks.append(c)
    r = sv.quantize_w4(w.cuda(), group, zero=zero, out=out)
    for c in checks:
        c()
    got = r["scale"].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(scale))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(scale.float()))
    if zero:
        assert torch.equal(r["zero"].cpu(), z)
    assert torch.equal(SP.unpack(r["packed"].cpu()), q)
    odd = torch.isnan(scale).any(1)
    assert torch.equal(r["status"].cpu(), odd.int() * 1)
    for dt in (BF, F32):
        o, c = guarded((V, H), dt)
        back = sv.dequantize_w4(r["packed"], r["scale"], r.get("zero"), group=group, out={"weight": o}, dtype=dt)["weight"]
        c()
        want = SP.weights(q, scale, z if zero else None, group).to(dt)
        fine = ~torch.isnan(want)
        assert torch.equal(torch.isnan(back.cpu()), ~fine) and torch.equal(back.cpu()[fine], want[fine])


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("V,H", [(1, 32), (3, 96), (17, 160), (200, 1184), (5, 2048), (1300, 288)])
def test_quantize(sv, V, H, group, dtype, zero):
    g = gen(V + H + group)
    w = torch.randn(V, H, generator=g) * torch.exp(torch.randn(V, 1, generator=g) * 3)
    w[torch.randint(0, V, (V,), generator=g), torch.randint(0, H, (V,), generator=g)] *= 8
    check_quantize(sv, w.to(dtype), group, zero)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_at_the_edges(sv, dtype, zero):
    """Ties, groups of one sign, of zeros, of the smallest and the largest values,
    NaN and infinities."""
    H, g = 256, gen(7)
    w = torch.randn(16, H, generator=g)
    w[0] = 0
    w[1, :128] = (torch.arange(128) % 29 - 14).float() / 2                  # halves of s = 1
    w[1, 128:] = (torch.arange(128) % 31).float() / 2
    w[2] = w[2].abs()
    w[3] = -w[3].abs()
    w[4] *= 1e-41
    w[5] *= 1e-37
    w[6] = torch.where(w[6] > 0, 3e38, -3e38)
    w[7, 5], w[8, 200], w[9, 130] = NAN, INF, -INF
    w[10] = 1e-45
    w[11] = 0.1
    w[12, 0], w[12, 1] = 1e30, -1e-30
    w[13] = torch.where(torch.arange(H) == 40, 5.0, 0.0)
    w[14] *= 1e-33
    w[15] = torch.linspace(-1, 1, H) * 7
    for group in (32, 128):
        check_quantize(sv, w.to(dtype), group, zero)


@pytest.mark.parametrize("zero", [False, True])
def test_quantize_large_and_offset(sv, zero):
    """Several rows a warp, and weights that start on an odd 16-byte boundary."""
    for dtype, V, H, group in ((BF, 20000, 160, 64), (F32, 12000, 96, 32), (F32, 12000, 288, 128), (BF, 10001, 544, 128)):
        w = (torch.randn(V, H, generator=gen(V)) * torch.rand(V, 1, generator=gen(H))).to(dtype)
        w[5], w[V - 1, 3], w[7] = 0, INF, w[7] * 1e-38
        buf = torch.zeros(w.numel() + 16, dtype=dtype, device="cuda")
        off = 16 // dtype.itemsize
        dev = buf[off:off + w.numel()].view(V, H)
        dev.copy_(w)
        assert dev.data_ptr() % 32 == 16
        q, scale, z = SP.quantize(w, group, zero)
        r = sv.quantize_w4(dev, group, zero=zero)
        assert torch.equal(SP.unpack(r["packed"].cpu()), q)
        assert torch.equal(r["scale"].cpu().view(torch.int16).bitwise_and(0x7FC0) == 0x7FC0, torch.isnan(scale))
        assert torch.equal(torch.nan_to_num(r["scale"].cpu().float()), torch.nan_to_num(scale.float()))
        assert not zero or torch.equal(r["zero"].cpu(), z)
        assert r["status"].cpu().nonzero().flatten().tolist() == [V - 1]


def weights_of(V, H, group, zero, seed):
    g = gen(seed)
    q = torch.randint(0, 16, (V, H), generator=g)
    G = -(-H // group)
    scale = ((torch.rand(V, G, generator=g) + 0.25) / math.sqrt(H)).to(BF)
    z = torch.randint(0, 16, (V, G), generator=g, dtype=torch.uint8) if zero else None
    return q, scale, z


def check_linear(sv, n, V, H, group, zero, dtype, seed=0, shape=None, special=None):
    q, scale, z = weights_of(V, H, group, zero, seed + V + H)
    x = torch.randn(n, H, generator=gen(seed + n)).to(BF)
    if special:
        special(x, scale)
    w = SP.weights(q, scale, z, group)
    want = x.double() @ w.t()
    mag = x.double().abs() @ w.abs().t()
    out, guard = guarded((n, V), dtype)
    r = sv.linear_w4(x.cuda(), SP.pack(q).cuda(), scale.cuda(), cuda(z), group=group, dtype=dtype, out={"logits": out})
    guard()
    got = r["logits"].cpu().double()
    tol = (8 + math.sqrt(H)) * 2.0 ** -23 * mag + HALF[dtype] * want.abs()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    bad = ((got - want).abs() > tol) & ~nan & (got != want)
    assert not bad.any(), (bad.sum(), bad.nonzero()[:5], got[bad][:5], want[bad][:5])
    return got


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 128, 129, 300])
def test_linear_rows(sv, n):
    check_linear(sv, n, 1000, 544, 128, False, BF)
    check_linear(sv, n, 300, 1184, 32, True, F32)


@pytest.mark.parametrize("n", [1, 9, 40, 130])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("V,H", [(1, 32), (3, 64), (127, 96), (128, 128), (129, 160), (257, 256), (1001, 288),
                                 (4099, 992), (64, 4096), (2048, 2048), (20000, 512)])
def test_linear_sizes(sv, V, H, group, n):
    check_linear(sv, n, V, H, group, (V + n) % 2 == 0, F32 if V % 2 else BF)


@pytest.mark.parametrize("n,V,H,group", [(1, 151936, 2048, 128), (8, 151936, 2048, 64), (3, 40001, 8192, 32),
                                         (64, 50000, 1024, 128), (200, 33000, 640, 64)])
def test_linear_large(sv, n, V, H, group):
    check_linear(sv, n, V, H, group, n == 3, F32)


@pytest.mark.parametrize("n", [1, 20, 64, 65, 200])
@pytest.mark.parametrize("V,H", [(130, 4096), (2500, 4352), (5000, 8192), (19000, 4160), (25000, 2080)])
def test_linear_split(sv, V, H, n):
    """Tiles whose k is split over two or four CTAs, or not, with a ragged end."""
    check_linear(sv, n, V, H, (32, 64, 128)[n % 3], V % 2 == 0, F32)


@pytest.mark.parametrize("n", [3, 70])
def test_linear_odd_starts(sv, n):
    """Outputs and scales off their vector boundaries, odd vocabularies."""
    H, group = 512, 64
    for V in (1001, 1002):
        q, scale, z = weights_of(V, H, group, True, 3)
        x = torch.randn(n, H, generator=gen(n)).to(BF)
        sbuf = torch.zeros(scale.numel() + 1, dtype=BF, device="cuda")
        sc = sbuf[1:].view(scale.shape)
        sc.copy_(scale)
        want = sv.linear_w4(x.cuda(), SP.pack(q).cuda(), scale.cuda(), z.cuda(), group=group)["logits"]
        for elems in (1, 2, 3):
            out, guard = guarded((n, V), BF, elems)
            sv.linear_w4(x.cuda(), SP.pack(q).cuda(), sc, z.cuda(), group=group, out={"logits": out})
            guard()
            assert torch.equal(out, want)


def test_linear_long_rows(sv):
    check_linear(sv, 2, 40, 65536, 128, True, F32)
    check_linear(sv, 70, 5, 32768, 32, False, F32)


@pytest.mark.parametrize("n", [4, 24, 100])
def test_linear_nonfinite(sv, n):
    """A NaN or infinity reaches its own row or column."""
    def special(x, scale):
        x[1, 3], x[2, 40] = NAN, INF
        scale[7, 0] = NAN
    q_ok = check_linear(sv, n, 500, 160, 32, False, F32, special=special)
    assert torch.isnan(q_ok[1]).all() and torch.isnan(q_ok[:, 7]).all()


def test_linear_shapes_streams_and_graphs(sv):
    """[B, R, H] hidden states, a stream of one's own, the same bits again, and a
    captured call whose inputs change between replays."""
    V, H = 3000, 512
    q, scale, _ = weights_of(V, H, 128, False, 5)
    packed, sc = SP.pack(q).cuda(), scale.cuda()
    x = torch.randn(3, 5, H, generator=gen(2)).to(BF).cuda()
    a = sv.linear_w4(x, packed, sc)["logits"]
    assert a.shape == (3, 5, V) and a.dtype == BF
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = sv.linear_w4(x, packed, sc)["logits"]
    s.synchronize()
    assert torch.equal(a, b)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = sv.linear_w4(xs, packed, sc, dtype=F32)["logits"]
    for k in range(3):
        xs.copy_(x * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, sv.linear_w4(x * (k + 1), packed, sc, dtype=F32)["logits"])


def test_linear_offsets_past_32_bits(sv):
    """More than 2^31 logits, and more than 2^31 bytes of weights."""
    n, V, H = 33, 70_000_001, 64
    packed = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device="cuda")
    scale = torch.rand(V, 2, device="cuda").to(BF)
    x = torch.randn(n, H, generator=gen(3)).to(BF)
    y = sv.linear_w4(x.cuda(), packed, scale, group=32)["logits"]
    at = torch.cat([torch.arange(64), torch.randint(0, V, (2000,), generator=gen(4)), torch.arange(V - 64, V)])
    w = SP.weights(SP.unpack(packed[at.cuda()].cpu()), scale[at.cuda()].cpu(), None, 32)
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    got = y[:, at.cuda()].cpu().double()
    assert ((got - want).abs() <= 16 * 2.0 ** -23 * mag + HALF[BF] * want.abs()).all()


@pytest.mark.parametrize("n,V,H", [(1, 500, 1024), (8, 30000, 1024), (100, 30000, 1024), (5, 700, 8192), (60, 300, 4096)])
def test_linear_waits_that_run_out(sv, n, V, H):
    """With a limit of one cycle a call ends, and a logit is right or NaN; the next call is right
    (the last two split their k over a cluster)."""
    q, scale, _ = weights_of(V, H, 128, False, 9)
    packed, sc, x = SP.pack(q).cuda(), scale.cuda(), torch.randn(n, H, generator=gen(2)).to(BF).cuda()
    want = sv.linear_w4(x, packed, sc, dtype=F32)["logits"]
    try:
        sv.set_wait_limit(1)
        got = sv.linear_w4(x, packed, sc, dtype=F32)["logits"]
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(0)
    assert (torch.isnan(got) | (got == want)).all()
    assert torch.equal(sv.linear_w4(x, packed, sc, dtype=F32)["logits"], want)


# ---------------------------------------------------------------- adjusted logits

def request(B, R, V, L, seed, D=None, biases=0, allowed=None, dtype=BF, few=None):
    """Rows and everything that can be given with them; tokens of `few` values."""
    g = gen(seed)
    few = few or V
    D = R if D is None else D
    tok = lambda *s: (torch.rand(*s, generator=g) ** 3 * few).long().clamp(max=V - 1).int()   # noqa: E731
    n = torch.randint(0, L + 1, (B,), generator=g).int()
    a = dict(history=tok(B, L), history_len=n, prompt_len=(n * torch.rand(B, generator=g)).int(),
             repetition=torch.rand(B, generator=g) + 0.5, frequency=torch.randn(B, generator=g),
             presence=torch.randn(B, generator=g))
    if D:
        a.update(draft_tokens=tok(B, D), gamma=torch.randint(0, D + 1, (B,), generator=g).int())
    if biases:
        a.update(bias_index=tok(B, biases) - 1, bias_value=torch.randn(B, biases, generator=g) * 4)
    if allowed is not None:
        W = -(-V // 32)
        keep = torch.rand(B, R, W, 32, generator=g) < allowed
        word = (keep.long() << torch.arange(32)).sum(3)
        a["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
    x = (torch.randn(B, R, V, generator=g) * 3).to(dtype)
    return x, a


def check_adjust(sv, x, a, status=None, in_elems=0, out_elems=0):
    """Out of place and in place against the definition."""
    B, R, V = x.shape
    ok = [b for b in range(B) if status is None or status[b] == 0]
    y, mag, touched = x.double().clone(), torch.zeros(B, R, V, dtype=torch.double), torch.zeros(B, R, V, dtype=torch.bool)
    sel = torch.tensor(ok)
    if ok:
        y[sel], mag[sel], touched[sel] = SP.adjust(x[sel], **{k: v[sel] for k, v in a.items()})
    dev = {k: v.cuda() for k, v in a.items()}
    # what lies past the type's largest value rounds to an infinity: finfo(bf16).min * 1.14
    # is -3.88e38, below -(2 - 2^-8) 2^127, where rounding to nearest leaves the finite values
    y = torch.where(torch.isinf(y.float().to(x.dtype)), y.float().to(x.dtype).double(), y)
    tol = 4 * 2.0 ** -24 * mag + HALF[x.dtype] * y.abs()
    behind = torch.zeros(B, R, dtype=torch.bool)
    if "gamma" in a:
        for b in ok:
            behind[b, int(a["gamma"][b]) + 1:] = True
    for place in ("out", "in"):
        src, g0 = guarded(x.shape, x.dtype, in_elems)
        src.copy_(x)
        if place == "out":
            dst, g1 = guarded(x.shape, x.dtype, out_elems)
            dst.fill_(77.0)
            r = sv.adjust_logits(src, **dev, out={"logits": dst})
            assert torch.equal(src.cpu().view(torch.uint8), x.view(torch.uint8))
            g1()
        else:
            r = sv.adjust_logits(src, **dev)
            assert r["logits"] is src
        g0()
        got = r["logits"].cpu()
        st = r["status"].cpu().tolist()
        assert st == (status if status is not None else [0] * B), st
        if place == "out":
            assert got[behind].eq(77.0).all()
            got[behind] = x[behind]
        same = got.view(torch.int16 if x.dtype == BF else torch.int32).eq(x.view(torch.int16 if x.dtype == BF else torch.int32))
        assert (same | touched).all()
        z = got.double()
        close = ((z - y).abs() <= tol) | (z == y) | (torch.isnan(z) & torch.isnan(y))
        assert close.all(), (place, (~close).nonzero()[:5], z[~close][:5], y[~close][:5])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,R,V,L", [(1, 1, 2, 1), (2, 3, 7, 5), (1, 8, 1000, 100), (3, 2, 4096, 40), (2, 4, 4097, 300),
                                     (2, 9, 10007, 1000), (5, 1, 33003, 64), (1, 32, 9000, 700), (70, 2, 5000, 20),
                                     (3, 3, 151936, 500)])
def test_adjust(sv, B, R, V, L, dtype):
    x, a = request(B, R, V, L, V + L, D=min(32, R), biases=9, allowed=0.7, dtype=dtype)
    check_adjust(sv, x, a)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("keep", [("history", "history_len", "prompt_len", "repetition"), ("history", "frequency"),
                                  ("history", "presence"), ("draft_tokens", "presence", "frequency"),
                                  ("draft_tokens", "gamma", "repetition"), ("bias_index", "bias_value"), ("mask",),
                                  ("history", "history_len", "repetition", "mask"), ()])
def test_adjust_parts(sv, keep, dtype):
    """Each kind alone: what is not given has no effect."""
    x, a = request(3, 4, 6001, 200, 11, biases=40, allowed=0.5, dtype=dtype)
    check_adjust(sv, x, {k: v for k, v in a.items() if k in keep})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("in_elems,out_elems", [(0, 0), (1, 1), (3, 3), (0, 1), (5, 2)])
def test_adjust_alignment(sv, in_elems, out_elems, dtype):
    for V in (4100, 8200, 5003):
        x, a = request(2, 3, V, 300, 13, biases=12, allowed=0.8, dtype=dtype)
        check_adjust(sv, x, a, in_elems=in_elems, out_elems=out_elems)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_adjust_few_tokens_many_times(sv, dtype):
    """Histories of a handful of tokens, drafts that repeat them, one bias listed many times."""
    x, a = request(3, 6, 9001, 5000, 17, biases=200, dtype=dtype, few=12)
    check_adjust(sv, x, a)
    a["bias_index"][:] = 5
    check_adjust(sv, x, a)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 8192, 40000])
def test_adjust_masks(sv, V, dtype):
    """Rows without an allowed token, with one, with all; NaN and infinities in places that a mask removes, or not."""
    B, R = 2, 5
    x, a = request(B, R, V, 50, 19, biases=20, allowed=0.5, dtype=dtype)
    a["mask"][:, 0] = 0
    a["mask"][:, 1] = 0
    a["mask"][:, 1, (V - 1) // 32] = torch.tensor(1 << ((V - 1) % 32)).to(torch.int32) if (V - 1) % 32 < 31 else -(1 << 31)
    a["mask"][:, 2] = -1
    a["mask"][:, 3, ::2] = 0
    x[:, :, 3], x[:, :, 64], x[:, :, 50], x[:, :, V - 2] = NAN, INF, -INF, torch.finfo(dtype).min
    a["history"][:, :3] = torch.tensor([3, 64, 50])
    a["history_len"][:] = 50
    for gamma in (None, a["gamma"]):
        b = {k: v for k, v in a.items() if k != "gamma"}
        if gamma is not None:
            b["gamma"] = gamma
        check_adjust(sv, x, b)


def test_adjust_bans(sv):
    """Biases of -inf, and padding tokens of -1 in every list."""
    x, a = request(2, 3, 3001, 60, 23, biases=30)
    a["bias_value"][:, ::3] = -INF
    a["bias_index"][:, 5:9] = -1
    a["bias_value"][:, 5:9] = NAN
    a["history"][:, ::4] = -1
    a["draft_tokens"][:, 1] = -1
    check_adjust(sv, x, a)


def test_adjust_refused_requests(sv):
    """A request with a bad argument is left as it is, and says why; the others are not."""
    B = 12
    x, a = request(B, 3, 9001, 40, 29, biases=6, allowed=0.6)
    a["history_len"][:] = 40
    a["prompt_len"][:] = 7
    a["gamma"][:] = 2
    a["history"][0, 11] = 9001
    a["history"][1, 39] = -2
    a["draft_tokens"][2, 1] = 9001
    a["bias_index"][3, 5] = -7
    a["history_len"][4] = 41
    a["prompt_len"][5] = 41
    a["gamma"][6] = 4
    a["repetition"][7] = 0
    a["frequency"][8] = NAN
    a["bias_value"][9, 2], a["bias_index"][9, 2] = INF, 4
    a["presence"][10], a["draft_tokens"][10, 0] = -INF, -9
    a["draft_tokens"][11, 2] = 123456                   # behind gamma: not looked at
    st = [2, 2, 2, 2, 512, 512, 4, 256, 256, 256, 258, 0]
    check_adjust(sv, x, a, status=st)


def test_adjust_streams_graphs_and_repeats(sv):
    x, a = request(4, 5, 30011, 400, 31, biases=16, allowed=0.9)
    dev = {k: v.cuda() for k, v in a.items()}
    src = x.cuda()
    first = sv.adjust_logits(src, **dev, out={"logits": torch.zeros_like(src)})["logits"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = sv.adjust_logits(src, **dev, out={"logits": torch.zeros_like(src)})["logits"]
    s.synchronize()
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    buf, out = src.clone(), torch.zeros_like(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.adjust_logits(buf, **dev, out={"logits": out})
    for k in range(2):
        buf.copy_(src * (k + 1))
        dev["history"].copy_(a["history"].roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        want = sv.adjust_logits((src * (k + 1)).contiguous(), **dev, out={"logits": torch.zeros_like(src)})["logits"]
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_adjust_offsets_past_32_bits(sv):
    """More than 2^32 bytes of logits, and a long history."""
    B, R, V, L = 18, 1, 1 << 27, 3000
    x = torch.zeros(B, R, V, dtype=BF, device="cuda")
    history = torch.randint(0, V, (B, L), generator=gen(1)).int()
    history[:, -1] = V - 1
    sv.adjust_logits(x, history.cuda(), presence=torch.ones(B, device="cuda"))
    for b in (0, 8, 16, 17):
        at = history[b].long().unique()
        assert x[b, 0, at.cuda()].eq(-1).all()
        assert int((x[b] != 0).sum()) == at.numel()


# ------------------------------------------------------------------- together

def test_a_decode_step(sv):
    """As they are used: the target's rows from 4-bit weights, adjusted for each candidate
    prefix, filtered, verified; the same step from the rows in 64 bits."""
    B, G, H, V = 6, 4, 256, 5003
    g = gen(37)
    target_w = torch.randn(V, H, generator=g)
    draft_w = target_w + 0.3 * torch.randn(V, H, generator=g)
    hidden = (torch.randn(B, G + 1, H, generator=g) * 0.25).to(BF)
    history = torch.randint(0, V, (B, 50), generator=g).int()
    T = torch.full((B,), 0.8).cuda()
    pen = dict(repetition=torch.full((B,), 1.2).cuda(), frequency=torch.full((B,), 0.1).cuda(),
               presence=torch.full((B,), 0.2).cuda())
    W = -(-V // 32)
    allowed = torch.rand(B, G + 1, W * 32, generator=g) < 0.8
    word = (allowed.view(B, G + 1, W, 32).long() << torch.arange(32)).sum(3)
    mask = torch.where(word >= 1 << 31, word - (1 << 32), word).int().cuda()
    rows = {}
    for name, w in (("target", target_w), ("draft", draft_w)):
        w4 = sv.quantize_w4(w.cuda(), 64, zero=True)
        assert w4["status"].eq(0).all()
        rows[name] = sv.linear_w4(hidden.cuda(), w4["packed"], w4["scale"], w4["zero"], group=64, dtype=F32)["logits"]
        back = sv.dequantize_w4(w4["packed"], w4["scale"], w4["zero"], group=64, dtype=F32)["weight"].cpu().double()
        want = hidden.double() @ back.t()
        mag = hidden.double().abs() @ back.abs().t()
        assert ((rows[name].cpu().double() - want).abs() <= (8 + 16) * 2.0 ** -23 * mag).all()
    # the drafter's chain: row i adjusted for the tokens drafted so far
    drafted = torch.full((B, G), -1, dtype=torch.int32, device="cuda")
    q = torch.empty(B, G, V, device="cuda")
    for i in range(G):
        row = rows["draft"][:, i:i + 1].contiguous()
        both = torch.cat([history.cuda(), drafted[:, :i]], 1).contiguous()
        sv.adjust_logits(row, both, **pen, mask=mask[:, i:i + 1].contiguous())
        q[:, i] = row[:, 0]
        drafted[:, i] = row[:, 0].argmax(1).int()
    # the same rows at once, each with its own prefix
    whole = sv.adjust_logits(rows["draft"][:, :G].contiguous(), history.cuda(), draft_tokens=drafted, **pen,
                             mask=mask[:, :G].contiguous())["logits"]
    assert torch.equal(whole, q)
    p = sv.adjust_logits(rows["target"], history.cuda(), draft_tokens=drafted, **pen, mask=mask)
    assert p["status"].eq(0).all()
    p = p["logits"]
    n = p.shape[0] * p.shape[1]
    sv.filter_top_k_top_p(p, top_k=torch.full((n,), 50, dtype=torch.int32).cuda())
    sv.filter_top_k_top_p(q, top_k=torch.full((B * G,), 50, dtype=torch.int32).cuda())
    u = torch.rand(B, G + 1, generator=g).cuda()
    r = sv.verify_sample(p, q, drafted, None, T, u)
    assert (r["status"] & ~16).eq(0).all()
    for b in range(B):
        k = int(r["accept_len"][b])
        tokens = r["tokens"][b].cpu().tolist()
        assert tokens[:k] == drafted[b, :k].cpu().tolist()
        for i, v in enumerate(tokens[:k + 1]):
            assert allowed[b, i, v]                       # the mask holds whatever was drawn
            pr = torch.softmax(p[b, i].cpu().double() / 0.8, 0)
            assert pr[v] > 0
            if i < k:
                qr = torch.softmax(q[b, i].cpu().double() / 0.8, 0)
                assert float(u[b, i]) * qr[v] < pr[v] * (1 + 1e-5)


# --------------------------------------------------------- calls beside one another

@pytest.mark.parametrize("n", [1, 5, 17, 33, 65, 130])
def test_linear_after_a_call_that_leaves_nan(sv, n):
    """Rows that a call does not have reach nothing, whatever the tile holds for them."""
    V, H = 3000, 512
    q, scale, _ = weights_of(V, H, 128, False, 6)
    packed, sc, x = SP.pack(q).cuda(), scale.cuda(), torch.randn(n, H, generator=gen(n)).to(BF).cuda()
    want = sv.linear_w4(x, packed, sc)["logits"]
    assert torch.isfinite(want).all()
    poison = torch.full((512, H), NAN, dtype=BF, device="cuda")
    for rows in (512, 64, 32, 16):
        assert torch.isnan(sv.linear_w4(poison[:rows], packed, sc)["logits"]).all()
        assert torch.equal(sv.linear_w4(x, packed, sc)["logits"], want)


def test_host_threads(sv):
    """Threads with a stream each, at once: the results of the same calls one after another."""
    import threading
    V, H, B, R = 5000, 512, 4, 5
    work = []
    for k in range(4):
        w = torch.randn(V, H, generator=gen(60 + k)).to(BF).cuda()
        x = torch.randn(B, R, H, generator=gen(70 + k)).to(BF).cuda()
        _, a = request(B, R, V, 300, 80 + k, biases=8, allowed=0.9)
        work.append((w, x, {n: v.cuda() for n, v in a.items()}))

    def step(w, x, a):
        w4 = sv.quantize_w4(w, 64, zero=True)
        rows = sv.linear_w4(x, w4["packed"], w4["scale"], w4["zero"], group=64)["logits"]
        return sv.adjust_logits(rows, **a)["logits"]
    want = [step(*w) for w in work]
    torch.cuda.synchronize()
    got, streams = [[] for _ in work], [torch.cuda.Stream() for _ in work]

    def run(k):
        with torch.cuda.stream(streams[k]):
            for _ in range(8):
                got[k].append(step(*work[k]))
            streams[k].synchronize()
    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k, w in enumerate(want):
        assert len(got[k]) == 8 and all(torch.equal(g.view(torch.int16), w.view(torch.int16)) for g in got[k])


def test_quantize_offsets_past_32_bits(sv):
    """More than 2^32 weights."""
    V, H, group = 70_000_001, 64, 32
    w = torch.randn(V, H, dtype=BF, device="cuda")
    r = sv.quantize_w4(w, group, zero=True)
    back = sv.dequantize_w4(r["packed"], r["scale"], r["zero"], group=group)["weight"]
    at = torch.cat([torch.arange(40), torch.randint(0, V, (2000,), generator=gen(8)), torch.arange(V - 40, V)])
    q, scale, z = SP.quantize(w[at.cuda()].cpu(), group, True)
    assert torch.equal(SP.unpack(r["packed"][at.cuda()].cpu()), q)
    assert torch.equal(r["scale"][at.cuda()].cpu(), scale) and torch.equal(r["zero"][at.cuda()].cpu(), z)
    assert torch.equal(back[at.cuda()].cpu(), SP.weights(q, scale, z, group).to(BF))
    assert r["status"].eq(0).all()


FIRST_CAPTURED = """
import torch
import speculative_decoding_verification_26_gb300 as sv
g = torch.Generator().manual_seed(3)
w = torch.randn(3000, 512, generator=g).bfloat16().cuda()
x = torch.randn(2, 3, 512, generator=g).bfloat16().cuda()
history = torch.randint(0, 3000, (2, 40), generator=g).int().cuda()
rep = torch.full((2,), 1.5).cuda()
def step():
    w4 = sv.quantize_w4(w, 64, zero=True)
    rows = sv.linear_w4(x, w4["packed"], w4["scale"], w4["zero"], group=64)["logits"]
    back = sv.dequantize_w4(w4["packed"], w4["scale"], w4["zero"], group=64)["weight"]
    return back, sv.adjust_logits(rows, history, repetition=rep)["logits"]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
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
