"""Comparisons of the calls around the vocabulary rows of a decode step with their
plain 64-bit implementations.  A tolerance holds where a finite value is expected;
infinities have to be equal, NaN to be NaN."""
import math

import torch

import serve_plain as SP

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def close(got, want, tol):
    """Element by element; `got` in 64 bits."""
    near = (got - want).abs() <= tol
    return torch.where(torch.isfinite(want), near & torch.isfinite(got), (got == want) | (torch.isnan(got) & torch.isnan(want)))


def all_close(got, want, tol):
    bad = ~close(got, want, tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5], got[bad][:5], want[bad][:5])


def in_type(y, dtype):
    """Finite values past the type's largest one are infinities there."""
    r = y.float().to(dtype).double()
    return torch.where(torch.isinf(r), r, y)


def adjusted(x, a, refused=()):
    """(rows, tolerances) of spec_adjust_logits: a quotient or product, a product with a sum, a
    difference and a sum, each off by half a step (2^-24) of what it is made of, and half a step of the
    type.  Requests in `refused` stay as they are, exactly."""
    y, mag = x.double().clone(), torch.zeros(x.shape, dtype=torch.double)
    sel = torch.tensor([b for b in range(x.shape[0]) if b not in refused], dtype=torch.long)
    if len(sel):
        y[sel], mag[sel], _ = SP.adjust(x[sel], **{k: v[sel] for k, v in a.items()})
    y = in_type(y, x.dtype)
    tol = 4 * 2.0 ** -24 * mag + HALF[x.dtype] * y.abs()
    if len(refused):
        tol[torch.tensor(list(refused))] = 0
    return y, tol


def product(x, q, scale, zero, group, dtype):
    """(logits, tolerances) of spec_linear_w4, by its formula: each group's sum times its scale.  Sums of
    exact products in fp32: (8 + sqrt H) 2^-23 of the magnitudes of all terms, and half a step of the type."""
    n, H = x.shape
    V = q.shape[0]
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, 1)[:, :H]
    w = q.double() - z
    want, mag = torch.zeros(n, V, dtype=torch.double), torch.zeros(n, V, dtype=torch.double)
    for g, k in enumerate(range(0, H, group)):
        h, part, s = x[:, k:k + group].double(), w[:, k:k + group], scale[:, g].double()
        # (a matrix product may leave out or reorder terms with infinities: these are summed one by one)
        sums = torch.stack([(h * part[v]).sum(1) for v in range(V)], 1) if not torch.isfinite(h).all() else h @ part.t()
        want += sums * s
        mag += (h.abs() @ part.abs().t()).nan_to_num(math.inf) * s.abs()
    want = in_type(want, dtype)
    return want, (8 + math.sqrt(H)) * 2.0 ** -23 * mag + HALF[dtype] * want.abs()


def check_adjusted(call, x, a, refused=(), lay=lambda x: x, lay_out=lambda x: x):
    """`call` (adjust_logits) out of place and in place; lay and lay_out put a copy of rows where the
    call takes them from and where it writes them."""
    want, tol = adjusted(x, a, refused)
    gamma = a.get("gamma")
    for place in ("out", "in"):
        src = lay(x)
        r = call(src, **a, out={"logits": lay_out(torch.full_like(x, 77.0))}) if place == "out" else call(src, **a)
        got = r["logits"].cpu().double()
        for b in range(x.shape[0]) if gamma is not None else ():
            behind = slice(int(gamma[b]) + 1, None)               # neither read nor written
            assert got[b, behind].eq(77.0 if place == "out" else x[b, behind].double()).all()
            got[b, behind] = want[b, behind]
        status = r["status"].cpu()
        assert [b for b in range(x.shape[0]) if int(status[b])] == sorted(refused)
        all_close(got, want, tol)
