"""Comparisons of the calls around the vocabulary rows of a decode step with their
plain 64-bit implementations.  A tolerance holds where a finite value is expected;
infinities have to be equal, NaN to be NaN."""
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
