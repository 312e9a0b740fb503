"""The drafter-training operators: what is measured, and their plain forms.

Three operators on vocabulary rows:
  record   the K largest logits of a teacher row with the log mass of the rest
           (topk_logits);
  distill  the loss of a student row against such a record, KL + TV + CE, with
           or without the gradient by the student's logits (distill_topk);
  ce       the cross entropy of a vocabulary projection, hidden states times
           weight rows, without keeping the logits: "fwd" the losses, "bwd" the
           gradients by the hidden states and the weights (linear_ce_*).

`run` computes the plain form in 32 bits with elementary torch operations, or,
where `own` is true, makes the library's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request's gamma + 1 = 8 target rows, as a serving engine records them step by step
        {"name": "record one step", "op": "record", "n": 8, "V": 151936, "K": 64, "dtype": "bf16", "kept": 0},
        # the target rows of 64 requests at gamma = 7 (the verification workload), K = 64
        {"name": "record batch", "op": "record", "n": 512, "V": 151936, "K": 64, "dtype": "bf16", "kept": 0},
        # odd rows in fp32, the largest record, every fourth row filtered to 50 logits beforehand
        {"name": "record f32 ragged", "op": "record", "n": 333, "V": 100003, "K": 256, "dtype": "f32", "kept": 50},
        # the loss alone (evaluation) of one request's 7 draft rows
        {"name": "distill loss one chain", "op": "distill", "grad": False, "n": 7, "V": 151936, "K": 16,
         "dtype": "bf16", "tail": True, "kl": 1.0, "tv": 0.0, "ce": 0.0},
        # the loss alone of a batch, the stable mix of CE and TV
        {"name": "distill loss batch", "op": "distill", "grad": False, "n": 2048, "V": 128256, "K": 64,
         "dtype": "bf16", "tail": True, "kl": 0.0, "tv": 1.0, "ce": 0.1},
        # a training batch with its gradient, all three terms
        {"name": "distill step batch", "op": "distill", "grad": True, "n": 2048, "V": 151936, "K": 64,
         "dtype": "bf16", "tail": True, "kl": 1.0, "tv": 1.0, "ce": 0.1},
        # odd rows in fp32, a teacher without a tail (renormalised over its K logits)
        {"name": "distill step f32 ragged", "op": "distill", "grad": True, "n": 501, "V": 100003, "K": 128,
         "dtype": "f32", "tail": False, "kl": 1.0, "tv": 0.0, "ce": 0.0},
        # the loss of a single token: the weight matrix is read once
        {"name": "ce fwd one token", "op": "ce", "pass": "fwd", "n": 1, "H": 2048, "V": 151936},
        # a training batch, one token in ten without a label
        {"name": "ce fwd batch", "op": "ce", "pass": "fwd", "n": 4096, "H": 2048, "V": 151936},
        # the gradients of that batch
        {"name": "ce bwd batch", "op": "ce", "pass": "bwd", "n": 4096, "H": 2048, "V": 151936},
        # a small ragged batch and an odd vocabulary
        {"name": "ce bwd ragged", "op": "ce", "pass": "bwd", "n": 333, "H": 1160, "V": 40001},
        # a few draft chains (8 requests of 8 positions) against a large vocabulary
        {"name": "ce bwd few", "op": "ce", "pass": "bwd", "n": 64, "H": 1024, "V": 128256},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["record", "distill", "distill", "ce", "ce"])
    if op == "ce":
        kind = rng.choice(["fwd", "bwd"])
        V = _log(rng, 1000, 151936)
        H = 8 * _log(rng, 8, 320)
        n = min(_log(rng, 1, 4096), 4096 * 2048 * 151936 // (H * V))
        return {"op": op, "pass": kind, "n": n, "H": H, "V": V}
    V, dtype = _log(rng, 1000, 200000), rng.choice(["bf16", "bf16", "f32"])
    if op == "record":
        return {"op": op, "n": _log(rng, 1, 512), "V": V, "K": _log(rng, 1, 256), "dtype": dtype,
                "kept": rng.choice([0, 0, 50])}
    return {"op": op, "grad": rng.random() < 0.6, "n": _log(rng, 1, 1024), "V": V, "K": _log(rng, 1, 256),
            "dtype": dtype, "tail": rng.random() < 0.7, "kl": rng.choice([0.0, 1.0]),
            "tv": rng.choice([0.0, 1.0]), "ce": rng.choice([0.1, 1.0])}


# ------------------------------------------------------------------------------
# inputs

def _teacher(case, g, dev):
    """Logit rows with a Zipf bias per token: N(0, 3^2) - 1.1 ln(1 + rank)."""
    n, V = case["n"], case["V"]
    rank = torch.randperm(V, generator=g, device=dev).float()
    bias = -1.1 * torch.log1p(rank)
    x = torch.randn(n, V, generator=g, device=dev)
    return x.mul_(3.0).add_(bias).to(_DT[case["dtype"]])


def _ignored(n, g, dev):
    """One row in ten (none of fewer than ten), at seeded places."""
    return torch.randperm(n, generator=g, device=dev)[: n // 10]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, n, V = case["op"], case["n"], case["V"]
    s = {"case": case}
    if op == "ce":
        H = case["H"]
        # projection rows of norm 2, hidden states of unit variance leaning towards their label's row, so that
        # the label's probability runs from ~1e-6 to ~0.9
        w = torch.randn(V, H, generator=g, device=dev).mul_(2.0 / math.sqrt(H)).to(torch.bfloat16)
        label = torch.randint(0, V, (n,), generator=g, device=dev, dtype=torch.int64)
        lean = torch.rand(n, 1, generator=g, device=dev) * 4.5
        h = torch.randn(n, H, generator=g, device=dev) + lean * w[label].float()
        label[_ignored(n, g, dev)] = -1
        s.update(hidden=h.to(torch.bfloat16), weight=w, label=label.to(torch.int32))
        if case["pass"] == "bwd":
            # the mean over the labelled rows, with a weight each; lse as the forward pass left it
            s["grad_loss"] = (torch.rand(n, generator=g, device=dev) + 0.5) / max(1, n - n // 10)
            s["lse"] = _plain_ce_fwd(s["hidden"], w, s["label"])["lse"]
        return s
    s["temperature"] = torch.rand(n, generator=g, device=dev) * 0.6 + 0.6
    x = _teacher(case, g, dev)
    if op == "record":
        if case["kept"]:
            rows = x[3::4]
            if rows.numel():
                kth = rows.float().topk(min(case["kept"], V), dim=1).values[:, -1:]
                rows.masked_fill_(rows.float() < kth, -math.inf)
        s["logits"] = x
        return s
    r = _plain_record(x, case["K"], s["temperature"])
    s["top_logits"], s["top_index"] = r["top_logits"], r["top_index"]
    s["tail_lse"] = r["tail_lse"] if case["tail"] else None
    del r
    s["logits"] = x.float().add_(torch.randn(n, V, generator=g, device=dev), alpha=1.5).to(_DT[case["dtype"]])
    del x
    # labels: tokens of the teacher's record, now and then any token; position weights exp(-i/4) of chains of 7,
    # one row in ten padded (weight 0)
    pick = torch.randint(0, case["K"], (n, 1), generator=g, device=dev)
    label = s["top_index"].gather(1, pick)[:, 0]
    s["label"] = torch.where(torch.rand(n, generator=g, device=dev) < 0.1,
                             torch.randint(0, V, (n,), generator=g, device=dev, dtype=torch.int32), label)
    weight = torch.exp(-(torch.arange(n, device=dev) % 7).float() / 4)
    weight[_ignored(n, g, dev)] = 0
    s["row_weight"] = weight
    return s


# ------------------------------------------------------------------------------
# plain forms

def _plain_record(x, K, temperature):
    f = x.float()
    V = f.shape[1]
    # one integer key per logit: its order, then the lowest index first (-0 counts as 0)
    bits = (f + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (order << 32) | (0x7FFFFFFF - torch.arange(V, device=f.device))
    idx = 0x7FFFFFFF - (key.topk(K, dim=1).values & 0x7FFFFFFF)
    del bits, order, key
    top = f.gather(1, idx)
    T = temperature[:, None]
    m = top[:, :1]
    e = torch.exp((f - m) / T).scatter_(1, idx, 0.0)
    tail = (m / T)[:, 0] + torch.log(e.sum(1))
    return {"top_logits": top, "top_index": torch.where(torch.isinf(top), -1, idx).to(torch.int32), "tail_lse": tail}


def _plain_distill(s, c):
    z, T = s["logits"].float() / s["temperature"][:, None], s["temperature"][:, None]
    n, V = z.shape
    idx, w = s["top_index"].long(), s["row_weight"][:, None]
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    S = e.sum(1, keepdim=True)
    zk, ek = z.gather(1, idx), e.gather(1, idx)
    rest = e.scatter(1, idx, 0.0).sum(1, keepdim=True)
    # the teacher's buckets: its K logits and the rest
    xk = s["top_logits"] / T
    xr = s["tail_lse"][:, None] if s["tail_lse"] is not None else torch.full_like(T, -math.inf)
    mx = torch.maximum(xk.max(1, keepdim=True).values, xr)
    Z = torch.exp(xk - mx).sum(1, keepdim=True) + torch.exp(xr - mx)
    lpk, lpr = xk - mx - torch.log(Z), xr - mx - torch.log(Z)
    pk, pr = torch.exp(lpk), torch.exp(lpr)
    lqk, lqr = zk - m - torch.log(S), torch.log(rest) - torch.log(S)
    qk, qr = ek / S, rest / S
    kl = (pk * (lpk - lqk)).sum(1, keepdim=True) + torch.where(pr > 0, pr * (lpr - lqr), 0.0)
    tv = 0.5 * ((pk - qk).abs().sum(1, keepdim=True) + (pr - qr).abs())
    y = s["label"].long()[:, None]
    ce = m + torch.log(S) - z.gather(1, y)
    live = w != 0
    loss = w * (c["kl"] * kl + c["tv"] * tv + c["ce"] * ce)
    out = {"loss": loss[:, 0], "parts": torch.where(live, torch.cat([kl, tv, ce], 1), 0.0)}
    if c["grad"]:
        sk, sr = torch.sign(qk - pk), torch.sign(qr - pr)
        mean = 0.5 * ((sk * qk).sum(1, keepdim=True) + sr * qr)
        every = c["kl"] + c["tv"] * (0.5 * sr - mean) + c["ce"]      # factor of q_v, v in the rest
        g = e * ((every - c["kl"] * pr / qr) / S)
        g.scatter_(1, idx, qk * (c["kl"] + c["tv"] * (0.5 * sk - mean) + c["ce"]) - c["kl"] * pk)
        g.scatter_add_(1, y, torch.full_like(T, -c["ce"]))
        out["grad"] = (g * (w / T)).to(s["logits"].dtype)
    return out


def _plain_ce_fwd(h, w, label):
    logits = h.float() @ w.float().t()
    m = logits.max(1, keepdim=True).values
    lse = (m + torch.log(torch.exp(logits - m).sum(1, keepdim=True)))[:, 0]
    live = label >= 0
    z = logits.gather(1, label.clamp(min=0).long()[:, None])[:, 0]
    return {"loss": torch.where(live, lse - z, 0.0), "lse": torch.where(live, lse, 0.0)}


def _plain_ce_bwd(s):
    h, w = s["hidden"].float(), s["weight"].float()
    live = s["label"] >= 0
    p = torch.exp(h @ w.t() - s["lse"][:, None])
    y = s["label"].clamp(min=0).long()[:, None]
    p.scatter_add_(1, y, torch.full_like(s["lse"], -1.0)[:, None])
    p *= torch.where(live, s["grad_loss"], 0.0)[:, None]
    return {"grad_hidden": (p @ w).to(torch.bfloat16), "grad_weight": (p.t() @ h).to(torch.bfloat16)}


# ------------------------------------------------------------------------------
# one pass

def run(s):
    c = s["case"]
    if c["op"] == "record":
        if own:
            import speculative_decoding_verification_26_gb300 as sv
            r = sv.topk_logits(s["logits"], c["K"], s["temperature"])
            return {k: r[k] for k in ("top_logits", "top_index", "tail_lse")}
        return _plain_record(s["logits"], c["K"], s["temperature"])
    if c["op"] == "distill":
        if own:
            import speculative_decoding_verification_26_gb300 as sv
            r = sv.distill_topk(s["logits"], s["top_logits"], s["top_index"], s["tail_lse"], label=s["label"],
                                row_weight=s["row_weight"], temperature=s["temperature"], kl=c["kl"], tv=c["tv"],
                                ce=c["ce"], grad=c["grad"])
            return {k: r[k] for k in (("loss", "parts", "grad") if c["grad"] else ("loss", "parts"))}
        return _plain_distill(s, c)
    if c["pass"] == "fwd":
        if own:
            import speculative_decoding_verification_26_gb300 as sv
            r = sv.linear_ce_forward(s["hidden"], s["weight"], s["label"])
            return {k: r[k] for k in ("loss", "lse")}
        return _plain_ce_fwd(s["hidden"], s["weight"], s["label"])
    if own:
        import speculative_decoding_verification_26_gb300 as sv
        r = sv.linear_ce_backward(s["hidden"], s["weight"], s["label"], s["lse"], s["grad_loss"])
        return {k: r[k] for k in ("grad_hidden", "grad_weight")}
    return _plain_ce_bwd(s)


def work(case):
    """Bytes: each input once, each output once.  Operations: a comparison and
    an exponential with its sum per logit; products for the projection."""
    n, V = case["n"], case["V"]
    if case["op"] == "ce":
        H, live = case["H"], n - n // 10
        if case["pass"] == "fwd":
            return {"bytes": 2 * (live * H + V * H) + 12 * n, "flops": 2 * live * H * V}
        return {"bytes": 2 * 2 * (live * H + V * H) + 12 * n, "flops": 6 * live * H * V}
    es, K = (2 if case["dtype"] == "bf16" else 4), case["K"]
    if case["op"] == "record":
        return {"bytes": n * (V * es + 8 * K + 8), "flops": 4 * n * V}
    live = n - n // 10
    out = n * V * es if case["grad"] else 0
    return {"bytes": live * V * es + out + n * (8 * K + 32), "flops": (6 if case["grad"] else 4) * live * V}


# ------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    n, V = case["n"], case["V"]
    if case["op"] == "record":
        top, idx, tail = [], [], []
        for r0 in range(0, n, 64):
            x = s["logits"][r0:r0 + 64].double()
            T = s["temperature"][r0:r0 + 64].double()
            v, i = torch.sort(x, dim=1, descending=True, stable=True)
            K = case["K"]
            top.append(v[:, :K].float())
            idx.append(torch.where(v[:, :K] == -math.inf, -1, i[:, :K]).to(torch.int32))
            tail.append(torch.logsumexp(v[:, K:] / T[:, None], 1) if K < V else torch.full_like(T, -math.inf))
        return {"top_logits": torch.cat(top).double(), "top_index": torch.cat(idx), "tail_lse": torch.cat(tail)}
    if case["op"] == "distill":
        loss, parts, grads = [], [], []
        for r0 in range(0, n, 256):
            sl = slice(r0, r0 + 256)
            T = s["temperature"][sl].double()[:, None]
            w = s["row_weight"][sl].double()[:, None]
            lq = torch.log_softmax(s["logits"][sl].double() / T, 1)
            q = lq.exp()
            idx = s["top_index"][sl].long()
            inside = torch.zeros_like(q, dtype=torch.bool).scatter_(1, idx, True)
            tail = s["tail_lse"][sl].double()[:, None] if s["tail_lse"] is not None else torch.full_like(T, -math.inf)
            lp = torch.log_softmax(torch.cat([s["top_logits"][sl].double() / T, tail], 1), 1)
            p = lp.exp()
            qr = torch.where(inside, 0.0, q).sum(1, keepdim=True)
            qb = torch.cat([q.gather(1, idx), qr], 1)
            lqb = torch.cat([lq.gather(1, idx), qr.log()], 1)
            kl = torch.where(p > 0, p * (lp - lqb), 0.0).sum(1, keepdim=True)
            tv = 0.5 * (p - qb).abs().sum(1, keepdim=True)
            y = s["label"][sl].long()[:, None]
            ce = -lq.gather(1, y)
            loss.append((w * (case["kl"] * kl + case["tv"] * tv + case["ce"] * ce))[:, 0])
            parts.append(torch.cat([kl, tv, ce], 1) * (w != 0))
            if case["grad"]:
                # by the buckets: d(loss)/dq_b, spread over each bucket's tokens, then through the softmax
                db = case["kl"] * torch.where(p > 0, -p / qb, 0.0) + case["tv"] * 0.5 * torch.sign(qb - p)
                dq = db[:, -1:].expand(-1, V).clone().scatter_(1, idx, db[:, :-1])
                dq.scatter_add_(1, y, -case["ce"] / q.gather(1, y))
                grads.append(w / T * q * (dq - (q * dq).sum(1, keepdim=True)))
        out = {"loss": torch.cat(loss), "parts": torch.cat(parts)}
        if case["grad"]:
            out["grad"] = torch.cat(grads)
        return out
    h, w, live = s["hidden"].double(), s["weight"].double(), s["label"] >= 0
    y = s["label"].clamp(min=0).long()
    if case["pass"] == "fwd":
        loss, lse = [], []
        for r0 in range(0, n, 1024):
            logits = h[r0:r0 + 1024] @ w.t()
            lse.append(torch.logsumexp(logits, 1))
            loss.append(lse[-1] - logits.gather(1, y[r0:r0 + 1024, None])[:, 0])
        return {"loss": torch.where(live, torch.cat(loss), 0.0), "lse": torch.where(live, torch.cat(lse), 0.0)}
    gh, gw = [], torch.zeros_like(w)
    for r0 in range(0, n, 1024):
        sl = slice(r0, r0 + 1024)
        p = torch.exp(h[sl] @ w.t() - s["lse"][sl].double()[:, None])
        p[torch.arange(p.shape[0], device=p.device), y[sl]] -= 1
        p *= torch.where(live[sl], s["grad_loss"][sl].double(), 0.0)[:, None]
        gh.append(p @ w)
        gw.addmm_(p.t(), h[sl])
    return {"grad_hidden": torch.cat(gh), "grad_weight": gw}
