"""The operators around the vocabulary rows of a decode step: what is measured,
and their plain forms.

  quantize  a weight matrix to 4 bits with a scale (and a zero point) for each
            group of weights, and read back (quantize_w4, dequantize_w4);
  project   hidden states times such a matrix: the logits of a vocabulary
            projection, or any other linear layer (linear_w4);
  adjust    penalties for repeated tokens, biases and grammar masks on logit
            rows, each row with the history of its own candidate prefix
            (adjust_logits).

`run` computes the plain form in 32 bits with elementary torch operations, or,
where `own` is true, makes the library's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the vocabulary projection of a drafter, laid out once when it is loaded
        {"name": "quantize projection", "op": "quantize", "H": 2048, "V": 151936, "group": 128, "zero": False, "dtype": "bf16"},
        # a master copy in fp32, an odd vocabulary, short groups with zero points
        {"name": "quantize f32 ragged", "op": "quantize", "H": 1184, "V": 40001, "group": 32, "zero": True, "dtype": "f32"},
        # one square layer
        {"name": "quantize layer", "op": "quantize", "H": 2048, "V": 2048, "group": 64, "zero": False, "dtype": "bf16"},
        # the draft step of a single request: the weights are read once
        {"name": "project one token", "op": "project", "n": 1, "H": 2048, "V": 151936, "group": 128, "zero": False, "out": "bf16"},
        # a small layer for the 8 rows of one chain: latency
        {"name": "project small layer", "op": "project", "n": 8, "H": 2048, "V": 2048, "group": 64, "zero": False, "out": "bf16"},
        # the draft step of 64 requests (the verification workload)
        {"name": "project draft step", "op": "project", "n": 64, "H": 2048, "V": 151936, "group": 128, "zero": False, "out": "bf16"},
        # odd sizes, short groups with zero points, fp32 logits
        {"name": "project ragged", "op": "project", "n": 7, "H": 1184, "V": 40001, "group": 32, "zero": True, "out": "f32"},
        # the target rows of 64 requests at gamma = 7
        {"name": "project target rows", "op": "project", "n": 512, "H": 2048, "V": 151936, "group": 128, "zero": False, "out": "bf16"},
        # the target rows of one request at gamma = 7, a short history; the rows as they were are kept
        {"name": "adjust one request", "op": "adjust", "B": 1, "R": 8, "V": 151936, "L": 512, "penalties": True, "biases": 0,
         "allowed": 1.0, "place": "out", "dtype": "bf16"},
        # the target rows of 64 requests with all three kinds
        {"name": "adjust batch", "op": "adjust", "B": 64, "R": 8, "V": 151936, "L": 2048, "penalties": True, "biases": 32,
         "allowed": 0.9, "place": "out", "dtype": "bf16"},
        # odd rows in fp32, long histories, many biases
        {"name": "adjust f32 ragged", "op": "adjust", "B": 13, "R": 5, "V": 100003, "L": 8192, "penalties": True, "biases": 300,
         "allowed": 0.5, "place": "out", "dtype": "f32"},
        # a grammar that leaves few tokens, in place
        {"name": "mask in place", "op": "adjust", "B": 64, "R": 8, "V": 151936, "L": 0, "penalties": False, "biases": 0,
         "allowed": 0.02, "place": "in", "dtype": "bf16"},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["quantize", "project", "project", "adjust", "adjust"])
    if op == "adjust":
        V, place = _log(rng, 1000, 200000), rng.choice(["out", "out", "in"])
        B, R, dtype = _log(rng, 1, 64), rng.randint(1, 9), rng.choice(["bf16", "bf16", "f32"])
        B = max(1, min(B, 64 * 8 * 151936 * 2 // (R * V * (2 if dtype == "bf16" else 4))))
        if place == "in":
            return {"op": op, "B": B, "R": R, "V": V, "L": 0, "penalties": False, "biases": 0,
                    "allowed": rng.choice([0.02, 0.5, 0.98]), "place": place, "dtype": dtype}
        return {"op": op, "B": B, "R": R, "V": V, "L": _log(rng, 1, 8192), "penalties": True,
                "biases": rng.choice([0, 1, 32, 300]), "allowed": rng.choice([1.0, 0.9, 0.1]), "place": place, "dtype": dtype}
    V, H = _log(rng, 512, 151936), 32 * _log(rng, 8, 160)
    V = min(V, 2048 * 151936 // H)
    case = {"op": op, "H": H, "V": V, "group": rng.choice([32, 64, 128, 128]), "zero": rng.random() < 0.4}
    if op == "quantize":
        case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if case["dtype"] == "f32":
            case["V"] = max(1, V // 2)
    else:
        case["out"] = rng.choice(["bf16", "bf16", "f32"])
        case["n"] = _log(rng, 1, 512 if case["out"] == "bf16" else 256)
    return case


# ------------------------------------------------------------------------------
# inputs

# the place (nibble of a 32-bit word) of each of 8 weights in a row
_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    op, V = case["op"], case["V"]
    if op == "quantize":
        # rows of different norms, a few weights that stand out
        H = case["H"]
        w = torch.randn(V, H, generator=g, device=dev)
        w *= (torch.rand(V, 1, generator=g, device=dev) + 0.5) / math.sqrt(H)
        w[torch.randint(0, V, (V // 4,), generator=g, device=dev), torch.randint(0, H, (V // 4,), generator=g, device=dev)] *= 6
        s["weight"] = w.to(_DT[case["dtype"]])
        return s
    if op == "project":
        n, H, G = case["n"], case["H"], -(-case["H"] // case["group"])
        q = torch.randn(V, H, generator=g, device=dev).mul_(2.7).round_().add_(8).clamp_(0, 15).to(torch.int32)
        shift = torch.tensor([4 * j for j in _NIBBLE], dtype=torch.int32, device=dev)
        word = (q.view(V, H // 8, 8) << shift).sum(2, dtype=torch.int32)
        del q
        s["packed"] = word.view(torch.uint8).view(V, H // 2)
        s["scale"] = ((torch.rand(V, G, generator=g, device=dev) + 0.5) * (2.0 / 2.7 / math.sqrt(H))).to(torch.bfloat16)
        s["zero"] = torch.randint(6, 11, (V, G), generator=g, device=dev, dtype=torch.uint8) if case["zero"] else None
        s["hidden"] = torch.randn(n, H, generator=g, device=dev).to(torch.bfloat16)
        return s
    B, R, L, dt = case["B"], case["R"], case["L"], _DT[case["dtype"]]
    x = torch.randn(B, R, V, generator=g, device=dev).mul_(3.0)
    rank = torch.randperm(V, generator=g, device=dev)
    x -= 1.1 * torch.log1p(rank.float())
    s["logits"] = x.to(dt)
    s["adjusted"] = torch.empty_like(s["logits"]) if case["place"] == "out" else s["logits"]

    def tokens(*shape):
        """Frequent tokens more often: ranks uniform in their logarithm."""
        by_rank = torch.argsort(rank)
        u = torch.rand(*shape, generator=g, device=dev, dtype=torch.float64)
        return by_rank[(torch.exp(u * math.log(V)) - 1).long().clamp_(0, V - 1)].to(torch.int32)

    s["history"] = s["history_len"] = s["prompt_len"] = s["draft_tokens"] = None
    s["repetition"] = s["frequency"] = s["presence"] = None
    if case["penalties"]:
        # histories of different lengths (one request in eight has none yet), the first half of each a prompt
        s["history"] = tokens(B, L)
        length = torch.randint(L // 2, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        length[7::8] = 0
        s["history_len"], s["prompt_len"] = length, length // 2
        s["draft_tokens"] = tokens(B, R)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device=dev)
        s["frequency"] = torch.rand(B, generator=g, device=dev)
        s["presence"] = torch.rand(B, generator=g, device=dev)
    s["bias_index"] = s["bias_value"] = None
    if case["biases"]:
        s["bias_index"] = tokens(B, case["biases"])
        s["bias_value"] = torch.randn(B, case["biases"], generator=g, device=dev) * 4
    s["mask"] = None
    if case["allowed"] < 1.0:
        W = -(-V // 32)
        keep = (torch.rand(B, R, W * 32, generator=g, device=dev) < case["allowed"]).view(B, R, W, 32)
        bit = torch.arange(32, device=dev, dtype=torch.int32)
        s["mask"] = (keep.to(torch.int32) << bit).sum(3, dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------
# plain forms

def _groups(x, group):
    """[V, H] as [V, groups, group], the last one filled up with zeros."""
    V, H = x.shape
    G = -(-H // group)
    return torch.nn.functional.pad(x, (0, G * group - H)).view(V, G, group)


def _plain_quantize(weight, group, zero):
    # in 64 bits: quotients next to a half
    V, H = weight.shape
    w = _groups(weight.double(), group)
    if zero:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).to(torch.bfloat16)
        s = scale.double()
        z = torch.where(s > 0, (-lo / s).round().clamp(0, 15), 8.0)
    else:
        scale = (w.abs().amax(2) / 7).to(torch.bfloat16)
        s = scale.double()
        z = torch.full_like(s, 8.0)
    w /= s[:, :, None]
    q = torch.where(s[:, :, None] > 0, (w.round_() + z[:, :, None]).clamp_(0, 15), z[:, :, None])
    del w
    back = ((q - z[:, :, None]) * s[:, :, None]).view(V, -1)[:, :H].to(weight.dtype)
    return {"scale": scale, "zero": z.to(torch.uint8) if zero else None, "weight": back}


def _plain_weight(packed, scale, zero, group):
    V, H = packed.shape[0], 2 * packed.shape[1]
    shift = torch.tensor(_NIBBLE, dtype=torch.int32, device=packed.device) * 4
    q = ((packed.view(torch.int32)[:, :, None] >> shift) & 15).view(V, H).float()
    z = 8.0 if zero is None else zero.float().repeat_interleave(group, 1)[:, :H]
    return (q - z) * scale.float().repeat_interleave(group, 1)[:, :H]


def _plain_adjust(s, c):
    x = s["logits"].float()
    B, R, V = x.shape
    if s["history"] is not None:
        at = torch.arange(c["L"], device=x.device)
        live = at < s["history_len"][:, None]
        told = live & (at >= s["prompt_len"][:, None])
        tok = s["history"].long()
        seen = torch.zeros(B, V, device=x.device).scatter_add_(1, tok, live.float())
        count = torch.zeros(B, V, device=x.device).scatter_add_(1, tok, told.float())
        # row i has the drafts before it: y_0 .. y_{i - 1}
        mine = torch.zeros(B, R, V, device=x.device)
        mine[:, 1:].scatter_(2, s["draft_tokens"][:, :R - 1, None].long(), 1.0)
        mine = mine.cumsum(1)
        seen = (seen[:, None] + mine) > 0
        mine += count[:, None]
        rep, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - (mine * freq + (mine > 0) * pres)
    if s["bias_index"] is not None:
        bias = torch.zeros(B, V, device=x.device).scatter_add_(1, s["bias_index"].long(), s["bias_value"])
        x = x + bias[:, None]
    if s["mask"] is not None:
        bit = torch.arange(32, device=x.device, dtype=torch.int32)
        keep = ((s["mask"][..., None] >> bit) & 1).view(B, R, -1)[:, :, :V]
        x = torch.where(keep > 0, x, -math.inf)
    return s["adjusted"].copy_(x)


# ------------------------------------------------------------------------------
# one pass

def run(s):
    c = s["case"]
    if c["op"] == "quantize":
        if own:
            import speculative_decoding_verification_26_gb300 as sv
            r = sv.quantize_w4(s["weight"], c["group"], zero=c["zero"])
            zero = r["zero"] if c["zero"] else None
            back = sv.dequantize_w4(r["packed"], r["scale"], zero, group=c["group"], dtype=s["weight"].dtype)["weight"]
            return {"scale": r["scale"], "zero": zero, "weight": back}
        return _plain_quantize(s["weight"], c["group"], c["zero"])
    if c["op"] == "project":
        if own:
            import speculative_decoding_verification_26_gb300 as sv
            return sv.linear_w4(s["hidden"], s["packed"], s["scale"], s["zero"], group=c["group"], dtype=_DT[c["out"]])["logits"]
        w = _plain_weight(s["packed"], s["scale"], s["zero"], c["group"])
        return (s["hidden"].float() @ w.t()).to(_DT[c["out"]])
    if own:
        import speculative_decoding_verification_26_gb300 as sv
        r = sv.adjust_logits(s["logits"], s["history"], s["history_len"], prompt_len=s["prompt_len"],
                             draft_tokens=s["draft_tokens"], repetition=s["repetition"], frequency=s["frequency"],
                             presence=s["presence"], bias_index=s["bias_index"], bias_value=s["bias_value"],
                             mask=s["mask"], out={"logits": s["adjusted"]})
        return r["logits"]
    return _plain_adjust(s, c)


def work(case):
    """Bytes: each input once, each output once; in place, the logits that a
    mask removes are written and the others are not touched.  Operations: a
    product and a sum for each weight and row of a projection; quotient,
    rounding and reading back of each quantised weight; a few for each logit."""
    V = case["V"]
    if case["op"] == "adjust":
        B, R, es = case["B"], case["R"], 2 if case["dtype"] == "bf16" else 4
        rows = 2 * B * R * V * es if case["place"] == "out" else (1 - case["allowed"]) * B * R * V * es
        mask = B * R * V / 8 if case["allowed"] < 1.0 else 0
        return {"bytes": rows + mask + 4 * B * case["L"] + 8 * B * case["biases"], "flops": 4 * B * R * V}
    H, G = case["H"], -(-case["H"] // case["group"])
    store = V * H / 2 + V * G * (3 if case["zero"] else 2)
    if case["op"] == "quantize":
        return {"bytes": store + 2 * V * H * (2 if case["dtype"] == "bf16" else 4), "flops": 6 * V * H}
    n = case["n"]
    return {"bytes": store + 2 * n * H + n * V * (2 if case["out"] == "bf16" else 4), "flops": 2 * n * H * V}


# ------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_quantize(w, group, zero):
    scales, zeros, backs = [], [], []
    for k in range(0, w.shape[1], group):
        x = w[:, k:k + group].double()
        if zero:
            lo, hi = torch.clamp(x.min(1).values, max=0.0), torch.clamp(x.max(1).values, min=0.0)
            s = ((hi - lo) / 15.0).bfloat16().double()
            z = torch.clamp(torch.round(-lo / s), 0, 15)
        else:
            s = (x.abs().max(1).values / 7.0).bfloat16().double()
            z = torch.full_like(s, 8)
        none = s == 0
        z = torch.where(none, 8.0, z)
        level = torch.clamp(torch.round(x / s[:, None]), -z[:, None], 15 - z[:, None])
        scales.append(s)
        zeros.append(z)
        backs.append(torch.where(none[:, None], 0.0, level * s[:, None]))
    return torch.stack(scales, 1), torch.stack(zeros, 1).to(torch.uint8), torch.cat(backs, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        scale, zero, back = _exact_quantize(s["weight"], case["group"], case["zero"])
        return {"scale": scale, "zero": zero if case["zero"] else None, "weight": back}
    if case["op"] == "project":
        h, out = s["hidden"].double(), []
        for v in range(0, case["V"], 16384):
            word = s["packed"][v:v + 16384].view(torch.int32).long() & 0xFFFFFFFF
            w = torch.empty(word.shape[0], case["H"], dtype=torch.float64, device=word.device)
            for k in range(8):
                w[:, k::8] = ((word >> 4 * _NIBBLE[k]) % 16).double()
            for j in range(s["scale"].shape[1]):
                part = w[:, j * case["group"]:(j + 1) * case["group"]]
                part -= 8 if s["zero"] is None else s["zero"][v:v + 16384, j, None].double()
                part *= s["scale"][v:v + 16384, j, None].double()
            out.append(h @ w.t())
        return torch.cat(out, 1)
    x = s["logits"].double()
    B, R, V = x.shape
    for b in range(B):
        bias = torch.zeros(V, dtype=torch.float64, device=x.device)
        if s["bias_index"] is not None:
            bias.index_add_(0, s["bias_index"][b].long(), s["bias_value"][b].double())
        for i in range(R):
            row = x[b, i]
            if s["history"] is not None:
                n, p = int(s["history_len"][b]), int(s["prompt_len"][b])
                said = torch.cat([s["history"][b, p:n], s["draft_tokens"][b, :i]]).long()
                count = torch.bincount(said, minlength=V).double()
                met = count > 0
                met[s["history"][b, :p].long()] = True
                rep = float(s["repetition"][b])
                row = torch.where(met, torch.where(row > 0, row / rep, row * rep), row)
                row = row - count * float(s["frequency"][b]) - torch.where(count > 0, float(s["presence"][b]), 0.0)
            row = row + bias
            if s["mask"] is not None:
                v = torch.arange(V, device=x.device)
                allowed = s["mask"][b, i][v // 32].long() >> (v % 32) & 1
                row = row.masked_fill(allowed == 0, -math.inf)
            x[b, i] = row
    return x
