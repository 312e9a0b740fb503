"""Plain 64-bit implementations of the calls around the vocabulary rows of a
decode step (CPU)."""
import math

import torch

PLACE = (0, 4, 1, 5, 2, 6, 3, 7)           # the nibble of weight i of a word


def pack(q):
    """Whole numbers [V, H] from 0 to 15 as packed bytes [V, H / 2]."""
    V, H = q.shape
    word = torch.zeros(V, H // 8, dtype=torch.int64)
    for i, p in enumerate(PLACE):
        word |= q[:, i::8].long() << 4 * p
    return torch.stack([(word >> 8 * k) & 255 for k in range(4)], 2).reshape(V, H // 2).to(torch.uint8)


def unpack(packed):
    V, B = packed.shape
    b = packed.long().view(V, B // 4, 4)
    word = b[:, :, 0] | b[:, :, 1] << 8 | b[:, :, 2] << 16 | b[:, :, 3] << 24
    return torch.stack([(word >> 4 * p) & 15 for p in PLACE], 2).reshape(V, 2 * B)


def two_step(x):
    """64 bits to fp32 and from there to bf16."""
    return x.float().to(torch.bfloat16)


def quantize(weight, group, zero):
    """(q [V, H], scale, zero) of spec_w4_quantize."""
    V, H = weight.shape
    q = torch.empty(V, H, dtype=torch.int64)
    scales, zeros = [], []
    for k in range(0, H, group):
        w = weight[:, k:k + group].double()
        odd = ~torch.isfinite(w).all(1)
        w = torch.where(odd[:, None], 0.0, w)
        if zero:
            lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
            scale = two_step((hi - lo) / 15)
        else:
            scale = two_step(w.abs().amax(1) / 7)
        s = scale.double()
        z = torch.full_like(s, 8.0)
        if zero:
            z = torch.where(s > 0, torch.round(-lo / s).clamp(0, 15), z)
        level = torch.where(s[:, None] > 0, torch.round(w / s[:, None]) + z[:, None], z[:, None]).clamp(0, 15)
        q[:, k:k + group] = level.long()
        scales.append(torch.where(odd, math.nan, scale.float()).to(torch.bfloat16))
        zeros.append(z.to(torch.uint8))
    return q, torch.stack(scales, 1), torch.stack(zeros, 1)


def weights(q, scale, zero, group):
    H = q.shape[1]
    s = scale.double().repeat_interleave(group, 1)[:, :H]
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, 1)[:, :H]
    return (q.double() - z) * s


def adjust(x, history=None, history_len=None, prompt_len=None, draft_tokens=None, gamma=None, repetition=None,
           frequency=None, presence=None, bias_index=None, bias_value=None, mask=None):
    """(rows in 64 bits, the sum of the magnitudes that made each, touched) by the
    definition, token by token; rows behind gamma as they were."""
    B, R, V = x.shape
    y = x.double().clone()
    mag = torch.zeros(B, R, V, dtype=torch.double)
    touched = torch.zeros(B, R, V, dtype=torch.bool)
    for b in range(B):
        h = [] if history is None else history[b].tolist()
        n = len(h) if history_len is None else int(history_len[b])
        p = 0 if prompt_len is None else int(prompt_len[b])
        d = [] if draft_tokens is None else draft_tokens[b].tolist()
        most = len(d) if d else R - 1
        gm = most if gamma is None else int(gamma[b])
        rep = 1.0 if repetition is None else float(repetition[b])
        freq = 0.0 if frequency is None else float(frequency[b])
        pres = 0.0 if presence is None else float(presence[b])
        bias = {}
        if bias_index is not None:
            for v, a in zip(bias_index[b].tolist(), bias_value[b].tolist()):
                if v >= 0:
                    bias.setdefault(v, []).append(a)
        for i in range(min(R, gm + 1)):
            out = [v for v in h[p:n] + d[:min(i, gm)] if v >= 0]
            count = {}
            for v in out:
                count[v] = count.get(v, 0) + 1
            for v in set(out) | {v for v in h[:p] if v >= 0}:
                a = float(y[b, i, v])
                a = a / rep if a > 0 else a * rep
                m = abs(a)
                if count.get(v):
                    a -= count[v] * freq + pres
                    m += abs(count[v] * freq) + abs(pres)
                y[b, i, v], mag[b, i, v], touched[b, i, v] = a, m, True
            for v, values in bias.items():
                s = sum(values)
                mag[b, i, v] += (float(y[b, i, v].abs()) if not touched[b, i, v] else 0.0) + len(values) * sum(map(abs, values))
                y[b, i, v] += s
                touched[b, i, v] = True
            if mask is not None:
                v = torch.arange(V)
                ok = (mask[b, i].long()[v // 32] >> (v % 32) & 1).bool()
                y[b, i][~ok] = -math.inf
                touched[b, i] |= ~ok
    return y, mag, touched
