"""Plain 64-bit forms of the router on the CPU, with bounds of the rounding
errors of an fp32 evaluation.

Bounds (u = 2^-24, fp32's half step). A score is an exponential of an exact or
once rounded difference (off by (|difference| + 2) u relative), a sum of at most
E of them in fp32 (gamma(E) and the terms' own errors), a division and a
product with the scale: in all at most (2 |d| + 2 E + 16) u relative, |d| the
largest difference of a logit to the largest one, or the largest |logit| for
the sigmoid."""
import math

import torch

U = 2.0 ** -24
B = 2.0 ** -8


def select(logits, K, score, bias=None, groups=1, kept=1):
    """ids [T, K] (int64, -1 for none), one expert after the other."""
    T, E = logits.shape
    out = torch.full((T, K), -1)
    size = E // groups
    for t in range(T):
        l = [float(x) for x in logits[t].double()]
        part = [not math.isnan(x) and x != -math.inf for x in l]
        counts = v = l
        if score == "sigmoid":
            counts = torch.sigmoid(logits[t].double())
            if bias is not None:
                counts = counts + bias.double()
                v = counts.tolist()
            counts = counts.tolist()
        ok = [e for e in range(E) if part[e] and not math.isnan(v[e]) and v[e] != -math.inf]
        if groups > 1:
            value = {}
            for g in range(groups):
                mine = sorted((e for e in ok if e // size == g), key=lambda e: (-v[e], e))
                if mine:
                    value[g] = sum(counts[e] for e in mine[:2 if score == "sigmoid" else 1])
            best = sorted(value, key=lambda g: (-value[g], g))[:kept]
            ok = [e for e in ok if e // size in best]
        for k, e in enumerate(sorted(ok, key=lambda e: (-v[e], e))[:K]):
            out[t, k] = e
    return out


def probabilities(logits, score):
    """p [T, E] in 64 bits, 0 where an expert takes no part, and the bound."""
    l = logits.double()
    part = ~torch.isnan(l) & (l != -math.inf)
    if score == "sigmoid":
        return torch.where(part, torch.sigmoid(l), torch.zeros_like(l)), part
    l = torch.where(part, l, torch.full_like(l, -math.inf))
    m = l.amax(dim=1, keepdim=True)
    e = torch.where(part, torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m)),
                    torch.zeros_like(l))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300), part


def scores(logits, ids, score, renormalize, scale):
    """The scores of the ids in 64 bits and the relative error bound."""
    p, part = probabilities(logits, score)
    there = ids >= 0
    q = torch.where(there, torch.gather(p, 1, ids.clamp(min=0)), torch.zeros(()).double())
    if renormalize:
        q = q / q.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return q * scale, bound(logits, part, score)


def bound(logits, part, score):
    l = logits.double()
    l = l[part & torch.isfinite(l)]
    if l.numel() == 0:
        return 0.0
    d = float(l.abs().max()) if score == "sigmoid" else float(l.max() - l.min())
    return (2 * d + 2 * logits.shape[1] + 16) * U


def gradient(logits, ids, grad, score, renormalize, scale):
    """The logits' gradient in 64 bits by the formula, and a bound of the
    absolute error before its last rounding: every factor of a term is off by
    the scores' relative bound, the sum over K terms by gamma(K)."""
    p, part = probabilities(logits, score)
    rel = 4 * (bound(logits, part, score) + 32 * U)
    there = ids >= 0
    at = ids.clamp(min=0)
    zero = torch.zeros((), dtype=torch.float64)
    g = torch.where(there, grad.double() * scale, zero)
    pk = torch.where(there, torch.gather(p, 1, at), zero)
    total = pk.sum(dim=1, keepdim=True).clamp(min=1e-300)
    q = pk / total if renormalize else pk
    s = (g * q).sum(dim=1, keepdim=True)
    s_mag = (g * q).abs().sum(dim=1, keepdim=True)
    out, mag = torch.zeros_like(p), torch.zeros_like(p)
    if score == "softmax":
        if not renormalize:
            out, mag = -p * s, p * s_mag
            d, dm = q * g, q * g.abs()
        else:
            d, dm = q * (g - s), q * (g.abs() + s_mag)
    else:
        slope = pk * torch.sigmoid(-torch.gather(torch.nan_to_num(logits.double()), 1, at))
        if renormalize:
            d, dm = (g - s) / total * slope, (g.abs() + s_mag) / total * slope
        else:
            d, dm = g * slope, g.abs() * slope
    d, dm = torch.where(there, d, zero), torch.where(there, dm, zero)
    return out.scatter_add(1, at, d), rel * mag.scatter_add(1, at, dm)


# ---- MXFP4 ------------------------------------------------------------------

MIDDLES = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
UP = torch.tensor([False, True, False, True, False, True, False])   # a middle rounds to the even code


def quantize(x):
    """(values, scales) uint8 of x [..., k] by the definition, 64-bit
    arithmetic; a block with a NaN or infinity gets zeros and 255."""
    b = x.double().unflatten(-1, (-1, 32))
    lost = ~torch.isfinite(b).all(dim=-1, keepdim=True)
    b = torch.where(lost, torch.zeros_like(b), b)
    top = b.abs().amax(dim=-1, keepdim=True)
    e = torch.frexp(top)[1].double() - 3          # top = m 2^exponent, 1/2 <= m < 1
    e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    t = (b.abs() * torch.exp2(-e)).unsqueeze(-1)
    code = ((t > MIDDLES) | (UP & (t == MIDDLES))).sum(dim=-1)
    code += 8 * torch.signbit(torch.where(lost, torch.zeros_like(b), b)).long()
    code = code.flatten(-2).to(torch.uint8)
    scales = torch.where(lost, torch.full_like(e, 255), e + 127).squeeze(-1).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def decode(values, scales):
    """float64 [..., k]."""
    import expert_ref
    q = torch.stack((values & 15, values >> 4), dim=-1).flatten(-2).long()
    s = torch.ldexp(torch.ones((), dtype=torch.float64), scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return expert_ref.E2M1[q] * s.repeat_interleave(32, dim=-1)


def product(x, w, off):
    """out[r] = x[r] w[e]^T in 64 bits and the error bound of its sum in fp32 on
    the matrix cores: each of the k additions loses at most a whole unit (2 u)
    of the sum of the products' magnitudes, since they may truncate."""
    import expert_ref
    out, mag = expert_ref.linear(x, w, off)
    return out, 2 * expert_ref.gamma(x.shape[1]) * mag


def gate(pre, dpre, name):
    """act(g) * u of pre = [g | u] with errors dpre, and the error before the
    last rounding."""
    import expert_ref as er
    F = pre.shape[1] // 2
    g, u, dg, du = pre[:, :F], pre[:, F:], dpre[:, :F], dpre[:, F:]
    a = er.act(name, g)[0]
    da = er.SLOPE * dg + er.act_error(name, g)[0]
    h = a * u
    return h, da * (u.abs() + du) + a.abs() * du + 2 * U * h.abs()


# ---- The whole layer ---------------------------------------------------------

def layer(x, scores, ids, w13, w2, name):
    """y [T, D] in 64 bits and the error bound before its last rounding, for
    x [T, D], w13 [E, 2F, D], w2 [E, D, F] as numbers of any type.

    h = act(g) * u is off by the fp32 evaluation (gate()); as two bf16 it loses
    B^2 |h| more, and what lies below bf16's normal numbers (2^-126). Its sum
    with w2 has 2 F terms of magnitude at most (1 + 2 B) |h w2|, joined from at
    most 8 parts; the sum over the slots has K terms."""
    import expert_ref as er
    T, K = ids.shape
    E, D, F = w2.shape
    y, err = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        off = [0, len(t)]
        pre, m = er.linear(x[t], w13[e:e + 1], off)
        h, dh = gate(pre, 2 * er.gamma(D + 8) * m, name)
        dh = dh + B * B * h.abs() + 2.0 ** -126
        w = w2[e].double()
        p = h @ w.t()
        pm = (1 + 2 * B) * (h.abs() + dh) @ w.abs().t()
        s = scores[t, k].double()[:, None]
        y.index_add_(0, t, s * p)
        mag.index_add_(0, t, s.abs() * pm)
        err.index_add_(0, t, s.abs() * (dh @ w.abs().t() + 2 * er.gamma(2 * F + 16) * pm))
    return y, err + 2 * er.gamma(K + 1) * mag
