"""Plain 64-bit forms of the expert feed-forward block and its gradients on
the CPU, with bounds of the rounding errors of a bf16 / fp32 evaluation.

Bounds. u = 2^-24 is fp32's half step, B = 2^-8 bf16's (relative to the
value). A sum of k products accumulated in fp32 in any order is off by at most
gamma(k) = k u / (1 - k u) times the sum of the products' magnitudes. act(g) in
fp32 is g times a sigmoid whose exponential has relative error below
(|z| + 8) 2^-22, z being the sigmoid's argument (one rounding of the scaled
argument, exp2, one addition, one reciprocal)."""
import math

import torch

U = 2.0 ** -24
B = 2.0 ** -8
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)
ALPHA, BETA = math.sqrt(2 / math.pi), 0.044715
SLOPE, CURVE = 1.13, 1.2   # bounds of |act'| and |act''| for both activations


def gamma(k):
    return k * U / (1 - k * U)


def offsets_of(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + int(c))
    return off


def segments(off):
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def act(name, g):
    """Value, slope and the sigmoid's argument."""
    if name == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        z = 2 * ALPHA * (g + BETA * g ** 3)
        dz = 2 * ALPHA * (1 + 3 * BETA * g ** 2)
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    return g * p, p + g * p * q * dz, z


def act_error(name, g):
    """Bound of the fp32 evaluation's error in act(g) for a given g, and of
    the slope's."""
    value, slope, z = act(name, g)
    rel = (z.abs() + 8) * 2.0 ** -22
    dz = torch.ones_like(g) if name == "silu" else 2 * ALPHA * (1 + 3 * BETA * g ** 2)
    p = torch.sigmoid(z)
    pq = p * torch.sigmoid(-z)
    # slope = p + g p (1 - p) dz: p's relative error enters both factors, and
    # 1 - p carries an absolute half step.
    return value.abs() * rel, p * rel + (g * dz).abs() * (2 * pq * rel + p * 2 * U)


def linear(x, w, off):
    """out[r] = x[r] w[e]^T in 64 bits and the sum of the magnitudes."""
    out = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e, a, b in segments(off):
        xe, we = x[a:b].double(), w[e].double()
        out[a:b] = xe @ we.t()
        mag[a:b] = xe.abs() @ we.abs().t()
    return out, mag


def gated(x, w, off, name):
    """h, its error bound before the last rounding, and [g | u] with theirs."""
    F = w.shape[1] // 2
    pre, mag = linear(x, w, off)
    dpre = gamma(x.shape[1]) * mag
    g, u = pre[:, :F], pre[:, F:]
    dg, du = dpre[:, :F], dpre[:, F:]
    a, _, _ = act(name, g)
    da = SLOPE * dg + act_error(name, g)[0]
    h = a * u
    return h, da * (u.abs() + du) + a.abs() * du + 2 * U * h.abs(), pre, dpre


def gated_grad(dy, w_down, pre, off, name):
    """[dh*u*act' | dh*act] from dy and the rounded pre, with the error bound
    before the last rounding."""
    F = w_down.shape[2]
    dh, mag = linear(dy, w_down.transpose(1, 2).contiguous(), off)
    ddh = gamma(dy.shape[1]) * mag
    g, u = pre[:, :F].double(), pre[:, F:].double()
    a, s, _ = act(name, g)
    ea, es = act_error(name, g)
    out = torch.cat((dh * u * s, dh * a), 1)
    err = torch.cat((ddh * (u * s).abs() + (dh.abs() + ddh) * u.abs() * es,
                     ddh * a.abs() + (dh.abs() + ddh) * ea), 1)
    return out, err + 4 * U * out.abs()


def wgrad(dy, x, off):
    E = len(off) - 1
    out = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    terms = torch.zeros(E, 1, 1, dtype=torch.float64)
    for e, a, b in segments(off):
        d, xe = dy[a:b].double(), x[a:b].double()
        out[e] = d.t() @ xe
        mag[e] = d.abs().t() @ xe.abs()
        terms[e] = gamma(b - a)
    return out, terms * mag


def mxfp4_weights(values, scales):
    """uint8 [E, N, K/2] and [E, N, K/32] to float64 [E, N, K]."""
    q = torch.stack((values & 15, values >> 4), dim=3).flatten(2).long()
    s = torch.ldexp(torch.ones((), dtype=torch.float64), scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return E2M1[q] * s.repeat_interleave(32, dim=2)


def check(got, want, err, half_step, what):
    """|got - want| <= err + half_step * |got| everywhere."""
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    # A result below the smallest normal number rounds to a multiple of 2^-133
    # (bf16) or 2^-149: the absolute term.
    bound = err + half_step * got.abs() + 2.0 ** -133
    bad = (got - want).abs() > bound
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / bound).max()))
