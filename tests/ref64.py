"""Plain 64-bit forms of the rotation, packed causal attention and its gradient, and the adapters'
orthogonalised update, with the rounding bounds their tests use.

Bounds.  A rounding to BF16 is off by at most H = 2^-8 of the value, one to FP32 by 2^-24; a sum
of n FP32 products in any order, truncating or rounding, by (n + 8) 2^-22 of the sum of magnitudes
(2^-22 leaves room for the tensor core's truncation and for the exponential's 2^-22).
Below 2^-126 those relative errors do not hold: FP32 and BF16 have no normal numbers there, and an
exponential or a product may come out as zero.  Such a value is off by less than T = 2^-125 itself,
and a sum by that much times its other factors."""
import math

import torch

H = 2.0 ** -8
F = 2.0 ** -24
U = 2.0 ** -22
T = 2.0 ** -125
NS = (3.4445, -4.7750, 2.0315)


def rope(x, pos, inv_freq, heads, inverse=False):
    """(y, bound): the angle is off by pi 2^-24 at most, its cosine and sine by two FP32 steps, the two
    products and the sum by one each."""
    M, cols = x.shape
    half = cols // heads // 2
    t = pos.double()[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64, device=x.device)
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None] * (-1 if inverse else 1)
    z = x.double().reshape(M, heads, 2, half)
    a, b = z[:, :, 0], z[:, :, 1]
    y = torch.stack([a * c - b * s, b * c + a * s], 2).reshape(M, cols)
    size = (a.abs() + b.abs())[:, :, None].expand(-1, -1, 2, -1).reshape(M, cols)
    return y, H * y.abs() + 8 * 2.0 ** -23 * size


def spans(starts):
    return [(a, b) for a, b in zip(starts, starts[1:]) if b > a]


def attention(q, k, v, starts, heads, kv_heads, scale, do=None, o=None):
    """Forward: {o, lse}, and with the gradient do {dq, dk, dv} (delta from the given o), each a pair
    (value, bound), zero outside the sequences."""
    M, D = q.shape[0], q.shape[1] // heads
    group = heads // kv_heads
    z = lambda n: torch.zeros((M, n, D), dtype=torch.float64, device=q.device)
    out = {"o": (z(heads), z(heads)), "lse": tuple(torch.zeros((heads, M), dtype=torch.float64, device=q.device)
                                                   for _ in range(2))}
    if do is not None:
        out |= {"dq": (z(heads), z(heads)), "dk": (z(kv_heads), z(kv_heads)), "dv": (z(kv_heads), z(kv_heads))}
    part = lambda t, n, a, b, h: t[a:b].double().reshape(b - a, n, D)[:, h]
    for a, b in spans(starts):
        n = b - a
        hide = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
        for h in range(heads):
            g = h // group
            Q, K, V = part(q, heads, a, b, h), part(k, kv_heads, a, b, g), part(v, kv_heads, a, b, g)
            S = (Q @ K.T) * scale
            # error of a score in FP32, and of its distance to the row's log-sum
            eS = (D + 8) * U * abs(scale) * (Q.abs() @ K.abs().T)
            S = S.masked_fill(hide, -math.inf)
            lse = torch.logsumexp(S, -1)
            P = torch.exp(S - lse[:, None])
            eL = (P * eS).sum(-1) + n * U + U * lse.abs()
            rel = (eS + eL[:, None] + 8 * U * S.masked_fill(hide, 0).abs())     # relative error of P
            out["lse"][0][h, a:b] = lse
            out["lse"][1][h, a:b] = 2 * eL + 4 * U * (1 + lse.abs())
            out["o"][0][a:b, h] = O = P @ V
            PV = P @ V.abs()
            out["o"][1][a:b, h] = H * O.abs() + 1.02 * ((H + n * U) * PV + (P * rel + T) @ V.abs()) + T
            if do is None:
                continue
            G, Ob = part(do, heads, a, b, h), part(o, heads, a, b, h)
            delta = (G * Ob).sum(-1, keepdim=True)
            dP = G @ V.T
            dS = P * (dP - delta)
            e = (D + 8) * U * (G.abs() @ V.abs().T + (G * Ob).abs().sum(-1, keepdim=True))
            edS = 1.02 * ((H + rel) * dS.abs() + P * e) + T * (1 + (dP - delta).abs())
            many = (n * group + 8) * U                                        # FP32 sums of the products
            out["dq"][0][a:b, h] = scale * (dS @ K)
            out["dq"][1][a:b, h] = abs(scale) * ((edS + many * dS.abs()) @ K.abs())
            out["dk"][0][a:b, g] += scale * (dS.T @ Q)
            out["dk"][1][a:b, g] += abs(scale) * ((edS + many * dS.abs()).T @ Q.abs())
            out["dv"][0][a:b, g] += P.T @ G
            out["dv"][1][a:b, g] += 1.02 * ((H + many + rel) * P + T).T @ G.abs()
    for name in ("dq", "dk", "dv"):
        if name in out:
            out[name][1].add_(H * out[name][0].abs() + T)
    return {name: tuple(t.reshape(M, -1) if name != "lse" else t for t in pair) for name, pair in out.items()}


def orthogonal(u):
    """The Newton-Schulz products of one matrix."""
    tall = u.shape[0] > u.shape[1]
    x = u.T if tall else u
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        s = x @ x.T
        x = NS[0] * x + (NS[1] * s + NS[2] * (s @ s)) @ x
    return x.T if tall else x


def muon(w, g, m, lr, mu, wd, nesterov=True):
    """(m', bound), (W', bound).  u is rounded to FP32 twice (m' and u), by at most e in norm; the
    products' map of u / |u| changes by at most 3.4445^5 = 485 times as much (its steepest slope, at
    zero singular values) and the normalisation doubles it."""
    w, g, m = w.double(), g.double(), m.double()
    m1 = mu * m + g
    u = g + mu * m1 if nesterov else m1
    em = 2 * F * ((mu * m).abs() + g.abs())
    eu = (2 * F * (g.abs() + abs(mu) * m1.abs()) + abs(mu) * em).norm() / max(u.norm().item(), 1e-300)
    x = orthogonal(u)
    step = lr * math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
    w1 = (1 - lr * wd) * w - step * x
    ew = F * w1.abs() + abs(step) * (2 * 485 * eu + F * x.abs()) + 1e-30
    return (m1, em + 1e-45), (w1, ew)


def within(got, pair, what):
    value, bound = pair
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} outside; first {i}: got {got[i].item()!r}, "
                             f"exact {value[i].item()!r}, bound {bound[i].item()!r}; worst error/bound "
                             f"{(err / bound.clamp_min(1e-300)).nan_to_num(nan=math.inf).max().item():.3g}")
