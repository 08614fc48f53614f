"""Float64 definitions of the attention operators of fixed memory, with bounds on the error that
the kernels' roundings may cause.

Kernels: q, k, v and dO enter as given (exact in the reference), products accumulate in float32,
the softmax weights and the score gradients are rounded once to the operand type as operands of
the next product, results once at the end.  With u the half step of the type
(torch.finfo(t).eps / 2) and A = max scale * sum_i |q_i k_i| over a token's keys, a weight
p = exp(s - lse) computed in float32 is off by at most the relative
    e = 2^-24 (2 (D + 4) A + n + 16)
(D-term dot products in s and again in lse, the rounded product s * log2 e and the exponential,
an n-term sum), so
    |o'  - o|  <= (2 e + u) sum p |v| + u |o|
    |dv' - dv| <= (2 e + u) sum p |dO| + u |dv|
and for ds = p (dp - delta), with delta taken from the rounded o,
    r = |dO| . |o' - o| + 2^-24 (D + 4) (|dO| . |v| + |dO| . |o|)        (dp - delta)
    |ds' - ds| <= p r + (2 e + u) |ds|
    |dq' - dq| <= scale sum |ds' - ds| |k| + 2^-24 n scale sum |ds| |k| + u |dq|,   dk alike.
Below float32's normal range (f = 2^-126) a value counts as zero, off by at most f: a weight by f,
so ds by f (1 + |dp| + |delta|), and every result by f once more (a weight of 1e-56, whose
true dk is 1e-55, gives an exact zero).
"""
import math

import torch

F32 = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dt):
    return torch.finfo(dt).eps / 2


def visible(T, window, sinks, n, dev):
    t = torch.arange(T, device=dev)
    d = t[:, None] - t[None, :]
    return (d >= 0) & ((d < window) | (t[None, :] < sinks)) & (t[:, None] < n) & (t[None, :] < n)


def swa(q, k, v, window, sinks, scale, lens, dO=None):
    """{name: (value, bound)} of o, lse and with dO of dq, dk, dv, in float64."""
    B, Hq, T, D = q.shape
    Hkv, dev, u = k.shape[1], q.device, half_step(q.dtype)
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=dev)  # noqa: E731
    out = {"o": (z(q), z(q)), "lse": (torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=dev),
                                      torch.zeros((B, Hq, T), dtype=torch.float64, device=dev))}
    if dO is not None:
        out.update(dq=(z(q), z(q)), dk=(z(k), z(k)), dv=(z(k), z(k)))
    for b in range(B):
        n = T if lens is None else max(0, min(T, int(lens[b])))
        if n == 0:
            continue
        see = visible(n, window, sinks, n, dev)
        for h in range(Hq):
            qq, kk, vv = q[b, h, :n].double(), k[b, h // G, :n].double(), v[b, h // G, :n].double()
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, None])
            o = p @ vv
            A = (qq.abs() @ kk.abs().T * scale).masked_fill(~see, 0.0).amax(-1, keepdim=True)
            e = F32 * (2 * (D + 4) * A + n + 16)
            to = (2 * e + u) * (p @ vv.abs()) + u * o.abs() + TINY * (1 + vv.abs().sum(0))
            out["o"][0][b, h, :n], out["o"][1][b, h, :n] = o, to
            out["lse"][0][b, h, :n], out["lse"][1][b, h, :n] = lse, e[:, 0] + 4 * F32 * lse.abs()
            if dO is None:
                continue
            g = dO[b, h, :n].double()
            dp = g @ vv.T
            ds = p * (dp - (g * o).sum(-1, keepdim=True))
            r = (g.abs() * to).sum(-1, keepdim=True) + F32 * (D + 4) * (g.abs() @ vv.abs().T +
                                                                       (g.abs() * o.abs()).sum(-1, keepdim=True))
            tds = p * r + (2 * e + u + n * F32) * ds.abs() + TINY * see * (1 + dp.abs() + (g * o).sum(-1, keepdim=True).abs())
            out["dq"][0][b, h, :n] = scale * ds @ kk
            out["dq"][1][b, h, :n] = scale * tds @ kk.abs()
            out["dk"][0][b, h // G, :n] += scale * ds.T @ qq
            out["dk"][1][b, h // G, :n] += scale * tds.T @ qq.abs()
            out["dv"][0][b, h // G, :n] += p.T @ g
            out["dv"][1][b, h // G, :n] += (p * (2 * e + u + n * F32) + TINY * see).T @ g.abs()
    if dO is not None:
        for name in ("dq", "dk", "dv"):
            out[name] = (out[name][0], out[name][1] + u * out[name][0].abs() + TINY * (out[name][1] > 0))
    return out


def weights(q, k, window, sinks, scale, lens):
    """Column sums of the weights, and their bound (lse rounded to float32 on the way)."""
    B, Hq, T, D = q.shape
    Hkv, dev = k.shape[1], q.device
    scale = D ** -0.5 if scale is None else scale
    a = torch.zeros((B, Hkv, T), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(a)
    for b in range(B):
        n = T if lens is None else max(0, min(T, int(lens[b])))
        if n == 0:
            continue
        see = visible(n, window, sinks, n, dev)
        for h in range(Hq):
            qq, kk = q[b, h, :n].double(), k[b, h * Hkv // Hq, :n].double()
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - lse)
            A = (qq.abs() @ kk.abs().T * scale).masked_fill(~see, 0.0).amax(-1, keepdim=True)
            e = F32 * (2 * (D + 4) * A + 2 * n * (Hq // Hkv) + 16 + 4 * lse.abs())
            a[b, h * Hkv // Hq, :n] += p.sum(0)
            tol[b, h * Hkv // Hq, :n] += (2 * e * p).sum(0)
    return a, tol


def rows(q, k, v, live, scale):
    """One query [D] over the live rows of k, v [C,D]: o, its bound, weights, their bound."""
    C, D = k.shape
    u = half_step(q.dtype)
    qq, kk, vv = q.double(), k.double(), v.double()
    kk = torch.where(live[:, None], kk, 0.0)
    vv = torch.where(live[:, None], vv, 0.0)
    s = (kk @ qq * scale).masked_fill(~live, -math.inf)
    p = torch.softmax(s, 0)
    A = (kk.abs() @ qq.abs() * scale).amax()
    e = F32 * (2 * (D + 4) * A + C + 32)
    o = p @ vv
    return o, (2 * e + u) * (p @ vv.abs()) + u * o.abs(), p, 2 * e * p


def within(x, ref, what):
    value, bound = ref
    x = x.double()
    assert x.shape == value.shape, what
    inf = torch.isinf(value)
    assert torch.equal(x[inf], value[inf]), what
    d = torch.where(inf, torch.zeros_like(x), (x - torch.where(inf, torch.zeros_like(value), value)).abs())
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float((d / bound.clamp(min=1e-300))[bad].max()):.3g} times at "
                           f"{torch.nonzero(bad)[0].tolist()}")
