"""Definition of rows in codes of 4 and 8 bits, in float64 by search in the table of values, and bounds for
the decode steps on caches of such rows.

What a code stands for is exact (a power of two times a value of four bits), so writing has one right
answer and reading back has no error.  A decode step's products are exact operands summed in
float32: with bf16 queries D terms a score, with float32 ones 3 D (three bf16 parts of q, exact
together), C and 3 C terms in the output; bf16 weights are rounded by half a step u, float32 ones are
not.  As in attention_ref.rows, with A the largest scale sum |q k|, a weight is off by at most the
relative e = 2^-24 (2 (n D + 4) A + n C + 32), n = 1 or 3, and o by (2 e + w) sum p |v| + u |o|, w = u for bf16
and 2^-23 for float32 (what is lost when three parts of a weight end below float32's last bit)."""
import torch

from tests.attention_ref import F32, half_step

GRID = {4: [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
        8: [j / 512 for j in range(8)] + [(8 + j) * 2.0 ** (e - 10) for e in range(1, 16) for j in range(8)][:-1]}
MOST, SCALES = {4: 7.0, 8: 464.0}, {4: range(-115, 126), 8: range(-115, 120)}


def written(x, bits):
    """(values, codes, scales) of rows x [..., D] on the CPU: values float64, the others uint8 as stored."""
    x = x.detach().cpu().double()
    d = x.shape[-1]
    x = x.reshape(-1, d // 32, 32)
    grid = torch.tensor(GRID[bits], dtype=torch.float64)
    steps = torch.tensor([2.0 ** e for e in SCALES[bits]], dtype=torch.float64)
    big = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    at = torch.searchsorted(MOST[bits] * steps, torch.where(fine, big, 0.0)).clamp(max=len(steps) - 1)
    a = torch.where(fine[..., None], x.abs(), 0.0) / steps[at][..., None]
    over = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)          # grid[over - 1] <= a <= grid[over], or past the end
    lo, hi = a - grid[over - 1], grid[over] - a
    code = torch.where((lo > hi) | ((lo == hi) & (over % 2 == 0)), over, over - 1)
    neg = torch.signbit(x)
    value = torch.where(neg, -1.0, 1.0) * grid[code] * steps[at][..., None]
    value = torch.where(fine[..., None], value, torch.nan).reshape(-1, d)
    code = torch.where(fine[..., None], code + neg * (1 << (bits - 1)), 0).reshape(-1, d)
    if bits == 4:
        code = code[:, 0::2] | code[:, 1::2] << 4
    scale = torch.where(fine, at + 127 + SCALES[bits][0], 255)
    return value, code.to(torch.uint8), scale.to(torch.uint8)


def values(codes, scales):
    """Float64 values of codes [..., D*bits/8] and scales [..., D/32], on the CPU."""
    codes, scales = codes.cpu().long(), scales.cpu().long()
    d = 32 * scales.shape[-1]
    bits = codes.shape[-1] * 8 // d
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    half = 1 << (bits - 1)
    grid = torch.tensor(GRID[bits] + ([torch.nan] if bits == 8 else []), dtype=torch.float64)
    up = torch.tensor([2.0 ** (s - 127) for s in range(255)] + [torch.nan], dtype=torch.float64)
    x = grid[codes % half] * torch.where(codes >= half, -1.0, 1.0)
    return (x.unflatten(-1, (-1, 32)) * up[scales][..., None]).flatten(-2)


def rows(q, k, v, live, scale):
    """One query [D] over the live rows of k, v [C,D] (float64 values): o, its bound, weights, their bound."""
    C, D = k.shape
    u = half_step(q.dtype)
    n, w = (1, u) if q.dtype == torch.bfloat16 else (3, 2 * F32)
    qq = q.double()
    kk, vv = torch.where(live[:, None], k, 0.0), torch.where(live[:, None], v, 0.0)
    s = (kk @ qq * scale).masked_fill(~live, -torch.inf)
    p = torch.softmax(s, 0)
    A = (kk.abs() @ qq.abs() * scale).amax()
    e = F32 * (2 * (n * D + 4) * A + n * C + 32)
    o = p @ vv
    return o, (2 * e + w) * (p @ vv.abs()) + u * o.abs(), p, 2 * e * p
