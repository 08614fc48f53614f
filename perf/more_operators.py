"""Timed cases of caches held in 4 or 8 bits: writing them, reading them back, attention over them.

A row of D values is held in blocks of 32 along D: every block has one scale byte s, for 2^(s - 127),
and every value a code of 4 bits (sign, exponents of 2, 1 bit behind the point: 0 .5 1 1.5 2 3 4 6, two
codes a byte, the first in the low half) or of 8 (sign, 4 and 3 bits, up to 448, the least 2^-9).
The scale is the least power of two, 2^-115 or more, at which the block's largest value is off by no
more than half a step: at most 7 (4 bits) or 464 (8 bits) times it, what is past the last code being
held as that code.  Values go to the nearest code, of two equally near ones to the even one.  A block
with a value that is not finite has scale byte 255 and codes 0, and is read as not a number.

The operators:

  rows    rows of a tensor written in codes and scales, and read back
  fill    the ring cache of sinks + window slots of a prompt, and its read back
  ring    attention of one new token on a ring cache, which takes the token's k and v first
  keep    the cache of a fixed number of slots made from a prompt by its tokens' weights, and its read back
  evict   one new token on that cache: it takes an empty slot or that of the least weight,
          attends, and adds its attention weights to the cache's

`run` computes them in plain torch operations in 32 bits, or calls the library (`own`).  Steps on a cache
return its codes and scales as they stand, whole numbers that have one right value each.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# bits of a code: bits behind the point, least exponent of a full mantissa, largest value, and the
# largest multiple of the scale that a block may hold
FORMATS = {4: (1, 0, 6.0, 7.0), 8: (3, -6, 448.0, 464.0)}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few rows, for a cache that the user's program keeps: launch latency
        dict(name="rows_few", op="rows", B=1, Hkv=4, T=100, D=128, bits=4, dtype="bf16"),
        # the keys of a batch of long prompts in 8 bits: bandwidth both ways
        dict(name="rows_many", op="rows", B=8, Hkv=4, T=16384, D=128, bits=8, dtype="bf16"),
        # a short prompt of one conversation; a padded batch of long ones
        dict(name="fill_short", op="fill", B=1, Hkv=4, T=500, D=128, window=256, sinks=4, ragged=False, bits=4, dtype="bf16"),
        dict(name="fill_batch", op="fill", B=32, Hkv=4, T=8192, D=128, window=4096, sinks=4, ragged=True, bits=4,
             dtype="bf16"),
        # one conversation, one token: latency
        dict(name="ring_one", op="ring", B=1, Hq=16, Hkv=4, D=128, window=1024, sinks=4, ragged=False, bits=4, dtype="bf16"),
        # a full serving batch with long windows: the cache's bandwidth
        dict(name="ring_batch", op="ring", B=256, Hq=16, Hkv=4, D=128, window=4096, sinks=4, ragged=True, bits=4,
             dtype="bf16"),
        # a batch of odd sizes in full precision on a cache in 8 bits
        dict(name="ring_f32", op="ring", B=33, Hq=14, Hkv=2, D=64, window=1999, sinks=3, ragged=True, bits=8, dtype="f32"),
        # a short prompt into a small cache, and long ones into large caches
        dict(name="keep_short", op="keep", B=1, Hkv=4, T=500, D=128, C=256, sinks=4, recent=32, ragged=False, bits=4,
             dtype="bf16"),
        dict(name="keep_long", op="keep", B=8, Hkv=4, T=32768, D=128, C=4096, sinks=4, recent=1024, ragged=True, bits=4,
             dtype="bf16"),
        # one conversation on a small cache; a serving batch on large ones, some still filling
        dict(name="evict_one", op="evict", B=1, Hq=16, Hkv=4, D=128, C=512, sinks=4, recent=64, ragged=False, bits=4,
             dtype="bf16"),
        dict(name="evict_batch", op="evict", B=64, Hq=16, Hkv=4, D=128, C=2048, sinks=4, recent=256, ragged=True, bits=4,
             dtype="bf16"),
        # the same in 8 bits, with narrow heads, many of them on a key head, and odd sizes
        dict(name="evict_wide", op="evict", B=17, Hq=40, Hkv=2, D=64, C=1001, sinks=1, recent=100, ragged=True, bits=8,
             dtype="bf16"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rows", "fill", "ring", "ring", "keep", "evict", "evict"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, B=log_int(1, 32), Hkv=Hkv, D=rng.choice([64, 128]), bits=rng.choice([4, 4, 8]),
             dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op != "rows":
        c["ragged"] = rng.random() < 0.5
    if op in ("ring", "evict"):
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 20])
    if op == "rows":
        c.update(T=log_int(1, 8192))
    elif op == "fill":
        c.update(T=log_int(1, 8192), window=log_int(16, 4096), sinks=rng.choice([0, 1, 4, 7, 64]))
    elif op == "ring":
        c.update(window=log_int(16, 8192), sinks=rng.choice([0, 1, 4, 7, 64]))
    elif op == "keep":
        C = log_int(16, 4096)
        c.update(T=log_int(16, 16384), C=C, sinks=rng.randint(0, C // 8), recent=rng.randint(1, C // 2))
        c["B"] = min(c["B"], 16)
    else:
        C = log_int(16, 4096)
        c.update(C=C, sinks=rng.randint(0, C // 8), recent=rng.randint(1, C // 2))
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev, dt, bits = DEVICE, DTYPES[case["dtype"]], case["bits"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    # a few channels of keys are far larger than the rest, as in trained models
    wide = torch.exp(torch.randn(Hkv, 1, D, generator=gen, device=dev))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def rows(n):
        return (normal(B, Hkv, n, D) * wide).to(dt), normal(B, Hkv, n, D).to(dt)

    def between(lo, hi, n):       # n whole numbers of [lo, hi]
        return torch.randint(lo, hi + 1, (n,), generator=gen, device=dev, dtype=torch.int32)

    def held(n):                  # a cache of n slots that holds tokens, in codes and scales
        kc, ks, vc, vs = _codes(normal(B, Hkv, n, D) * wide, bits) + _codes(normal(B, Hkv, n, D), bits)
        return dict(k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs)

    def vacant(n):
        code = torch.zeros(B, Hkv, n, D * bits // 8, device=dev, dtype=torch.uint8)
        scale = torch.zeros(B, Hkv, n, D // 32, device=dev, dtype=torch.uint8)
        return dict(k_codes=code, k_scales=scale, v_codes=code.clone(), v_scales=scale.clone())

    def one():                    # the new token
        k, v = rows(1)
        return dict(q=(normal(B, case["Hq"], D) * wide.mean().rsqrt()).to(dt), k=k[:, :, 0].contiguous(), v=v[:, :, 0].contiguous())

    s = dict(case)
    if case["op"] == "rows":
        s["x"] = rows(case["T"])[0]
    elif case["op"] in ("fill", "keep"):
        T = case["T"]
        s["k"], s["v"] = rows(T)
        s["lens"] = between((T + 1) // 2, T, B) if case["ragged"] else None
        if case["op"] == "fill":
            s.update(vacant(case["window"] + case["sinks"]))
        else:
            C = case["C"]
            # accumulated weights: positive, a few heavy tokens
            s["weights"] = torch.exp(2 * normal(B, Hkv, T))
            s.update(vacant(C), cache_w=torch.zeros(B, Hkv, C, device=dev),
                     cache_pos=torch.zeros(B, Hkv, C, device=dev, dtype=torch.int32))
    elif case["op"] == "ring":
        C = case["window"] + case["sinks"]
        s.update(held(C), **one())
        # tokens before this one: sequences that fill their window, or (ragged) some that do not
        s["pos"] = between(C // 2 if case["ragged"] else 2 * C, 4 * C, B)
    else:
        C = case["C"]
        s.update(held(C), **one())
        s["pos"] = between(C // 2 if case["ragged"] else 2 * C, 4 * C, B)
        # the positions a slot holds: its own index while the cache fills; after that the first
        # tokens, the recent ones, and a share of those between, in order
        slot = torch.arange(C, device=dev)[None, None]
        p = s["pos"].long()[:, None, None]
        old = C - case["sinks"] - (case["recent"] - 1)       # slots of neither kind
        gap = (p - case["recent"] + 1 - case["sinks"]).clamp(min=1)
        middle = case["sinks"] + (slot - case["sinks"]) * gap // max(old, 1)
        at = torch.where(slot < case["sinks"], slot, torch.where(slot < case["sinks"] + old, middle, p - C + slot))
        at = torch.where(p >= C, at, torch.where(slot < p, slot, torch.full_like(slot, -1)))
        s["cache_pos"] = at.expand(B, Hkv, C).to(torch.int32).contiguous()
        s["cache_w"] = torch.where(s["cache_pos"] >= 0, torch.exp(normal(B, Hkv, C)), 0.0)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"rows": _rows, "fill": _fill, "ring": _ring, "keep": _keep, "evict": _evict}[s["op"]](s)


def _own(s):
    from chunk_gated_delta_amd import carve
    if s["op"] == "rows":
        codes, scales = carve.mx_quant(s["x"], bits=s["bits"])
        return carve.mx_dequant(codes, scales, dtype=s["x"].dtype)
    rows = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    if s["op"] == "ring":
        o = carve.swa_decode_mx(s["q"], s["k"], s["v"], rows, s["pos"], window=s["window"], sinks=s["sinks"])
        return (o,) + rows
    if s["op"] == "evict":
        cache = rows + (s["cache_w"], s["cache_pos"])
        o, slot = carve.budget_decode_mx(s["q"], s["k"], s["v"], cache, s["pos"], sinks=s["sinks"], recent=s["recent"])
        return (o, slot) + cache
    if s["op"] == "fill":
        carve.swa_fill_mx(s["k"], s["v"], rows, window=s["window"], sinks=s["sinks"], lens=s["lens"])
        rest = ()
    else:
        rest = (s["cache_w"], s["cache_pos"])
        carve.budget_keep_mx(s["k"], s["v"], s["weights"], s["C"], sinks=s["sinks"], recent=s["recent"], lens=s["lens"],
                             cache=rows + rest)
    dt = s["k"].dtype
    return (carve.mx_dequant(*rows[:2], dtype=dt), carve.mx_dequant(*rows[2:], dtype=dt)) + rest


# ---- plain forms: 32 bits throughout, rounded once at the end
def _power(e):
    """2^e in 32 bits, for whole numbers e of [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x, bits):
    """Codes and scales, both uint8, of rows x [..., D]."""
    mant, least, top, most = FORMATS[bits]
    x = x.float().unflatten(-1, (-1, 32))
    big = x.abs().amax(-1)
    part, e = torch.frexp(big)                                             # big = part 2^e, part in [1/2, 1)
    most, lead = math.frexp(most)
    e = (e - lead + (part > most).int()).clamp(-115, 128 - lead)
    ok = torch.isfinite(big)
    a = (x.abs() * _power(-e)[..., None]).clamp(max=top)
    up = torch.where(a > 0, torch.frexp(a)[1] - 1, least).clamp(min=least)
    n = torch.round(a * _power(mant - up))                             # whole steps, ties to even
    code = n.nan_to_num(0).int() + (up - least) * (1 << mant) + torch.signbit(x).int() * (1 << (bits - 1))
    code = torch.where(ok[..., None], code, 0).flatten(-2)
    scale = torch.where(ok, e + 127, 255).to(torch.uint8)
    if bits == 4:
        code = code[..., 0::2] + 16 * code[..., 1::2]
    return code.to(torch.uint8), scale


def _table(bits, dev):
    """The value of every code of so many bits."""
    mant, least, _, _ = FORMATS[bits]
    code = torch.arange(1 << bits, device=dev)
    size = code % (1 << (bits - 1))
    up, part = size >> mant, size % (1 << mant)
    value = (part + torch.where(up > 0, 1 << mant, 0)) * _power(up.clamp(min=1) - 1 + least - mant)
    if bits == 8:                                                          # the last code stands for no number
        value = torch.where(size < 127, value, math.nan)
    return torch.where(code >= 1 << (bits - 1), -value, value)


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    bits = codes.shape[-1] * 8 // (scales.shape[-1] * 32)
    if bits == 4:
        codes = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
    x = _table(bits, codes.device)[codes.int()].unflatten(-1, (-1, 32))
    up = torch.arange(256, device=codes.device)
    up = torch.where(up < 255, _power((up - 127).clamp(-126, 127)) * torch.where(up > 0, 1.0, 0.5), math.nan)
    return (x * up[scales.int()][..., None]).flatten(-2)


def _rows(s):
    return _values(*_codes(s["x"], s["bits"])).to(s["x"].dtype)


def _fill(s):
    k, W, ns, C = s["k"], s["window"], s["sinks"], s["window"] + s["sinks"]
    B, Hkv, T, D = k.shape
    slot = torch.arange(C, device=k.device)
    n = torch.full((B, 1), T, device=k.device) if s["lens"] is None else s["lens"].long().view(B, 1)
    last = n - 1                                                           # the last token of every slot's residue
    p = torch.where(slot < ns, slot, last - (last - slot) % W)
    has = (p <= last) & (p >= torch.where(slot < ns, 0, ns))
    at = torch.where(has, p, 0)[:, None, :, None].expand(B, Hkv, C, D)
    for name in ("k", "v"):
        for part, new in zip(("_codes", "_scales"), _codes(torch.gather(s[name], 2, at), s["bits"])):
            cache = s[name + part]
            cache.copy_(torch.where(has[:, None, :, None], new, cache))
    return tuple(_values(s[x + "_codes"], s[x + "_scales"]).to(k.dtype) for x in ("k", "v"))


def _attend(s, live):
    """One query per head against the cached rows: o [B,Hq,D] and p [B,Hkv,G,C], in 32 bits."""
    q = s["q"]
    B, Hq, D = q.shape
    Hkv = s["k"].shape[1]
    k = _values(s["k_codes"], s["k_scales"])
    x = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), k.transpose(-1, -2).contiguous()) / math.sqrt(D)
    x = x.masked_fill(~live[:, :, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    return torch.matmul(p, _values(s["v_codes"], s["v_scales"])).reshape(B, Hq, D), p


def _ring(s):
    pos, ns, W = s["pos"].long(), s["sinks"], s["window"]
    B, Hkv, D = s["k"].shape
    slot = torch.where(pos < ns, pos, ns + (pos - ns) % W)
    b = torch.arange(B, device=pos.device)
    for name in ("k", "v"):
        for part, new in zip(("_codes", "_scales"), _codes(s[name], s["bits"])):
            s[name + part][b, :, slot] = new
    live = torch.arange(W + ns, device=pos.device) <= pos[:, None]         # a ring holds its last tokens from slot 0 up
    o, _ = _attend(s, live[:, None].expand(B, Hkv, W + ns))
    return o.to(s["q"].dtype), s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]


def _keep(s):
    w, C, dev = s["weights"], s["C"], s["weights"].device
    B, Hkv, T = w.shape
    t = torch.arange(T, device=dev)
    n = torch.full((B, 1, 1), T, device=dev) if s["lens"] is None else s["lens"].long().view(B, 1, 1)
    safe = (t < s["sinks"]) | (t >= n - s["recent"])
    key = torch.where(t >= n, -math.inf, torch.where(safe, math.inf, w))
    m = min(C, T)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :m]  # equal weights: the lowest position first
    at = torch.sort(torch.where(torch.arange(m, device=dev) < n, order, T), dim=-1)[0]
    has = at < T
    at = torch.where(has, at, 0)
    s["cache_pos"].fill_(-1)
    s["cache_w"].zero_()
    s["cache_pos"][..., :m] = torch.where(has, at, -1).to(torch.int32)
    s["cache_w"][..., :m] = torch.where(has, torch.gather(w, -1, at), 0.0)
    rows = at[..., None].expand(B, Hkv, m, s["k"].shape[-1])
    for name in ("k", "v"):
        for part, new in zip(("_codes", "_scales"), _codes(torch.gather(s[name], 2, rows), s["bits"])):
            cache = s[name + part]
            cache[:, :, :m] = torch.where(has[..., None], new, cache[:, :, :m])
    return tuple(_values(s[x + "_codes"], s[x + "_scales"]).to(s["k"].dtype) for x in ("k", "v")) + (s["cache_w"], s["cache_pos"])


def _evict(s):
    cw, cp = s["cache_w"], s["cache_pos"]
    B, Hkv, C = cw.shape
    pos = s["pos"].view(B, 1, 1)
    # the slot: that which holds this position already, else an empty one, else the least
    # weight among those that are neither first nor recent; the lowest of equals
    safe = (cp < s["sinks"]) | (cp > pos - s["recent"])
    key = torch.where(safe, math.inf, cw)
    key = torch.where(cp < 0, -1.0, key)
    key = torch.where(cp == pos, -2.0, key)
    index = torch.arange(C, device=cw.device)
    slot = torch.where(key == key.amin(-1, keepdim=True), index, C).amin(-1)
    at = slot[..., None]
    for name in ("k", "v"):
        for part, new in zip(("_codes", "_scales"), _codes(s[name], s["bits"])):
            s[name + part].scatter_(2, at[..., None].expand(B, Hkv, 1, new.shape[-1]), new[:, :, None])
    cp.scatter_(2, at, pos.expand(B, Hkv, 1))
    cw.scatter_(2, at, 0.0)
    o, p = _attend(s, cp >= 0)
    cw += p.sum(2)
    return (o.to(s["q"].dtype), slot.to(torch.int32), s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], cw, cp)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    held = D * case["bits"] // 8 + D // 32                                 # bytes of a row in the cache
    share = 0.75 if case.get("ragged") else 1.0
    if case["op"] == "rows":                                               # written, then read back
        return {"bytes": B * Hkv * case["T"] * 2 * (D * es + held), "flops": 4 * B * Hkv * case["T"] * D}
    if case["op"] in ("fill", "keep"):
        C = case["window"] + case["sinks"] if case["op"] == "fill" else case["C"]
        rows = 2 * B * Hkv * min(C, case["T"])
        out = 2 * B * Hkv * C * (held + D * es)                            # the whole cache is read back
        more = B * Hkv * (case["T"] * 4 * share + C * 8) if case["op"] == "keep" else 0
        return {"bytes": int(rows * (D * es + held) + out + more), "flops": 4 * rows * D}
    C = case["window"] + case["sinks"] if case["op"] == "ring" else case["C"]
    live = int(C * (0.95 if case.get("ragged") else 1.0))                  # some sequences are still short
    Hq = case["Hq"]
    more = 12 * B * Hkv * C if case["op"] == "evict" else 0
    return {"bytes": B * Hkv * live * 2 * held + more + (2 * Hq + 2 * Hkv) * B * D * es, "flops": 4 * D * B * Hq * live}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rows": _exact_rows, "fill": _exact_fill, "ring": _exact_ring, "keep": _exact_keep, "evict": _exact_evict}[case["op"]](s)


def _grid(bits):
    """The values of the codes without their sign, written out."""
    if bits == 4:
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return [j * 2.0 ** -9 for j in range(8)] + [(8 + j) * 2.0 ** (e - 10) for e in range(1, 16) for j in range(8)][:119]


def _written(x, bits):
    """(values that the rows x stand for once written, codes, scales), by search in the table of values."""
    grid = torch.tensor(_grid(bits), dtype=torch.float64, device=x.device)
    x = x.double().unflatten(-1, (-1, 32))
    big = x.abs().amax(-1, keepdim=True)
    up = torch.tensor([2.0 ** e for e in range(-115, 126 if bits == 4 else 120)], dtype=torch.float64, device=x.device)
    at = torch.searchsorted(up * (7.0 if bits == 4 else 464.0), big).clamp(max=len(up) - 1)
    a = x.abs() / up[at]
    middle = (grid[1:] + grid[:-1]) / 2
    code = torch.searchsorted(middle, a)                                   # of two equally near codes the lower
    tie = (code < len(middle)) & (middle[code.clamp(max=len(middle) - 1)] == a)
    code = code + (tie & (code % 2 == 1))
    neg = torch.signbit(x)
    value = (torch.where(neg, -grid[code], grid[code]) * up[at]).flatten(-2)
    code = (code + neg * len(grid) if bits == 4 else code + neg * 128).flatten(-2)
    if bits == 4:
        code = code[..., 0::2] + 16 * code[..., 1::2]
    return value, code.to(torch.uint8), (at[..., 0] + 12).to(torch.uint8)


def _read(codes, scales):
    """Float64 values of codes and scales."""
    bits = codes.shape[-1] * 8 // (scales.shape[-1] * 32)
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    grid = torch.tensor(_grid(bits), dtype=torch.float64, device=codes.device)
    half = 8 if bits == 4 else 128
    c = codes.long()
    value = grid[(c % half).clamp(max=len(grid) - 1)] * torch.where(c >= half, -1.0, 1.0)
    up = torch.tensor([2.0 ** (e - 127) for e in range(256)], dtype=torch.float64, device=codes.device)
    return (value.unflatten(-1, (-1, 32)) * up[scales.long()][..., None]).flatten(-2)


def _exact_rows(s):
    return _written(s["x"], s["bits"])[0]


def _exact_fill(s):
    out = []
    for x in (s["k"], s["v"]):
        B, Hkv, T, D = x.shape
        value = _written(x, s["bits"])[0]
        cache = torch.zeros(B, Hkv, s["window"] + s["sinks"], D, dtype=torch.float64, device=x.device)
        for b in range(B):
            n = T if s["lens"] is None else int(s["lens"][b])
            for p in list(range(min(s["sinks"], n))) + list(range(max(s["sinks"], n - s["window"]), n)):
                at = p if p < s["sinks"] else s["sinks"] + (p - s["sinks"]) % s["window"]
                cache[b, :, at] = value[b, :, p]
        out.append(cache)
    return tuple(out)


def _exact_keep(s):
    B, Hkv, T = s["weights"].shape
    C, dev = s["C"], s["weights"].device
    rows = [_written(s[x], s["bits"])[0] for x in ("k", "v")]
    out = [torch.zeros(B, Hkv, C, rows[0].shape[-1], dtype=torch.float64, device=dev) for _ in rows]
    cw = torch.zeros(B, Hkv, C, dtype=torch.float64, device=dev)
    held = torch.full((B, Hkv, C), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        n = T if s["lens"] is None else int(s["lens"][b])
        safe = set(range(min(s["sinks"], n))) | set(range(max(0, n - s["recent"]), n))
        for h in range(Hkv):
            w = s["weights"][b, h].tolist()
            rest = sorted((t for t in range(n) if t not in safe), key=lambda t: (-w[t], t))
            at = torch.tensor(sorted(list(safe) + rest[:max(0, C - len(safe))]), device=dev)
            m = len(at)
            out[0][b, h, :m], out[1][b, h, :m] = rows[0][b, h, at], rows[1][b, h, at]
            cw[b, h, :m], held[b, h, :m] = s["weights"][b, h, at].double(), at.to(torch.int32)
    return out[0], out[1], cw, held


def _exact_step(s, b, at, live):
    """Sequence b's token written to slot `at` (one for every key head) of copies in s: (o, p) over the live slots."""
    for name in ("k", "v"):
        _, code, scale = _written(s[name][b], s["bits"])
        for h in range(len(at)):
            s[name + "_codes"][b, h, at[h]], s[name + "_scales"][b, h, at[h]] = code[h], scale[h]
    k, v = (_read(s[x + "_codes"][b], s[x + "_scales"][b]) for x in ("k", "v"))
    Hkv, C, D = k.shape
    q = s["q"][b].double().view(Hkv, -1, D)
    x = torch.matmul(q, k.transpose(1, 2).contiguous()) * D ** -0.5
    p = torch.softmax(x.masked_fill(~live[:, None], -math.inf), -1)
    return torch.matmul(p, v).view(-1, D), p


def _exact_ring(s):
    s = {n: x.clone() if n.endswith(("_codes", "_scales")) else x for n, x in s.items()}
    B, Hkv, C = s["k_codes"].shape[:3]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, p in enumerate(s["pos"].tolist()):
        at = p if p < s["sinks"] else s["sinks"] + (p - s["sinks"]) % s["window"]
        live = torch.arange(C, device=o.device) < min(p + 1, C)
        o[b], _ = _exact_step(s, b, [at] * Hkv, live.expand(Hkv, C))
    return o, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]


def _exact_evict(s):
    s = {n: x.clone() if n.endswith(("_codes", "_scales", "_pos")) else x for n, x in s.items()}
    cp, cw = s["cache_pos"], s["cache_w"].double()
    B, Hkv, C = cp.shape
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    slot = torch.zeros(B, Hkv, dtype=torch.int32, device=o.device)
    for b, p in enumerate(s["pos"].tolist()):
        at = []
        for h in range(Hkv):
            held, w = cp[b, h].tolist(), cw[b, h].tolist()
            if p in held:
                at.append(held.index(p))
            elif min(held) < 0:
                at.append(next(j for j in range(C) if held[j] < 0))
            else:
                at.append(min((j for j in range(C) if s["sinks"] <= held[j] <= p - s["recent"]), key=lambda j: (w[j], j)))
            cp[b, h, at[h]], cw[b, h, at[h]] = p, 0.0
        slot[b] = torch.tensor(at, dtype=torch.int32)
        o[b], pr = _exact_step(s, b, at, cp[b] >= 0)
        cw[b] += pr.sum(1)
    return o, slot, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], cw, cp
