"""Rows in codes of 4 and 8 bits on the GPU: writing and reading back bit for bit, the caches of a prompt, and the
decode steps of both caches against float64 (tests/mx_ref.py states the definition and the bounds)."""
import math

import pytest
import torch

from chunk_gated_delta_amd import carve
from tests import attention_ref as ref
from tests import mx_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def same(x, y):
    """Equal values, not-a-number where the other has it."""
    return torch.equal(torch.isnan(x), torch.isnan(y)) and torch.equal(torch.nan_to_num(x, 7.0), torch.nan_to_num(y, 7.0))


def junk(cache):
    """A cache whose slots hold what must not be read: scale not a number, codes all ones."""
    for x in cache[:4]:
        x.fill_(255)
    return cache


def put(cache, b, h, at, k, v, bits):
    """The definition's k, v rows [n, D] in slots `at` of key head (b, h) of a CPU cache."""
    for i, x in ((0, k), (2, v)):
        _, code, scale = mx_ref.written(x, bits)
        cache[i][b, h, at], cache[i + 1][b, h, at] = code, scale


# ------------------------------------------------------------------ rows
def hard_rows():
    gen = torch.Generator().manual_seed(3)
    def randn(*shape):
        return torch.randn(shape, generator=gen)
    return {"every bf16": torch.arange(-32768, 32768, dtype=torch.int16).view(torch.bfloat16).float().view(-1, 128),
            "bits": torch.randint(-2 ** 31, 2 ** 31 - 1, (500, 128), generator=gen).int().view(torch.float32),
            "ties": torch.round(randn(300, 64) * 8) / 4, "small ties": torch.round(randn(300, 64) * 64) / 2 ** 9,
            "wide": randn(300, 64) * 2.0 ** torch.randint(-140, 127, (300, 1), generator=gen),
            "zeros": torch.tensor([0.0, -0.0]).repeat(5, 48), "few": randn(1, 32), "odd": randn(7, 3, 96)}


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("name", list(hard_rows()))
def test_rows_bit_for_bit(name, bits, dt):
    x = hard_rows()[name].to(DT[dt])
    value, code, scale = mx_ref.written(x, bits)
    codes, scales = carve.mx_quant(x.cuda(), bits=bits)
    assert codes.shape == x.shape[:-1] + (x.shape[-1] * bits // 8,) and scales.shape == x.shape[:-1] + (x.shape[-1] // 32,)
    assert torch.equal(scales.cpu().view(scale.shape), scale)
    assert torch.equal(codes.cpu().view(code.shape), code)
    for out in DT.values():
        y = carve.mx_dequant(codes, scales, dtype=out)
        assert y.dtype == out and y.shape == x.shape
        assert same(y.cpu().double().view(value.shape), value)
    again = carve.mx_quant(y, bits=bits)
    fine = (scales != 255).repeat_interleave(codes.shape[-1] // scales.shape[-1], -1)
    assert torch.equal(again[0][fine], codes[fine]) and torch.equal(again[1], scales)


@pytest.mark.parametrize("bits", [4, 8])
def test_every_code_and_scale_is_read(bits):
    """All bytes of codes with all scale bytes, rounded once to the type."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8 * (8 // bits)).cuda()
    want = mx_ref.values(codes, scales)
    assert same(carve.mx_dequant(codes, scales, dtype=torch.float32).cpu(), want.float())
    assert same(carve.mx_dequant(codes, scales).cpu(), want.float().bfloat16())    # (every value is a float32)


@pytest.mark.parametrize("n", [0, 1, 31, 33, 1000, 4097, 70001])
def test_rows_of_every_number_leave_what_is_behind(n):
    """n blocks, and 64 bytes behind the outputs stay."""
    for bits in (4, 8):
        for dt in DT:
            x = normal((n, 32), dt, n)
            codes = torch.full((n * 4 * bits + 64,), 99, dtype=torch.uint8, device="cuda")
            scales = torch.full((n + 64,), 99, dtype=torch.uint8, device="cuda")
            out = torch.full((n * 32 + 64,), 99.0, dtype=DT[dt], device="cuda")
            c, s, y = codes[:n * 4 * bits].view(n, 4 * bits), scales[:n].view(n, 1), out[:n * 32].view(n, 32)
            carve.mx_quant(x, bits=bits, codes=c, scales=s)
            carve.mx_dequant(c, s, dtype=DT[dt], out=y)
            assert (codes[n * 4 * bits:] == 99).all() and (scales[n:] == 99).all() and (out[n * 32:] == 99).all()
            value, code, scale = mx_ref.written(x[-500:], bits) if n else (x.cpu().double(), c.cpu(), s.cpu())
            assert torch.equal(c[-500:].cpu(), code) and torch.equal(s[-500:].cpu(), scale)
            assert torch.equal(y[-500:].cpu().double(), value)


def test_rows_refuse_what_does_not_fit():
    x = normal((4, 64), "bf16", 1)
    with pytest.raises(ValueError, match="multiple of 32"):
        carve.mx_quant(x[:, :48].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        carve.mx_quant(x[:, :32])
    with pytest.raises(ValueError, match="4 or 8"):
        carve.mx_quant(x, bits=5)
    with pytest.raises(TypeError):
        carve.mx_quant(x.half())
    codes, scales = carve.mx_quant(x)
    with pytest.raises(TypeError):
        carve.mx_dequant(codes, scales, dtype=torch.float16)
    with pytest.raises(ValueError):
        carve.mx_dequant(codes, scales, out=torch.empty(4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        carve.mx_dequant(codes.int(), scales)
    ring = carve.swa_cache_mx(1, 2, 64, 8)
    k = normal((1, 2, 5, 64), "bf16", 2)
    with pytest.raises(ValueError):
        carve.swa_fill_mx(k, k, ring, window=9)
    with pytest.raises(ValueError):
        carve.swa_fill_mx(k, k, ring[:3] + (ring[3][:, :, :, :1],), window=8)
    with pytest.raises(ValueError):
        carve.swa_fill_mx(k, k, carve.swa_cache_mx(1, 2, 64, 8, bits=8)[:2] + ring[2:], window=8)


# ------------------------------------------------------------------ the cache of a prompt
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hkv,T,D,window,sinks,lens", [
    (2, 40, 64, 16, 3, [40, 0, 2]), (1, 1, 128, 1, 0, None), (3, 100, 128, 33, 0, [99, 33, 1000]),
    (2, 50, 64, 200, 7, [50, 7, 6]), (1, 300, 128, 130, 64, None)])
def test_fill(Hkv, T, D, window, sinks, lens, bits, dt):
    B = 3 if lens else 2
    k, v = normal((B, Hkv, T, D), dt, 1), normal((B, Hkv, T, D), dt, 2)
    for b, n in enumerate(lens or []):
        k[b, :, max(n, 0):], v[b, :, max(n, 0):] = math.nan, math.nan
    ring = carve.swa_cache_mx(B, Hkv, D, window, sinks, bits=bits)
    for x in ring:
        x.fill_(77)
    want = [x.cpu().clone() for x in ring]
    carve.swa_fill_mx(k, v, ring, window, sinks, lens=ints(lens))
    for b in range(B):
        n = min(lens[b], T) if lens else T
        for p in list(range(min(sinks, n))) + list(range(max(sinks, n - window), n)):
            at = p if p < sinks else sinks + (p - sinks) % window
            for h in range(Hkv):
                put(want, b, h, [at], k[b, h, p:p + 1], v[b, h, p:p + 1], bits)
    for x, y in zip(ring, want):
        assert torch.equal(x.cpu(), y)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,C,D,sinks,recent,lens", [
    (200, 50, 64, 4, 10, [200, 130]), (30, 50, 128, 4, 10, [30, 0]), (0, 5, 64, 1, 2, [0, 0]), (700, 33, 128, 0, 33, None)])
def test_keep(T, C, D, sinks, recent, lens, bits, dt):
    """The same tokens, weights and positions as the cache of rows as they are; the rows in codes; other slots stay."""
    B, Hkv = 2, 2
    k, v = normal((B, Hkv, T, D), dt, 1), normal((B, Hkv, T, D), dt, 2)
    weights = torch.rand(B, Hkv, T, generator=torch.Generator().manual_seed(3)).cuda()
    at = dict(sinks=sinks, recent=recent, lens=ints(lens))
    plain = carve.budget_keep(k, v, weights, C, **at)
    cache = carve.budget_cache_mx(B, Hkv, D, C, bits=bits)
    for x in cache[:4]:
        x.fill_(77)
    want = [x.cpu().clone() for x in cache[:4]]
    got = carve.budget_keep_mx(k, v, weights, C, cache=cache, **at)
    assert all(a is b for a, b in zip(got, cache))
    assert torch.equal(cache[4], plain[2]) and torch.equal(cache[5], plain[3])
    for b in range(B):
        for h in range(Hkv):
            held = cache[5][b, h].cpu().long()
            m = int((held >= 0).sum())
            if m:
                put(want, b, h, slice(0, m), k[b, h, held[:m].cuda()], v[b, h, held[:m].cuda()], bits)
    for x, y in zip(cache, want):
        assert torch.equal(x.cpu(), y)
    new = carve.budget_keep_mx(k, v, weights, C, bits=bits, **at)
    assert new[0].shape[-1] == D * bits // 8 and torch.equal(new[5], cache[5])


# ------------------------------------------------------------------ ring cache, token by token
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,window,sinks,lens", [
    (2, 1, 64, 1500, 4, [1600, 900, 1503]), (24, 2, 128, 700, 0, [700, 699, 2000]),
    (4, 2, 64, 24, 3, [50, 0, 10]), (16, 1, 128, 7, 0, [5, 30, 1]), (6, 2, 64, 130, 64, [70, 300, 64]),
    (40, 1, 64, 50, 1, [20, 3, 90]), (3, 3, 128, 1, 0, [1, 2, 9]), (128, 2, 128, 200, 4, [0, 410, 199]),
    (17, 1, 128, 61, 2, [61, 62, 64])])
def test_ring_follows_the_sequence(Hq, Hkv, D, window, sinks, lens, bits, dt):
    """A prompt's cache, then tokens one by one: each output is the attention over what the codes of the tokens seen
    stand for, and the cache is the definition's, byte for byte.  Row 1 skips a step; what no token was written to
    holds scales that are not numbers, and keeps them."""
    B, steps, T, G = 3, 4, max(lens), Hq // Hkv
    q, k, v = (normal((B, n, T + steps, D), dt, 41 + i) for i, n in enumerate((Hq, Hkv, Hkv)))
    k = k * torch.exp(torch.randn(D, generator=torch.Generator().manual_seed(5))).cuda().to(k.dtype) * 0.5
    ring = junk(carve.swa_cache_mx(B, Hkv, D, window, sinks, bits=bits))
    want = [x.cpu().clone() for x in ring]
    carve.swa_fill_mx(k[:, :, :T].contiguous(), v[:, :, :T].contiguous(), ring, window, sinks, lens=ints(lens))
    have = list(lens)

    def slot(p):
        return p if p < sinks else sinks + (p - sinks) % window

    for b in range(B):
        seen = list(range(min(sinks, have[b]))) + list(range(max(sinks, have[b] - window), have[b]))
        for h in range(Hkv):
            if seen:
                put(want, b, h, [slot(p) for p in seen], k[b, h, seen], v[b, h, seen], bits)
    for step in range(steps):
        row, b = torch.tensor(have, device="cuda"), torch.arange(B, device="cuda")
        pos = [-1 if (i == 1 and step == 2) else n for i, n in enumerate(have)]
        o = carve.swa_decode_mx(q[b, :, row].contiguous(), k[b, :, row].contiguous(), v[b, :, row].contiguous(), ring,
                                ints(pos), window, sinks)
        for i in range(B):
            if pos[i] < 0:
                assert not o[i].any()
                continue
            n = have[i]
            count = min(n + 1, window + sinks)
            for h in range(Hkv):
                put(want, i, h, [slot(n)], k[i, h, n:n + 1], v[i, h, n:n + 1], bits)
                kk = mx_ref.values(want[0][i, h, :count], want[1][i, h, :count]).cuda()
                vv = mx_ref.values(want[2][i, h, :count], want[3][i, h, :count]).cuda()
                live = torch.ones(count, dtype=torch.bool, device="cuda")
                for g in range(h * G, h * G + G):
                    x = mx_ref.rows(q[i, g, n], kk, vv, live, D ** -0.5)
                    ref.within(o[i, g], x[:2], f"step {step} row {i} head {g}")
            have[i] += 1
        for x, y in zip(ring, want):
            assert torch.equal(x.cpu(), y), step


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits,D,Hq,window,B", [(4, 128, 8, 9000, 1), (8, 64, 8, 16389, 2), (4, 64, 80, 20001, 1), (8, 128, 2, 5003, 3)])
def test_ring_in_joined_ranges(bits, D, Hq, window, B, dt):
    """Long windows cut into ranges, with the token's slot in the first, a middle and the last range, and a batch of
    the same rows that needs no ranges."""
    Hkv, sinks = 2, 3
    C, G = window + sinks, Hq // 2
    ring = sum((carve.mx_quant(normal((B, Hkv, C, D), dt, 52 + i), bits=bits) for i in range(2)), ())
    q, k, v = normal((B, Hq, D), dt, 1), normal((B, Hkv, D), dt, 2), normal((B, Hkv, D), dt, 3)
    live = torch.ones(C, dtype=torch.bool, device="cuda")
    for at in (0, C // 2, C - 1):
        pos = [at if at < sinks else at + window] * B          # (position `at` itself lives in slot `at`)
        if at < sinks:
            pos = [at] * B
        now = [x.clone() for x in ring]
        o = carve.swa_decode_mx(q, k, v, now, ints(pos), window, sinks)
        many = [x.repeat(-(-600 // B), 1, 1, 1) for x in ring] if at == C - 1 else None
        n = min(pos[0] + 1, C)
        for b in range(B):
            for h in range(Hkv):
                want = [x[b:b + 1, h:h + 1].cpu().clone() for x in ring]
                put(want, 0, 0, [at], k[b, h][None], v[b, h][None], bits)
                for x, y in zip(now, want):
                    assert torch.equal(x[b, h].cpu(), y[0, 0])
                kk = mx_ref.values(want[0][0, 0], want[1][0, 0]).cuda()
                vv = mx_ref.values(want[2][0, 0], want[3][0, 0]).cuda()
                for g in (h * G, h * G + G - 1):
                    x = mx_ref.rows(q[b, g], kk, vv, live & (torch.arange(C, device="cuda") < n), D ** -0.5)
                    ref.within(o[b, g], x[:2], f"slot {at} row {b} head {g}")
                    if many and b == 0 and g == 0:
                        r = many[0].shape[0] // B
                        m = carve.swa_decode_mx(*[y.repeat(r, 1, 1) for y in (q, k, v)], many, ints(pos * r), window, sinks)
                        ref.within(m[0, 0], x[:2], "many, first")
                        ref.within(m[B * (r - 1), 0], x[:2], "many, last")


def test_ring_past_32_bits_of_offset():
    """One key head whose codes take more than 2^31 bytes: the last slots count as the first ones do.  Scores are zero but
    for chosen slots, so the output is the mean of the values there."""
    D, window = 64, (1 << 25) + 77
    ring = carve.swa_cache_mx(1, 1, D, window, bits=8)
    assert ring[0].numel() > 1 << 31
    for x in (ring[1], ring[3]):
        x.fill_(127)
    q = torch.ones(1, 1, D, device="cuda") * 8
    special = [5, (1 << 25) + 70, window - 2]
    for i, at in enumerate(special):
        ring[0][0, 0, at] = 0x48                               # 4.0: a score of 64 * 8 * 4 / 8
        ring[2][0, 0, at] = 0x38 + 8 * i                       # 1, 2, 4
    k, v = torch.full((1, 1, D), 4.0, device="cuda"), torch.full((1, 1, D), 8.0, device="cuda")
    o = carve.swa_decode_mx(q, k, v, ring, ints([window - 1]), window)
    # the other slots' weights are exp(-256) of these
    assert torch.equal(o, torch.full_like(o, (1 + 2 + 4 + 8) / 4))
    assert (ring[0][0, 0, window - 1].view(torch.float8_e4m3fn).float() == 256.0).all()       # 4 = 256 / 64, 8 = 256 / 32
    assert int(ring[1][0, 0, window - 1, 0]) == 127 - 6 and int(ring[3][0, 0, window - 1, 1]) == 127 - 5


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_large_scores(bits, dt):
    """Scores of several hundred, rising along the slots: the running maximum moves by more than a weight's range."""
    C, D = 1000, 128
    k = normal((1, 1, C, D), dt, 3) * torch.linspace(0.1, 6, C, device="cuda")[:, None].to(DT[dt])
    ring = carve.mx_quant(k, bits=bits) + carve.mx_quant(normal((1, 1, C, D), dt, 4), bits=bits)
    q = normal((1, 3, D), dt, 5) * 9
    o = carve.swa_decode_mx(q, k[:, :, 7].contiguous(), k[:, :, 8].contiguous(), ring, ints([5 * C - 3]), C)
    kk, vv = mx_ref.values(*ring[:2])[0, 0].cuda(), mx_ref.values(*ring[2:])[0, 0].cuda()
    for g in range(3):
        x = mx_ref.rows(q[0, g], kk, vv, torch.ones(C, dtype=torch.bool, device="cuda"), D ** -0.5)
        ref.within(o[0, g], x[:2], f"head {g}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_values_that_are_not_finite(dt):
    """A key that is not finite gives every head of its group a row that is not; a value, the elements of its block
    of 32; other key heads, rows and blocks have what they have without it.  A query reaches its own row."""
    B, Hq, Hkv, D, C = 2, 6, 2, 128, 70
    ring = carve.mx_quant(normal((B, Hkv, C, D), dt, 1)) + carve.mx_quant(normal((B, Hkv, C, D), dt, 2))
    q, k, v = normal((B, Hq, D), dt, 3), normal((B, Hkv, D), dt, 4), normal((B, Hkv, D), dt, 5)
    pos = ints([200, 200])
    clean = carve.swa_decode_mx(q, k, v, [x.clone() for x in ring], pos, C)
    for bad in (math.nan, math.inf, -math.inf):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        k2[0, 1, 5] = bad
        o = carve.swa_decode_mx(q, k2, v, [x.clone() for x in ring], pos, C)
        assert torch.isnan(o[0, 3:]).all() and torch.equal(o[0, :3], clean[0, :3]) and torch.equal(o[1], clean[1])
        v2[1, 0, 40] = bad
        o = carve.swa_decode_mx(q, k, v2, [x.clone() for x in ring], pos, C)
        assert torch.isnan(o[1, :3, 32:64]).all()
        for part in (slice(0, 32), slice(64, 128)):
            assert torch.equal(o[1, :3, part], clean[1, :3, part])
        assert torch.equal(o[1, 3:], clean[1, 3:]) and torch.equal(o[0], clean[0])
    q2[0, 2, 9] = math.nan
    o = carve.swa_decode_mx(q2, k, v, [x.clone() for x in ring], pos, C)
    assert torch.isnan(o[0, 2]).all()
    keep = torch.ones(B, Hq, dtype=torch.bool)
    keep[0, 2] = False
    assert torch.equal(o[keep], clean[keep])


# ------------------------------------------------------------------ cache kept by weight
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D,C,sinks,recent,steps", [
    (4, 2, 64, 8, 1, 3, 14), (1, 1, 128, 1, 0, 1, 4), (16, 1, 64, 40, 4, 36, 44), (40, 2, 128, 9, 0, 1, 12),
    (6, 2, 64, 300, 2, 10, 6), (64, 1, 128, 37, 0, 5, 5)])
def test_budget_decode_follows_its_rule(Hq, Hkv, D, C, sinks, recent, steps, bits, dt):
    """Token after token from an empty cache (C = 300: from one that is nearly full) against the rule in float64: the
    slots and the rows in codes are the same, outputs and weights within their bounds (which add up over the steps)."""
    B, G = 2, Hq // Hkv
    cache = junk(carve.budget_cache_mx(B, Hkv, D, C, bits=bits))       # empty slots are not read
    cache[4].fill_(math.nan)
    start = 0
    if C == 300:
        start = 297
        for i in (0, 2):
            c, s = carve.mx_quant(normal((B, Hkv, start, D), dt, 91 + i), bits=bits)
            cache[i][:, :, :start], cache[i + 1][:, :, :start] = c, s
        cache[4][:, :, :start] = torch.rand(B, Hkv, start, generator=torch.Generator().manual_seed(93)).cuda()
        cache[5][:, :, :start] = torch.arange(start, dtype=torch.int32, device="cuda")
    want, mp = [x.cpu().clone() for x in cache[:4]], cache[5].cpu().clone()
    mw = cache[4].double().cpu()
    tw = torch.zeros_like(mw)
    for step in range(steps):
        p = start + step
        pos = [p, -1 if step == 3 else p - (1 if step > 3 else 0)]
        q, k, v = normal((B, Hq, D), dt, 200 + step), normal((B, Hkv, D), dt, 300 + step), normal((B, Hkv, D), dt, 400 + step)
        o, slot = carve.budget_decode_mx(q, k, v, cache, ints(pos), sinks=sinks, recent=recent)
        for b in range(B):
            if pos[b] < 0:
                assert not o[b].any() and (slot[b] == -1).all()
                continue
            for h in range(Hkv):
                held, w = mp[b, h].tolist(), mw[b, h].tolist()
                if min(held) < 0:
                    at = next(j for j in range(C) if held[j] < 0)
                else:
                    at = min((j for j in range(C) if sinks <= held[j] <= pos[b] - recent), key=lambda j: (w[j], j))
                assert int(slot[b, h]) == at, (step, b, h)
                put(want, b, h, [at], k[b, h][None], v[b, h][None], bits)
                mp[b, h, at], mw[b, h, at], tw[b, h, at] = pos[b], 0.0, 0.0
                live = (mp[b, h] >= 0).cuda()
                kk, vv = mx_ref.values(want[0][b, h], want[1][b, h]).cuda(), mx_ref.values(want[2][b, h], want[3][b, h]).cuda()
                for g in range(h * G, (h + 1) * G):
                    x = [y.cpu() for y in mx_ref.rows(q[b, g], kk, vv, live, D ** -0.5)]
                    ref.within(o[b, g].cpu(), x[:2], f"step {step} {b} {g}")
                    mw[b, h] += torch.where(live.cpu(), x[2], 0.0)
                    tw[b, h] += torch.where(live.cpu(), x[3] + 2 * ref.F32 * (mw[b, h].abs() + 1), 0.0)
        live = mp >= 0
        assert torch.equal(cache[5].cpu(), mp)
        ref.within(torch.where(live, cache[4].cpu(), 0.0),
                   (torch.where(live, mw, 0.0), tw + ref.F32 * mw.nan_to_num().abs()), f"weights {step}")
        for x, y in zip(cache, want):
            assert torch.equal(x.cpu(), y), step


def one_eviction(B, Hq, Hkv, D, C, bits, dt, sinks=4, recent=20, empty=0):
    """One step of a batch of full caches (but for `empty` slots in the middle, whose rows must not be read)."""
    G = Hq // Hkv
    cache = carve.budget_cache_mx(B, Hkv, D, C, bits=bits)
    for i in (0, 2):
        c, s = carve.mx_quant(normal((B, Hkv, C, D), dt, 5 + i), bits=bits)
        cache[i].copy_(c)
        cache[i + 1].copy_(s)
    cache[4].copy_(torch.rand(B, Hkv, C, generator=torch.Generator().manual_seed(7)))
    cache[5].copy_(torch.arange(C, dtype=torch.int32))
    if empty:
        gone = slice(C // 3, C // 3 + empty)
        for x in cache[:4]:
            x[:, :, gone] = 255
        cache[4][:, :, gone] = math.nan
        cache[5][:, :, gone] = -1
    was = [x.clone() for x in cache]
    q, k, v = normal((B, Hq, D), dt, 8), normal((B, Hkv, D), dt, 9), normal((B, Hkv, D), dt, 10)
    o, slot = carve.budget_decode_mx(q, k, v, cache, ints([C] * B), sinks=sinks, recent=recent)
    for b in sorted({0, B // 2, B - 1}):
        for h in sorted({0, Hkv - 1}):
            at = C // 3 if empty else sinks + int(was[4][b, h, sinks:C - recent + 1].argmin())
            assert int(slot[b, h]) == at
            want = [x[b:b + 1, h:h + 1].cpu().clone() for x in was[:4]]
            put(want, 0, 0, [at], k[b, h][None], v[b, h][None], bits)
            for x, y in zip(cache, want):
                assert torch.equal(x[b, h].cpu(), y[0, 0])
            held = was[5][b, h].clone()
            held[at] = C
            assert torch.equal(cache[5][b, h], held)
            live = held >= 0
            kk = mx_ref.values(want[0][0, 0], want[1][0, 0]).cuda()
            vv = mx_ref.values(want[2][0, 0], want[3][0, 0]).cuda()
            w, tol = was[4][b, h].double(), torch.zeros(C, dtype=torch.float64, device="cuda")
            w[at] = 0.0
            for g in range(h * G, h * G + G):
                x = mx_ref.rows(q[b, g], kk, vv, live, D ** -0.5)
                ref.within(o[b, g], x[:2], f"row {b} head {g}")
                w, tol = w + x[2], tol + x[3]
            ref.within(cache[4][b, h][live], (w[live], (tol + (G + 1) * ref.F32 * w.abs())[live]), "weights")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("empty", [0, 5])
@pytest.mark.parametrize("B,Hq,Hkv,D,C", [
    (1, 8, 2, 128, 500), (1, 2, 1, 64, 1023), (2, 16, 1, 128, 250), (1, 8, 2, 64, 2049), (1, 34, 1, 64, 700),
    (1, 128, 2, 128, 333), (75, 16, 4, 64, 500), (75, 8, 4, 128, 130), (150, 40, 4, 64, 140), (140, 4, 2, 128, 301), (130, 24, 4, 64, 260), (1, 40, 2, 64, 1024), (1, 16, 1, 128, 1281)])
def test_eviction(B, Hq, Hkv, D, C, empty, bits, dt):
    """Small caches of few and many key heads, scores near and far."""
    one_eviction(B, Hq, Hkv, D, C, bits, dt, empty=empty)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits,Hq,D,C", [(4, 8, 128, 9001), (8, 4, 64, 12003), (4, 40, 64, 20002), (8, 128, 128, 6007)])
@pytest.mark.parametrize("empty", [0, 300])
def test_eviction_in_joined_ranges(bits, Hq, D, C, empty, dt):
    one_eviction(1, Hq, 2, D, C, bits, dt, empty=empty)


def test_slots_by_ties_specials_and_repeats():
    """The slot rule of the cache of plain rows: both caches give the same slots, positions and, for one live token, weight."""
    B, Hkv, D, C = 1, 1, 64, 6
    q, k, v = normal((B, 1, D), "bf16", 1), normal((B, 1, D), "bf16", 2), normal((B, 1, D), "bf16", 3)
    for w, held, pos in (([0.0, 2.0, 1.0, 1.0, 5.0, 0.0], [0, 1, 2, 3, 4, 9], 10), ([0.0, math.nan, 7.0, math.inf, 8.0, 0.0], [0, 1, 2, 3, 4, 9], 10),
                         ([0.0, 2.0, -0.0, 0.0, 5.0, 0.0], [0, 1, 2, 3, 4, 9], 10), ([0.0, 2.0, 1.0, -3.0, 5.0, 0.0], [0, 1, 2, 3, 4, 9], 10),
                         ([9.0, 0.0, 1.0, 1.0, 5.0, 0.0], [0, 1, -1, -7, 4, 9], 10), ([9.0, 0.0, 1.0, 1.0, 5.0, 0.0], [0, 10, -1, -7, 4, 9], 10)):
        plain, coded = carve.budget_cache(B, Hkv, D, C), carve.budget_cache_mx(B, Hkv, D, C)
        for cw, cp in (plain[2:], coded[4:]):
            cw.copy_(torch.tensor(w).view(1, 1, C))
            cp.copy_(torch.tensor(held, dtype=torch.int32).view(1, 1, C))
        one = carve.budget_decode(q, k, v, plain, ints([pos]), sinks=1, recent=2)[1]
        two = carve.budget_decode_mx(q, k, v, coded, ints([pos]), sinks=1, recent=2)[1]
        assert torch.equal(one, two) and torch.equal(plain[3], coded[5])
    cache = carve.budget_cache_mx(B, Hkv, D, C)
    for _ in range(3):                        # the call repeated stores the token once
        _, slot = carve.budget_decode_mx(q, k, v, cache, ints([0]), sinks=1, recent=2)
        assert int(slot) == 0
    assert cache[5][0, 0].tolist() == [0, -1, -1, -1, -1, -1] and float(cache[4][0, 0, 0]) == 1.0


@pytest.mark.parametrize("C", [70, 5000])
def test_rows_without_a_token(C):
    """Rows with a negative position (in one range and in several): output zero, slot -1, the cache as it was."""
    B, Hq, Hkv, D = 3, 4, 2, 128
    ring = [torch.randint(0, 255, x.shape, dtype=torch.uint8, device="cuda") for x in carve.swa_cache_mx(B, Hkv, D, C)]
    kept = tuple(x.clone() for x in ring) + (torch.rand(B, Hkv, C, device="cuda"), torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1))
    q, k, v = normal((B, Hq, D), "bf16", 1), normal((B, Hkv, D), "bf16", 2), normal((B, Hkv, D), "bf16", 3)
    pos, before = ints([-1, 2 * C, -2147483648]), [x.clone() for x in kept]
    o = torch.full_like(q, 5.0)
    assert carve.swa_decode_mx(q, k, v, ring, pos, C, o=o) is o
    o2, slot = carve.budget_decode_mx(q, k, v, kept, pos, recent=3, o=torch.full_like(q, 5.0))
    for b in (0, 2):
        assert not o[b].any() and not o2[b].any() and (slot[b] == -1).all()
        assert all(torch.equal(x[b], y[b]) for x, y in zip(ring, before)) and all(torch.equal(x[b], y[b]) for x, y in zip(kept, before))
    assert o[1].any() and (slot[1] >= 0).all()


def test_numbers_held_by_tensors():
    """A scale given as a tensor counts as it is at the call, and so do window and sinks; other numbers are refused."""
    q, k, v = normal((1, 2, 64), "bf16", 1), normal((1, 1, 64), "bf16", 2), normal((1, 1, 64), "bf16", 3)
    ring = carve.mx_quant(normal((1, 1, 12, 64), "bf16", 4)) + carve.mx_quant(normal((1, 1, 12, 64), "bf16", 5))
    pos, scale, window, sinks = ints([30]), torch.tensor(0.5), torch.tensor(10), torch.tensor(2)

    def step(scale, window=10, sinks=2):
        return carve.swa_decode_mx(q, k, v, [x.clone() for x in ring], pos, window, sinks=sinks, scale=scale)

    assert torch.equal(step(scale, window, sinks), step(0.5))
    scale.fill_(0.125)
    window.fill_(9)
    sinks.fill_(3)
    assert torch.equal(step(scale, window, sinks), step(0.125, 9, 3)) and not torch.equal(step(0.125), step(0.5))
    with pytest.raises(TypeError):
        step(0.5, 10.0)
    for bad in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(RuntimeError):
            step(bad)


def test_most_key_heads():
    """65,535 sequences of one head, the most that a call takes: prompt, read back and one token, all rows checked."""
    B, D, W, T = 65535, 64, 4, 3
    k, v = normal((B, 1, T, D), "bf16", 1), normal((B, 1, T, D), "bf16", 2)
    ring = carve.swa_cache_mx(B, 1, D, W)
    carve.swa_fill_mx(k, v, ring, W)
    q1, k1, v1 = normal((B, 1, D), "bf16", 3), normal((B, 1, D), "bf16", 4), normal((B, 1, D), "bf16", 5)
    kk, vv = (torch.cat([mx_ref.written(x.view(-1, D), 4)[0].view(B, T, D), mx_ref.written(y.view(-1, D), 4)[0].view(B, 1, D)], 1).cuda()
              for x, y in ((k, k1), (v, v1)))
    assert torch.equal(carve.mx_dequant(*ring[:2], dtype=torch.float32)[:, 0, :T].double(), kk[:, :T])
    o = carve.swa_decode_mx(q1, k1, v1, ring, torch.full((B,), T, dtype=torch.int32, device="cuda"), W)
    kept = carve.budget_keep_mx(k, v, torch.ones(B, 1, T, device="cuda"), W)
    o2, slot = carve.budget_decode_mx(q1, k1, v1, kept, torch.full((B,), T, dtype=torch.int32, device="cuda"))
    assert (slot == T).all() and torch.equal(o2, o)
    p = torch.softmax((kk * q1.double()).sum(-1) * D ** -0.5, -1)[..., None]
    want, size = (p * vv).sum(1), (p * vv.abs()).sum(1)
    A = (kk.abs() * q1.double().abs()).sum(-1).amax() * D ** -0.5
    u = ref.half_step(torch.bfloat16)
    ref.within(o[:, 0], (want, (2 * ref.F32 * (2 * (D + 4) * A + W + 32) + u) * size + u * want.abs()), "o")
    for x, y in zip(ring, kept):
        assert torch.equal(x, y)


def test_written_in_bf16_read_in_float32():
    """A cache has no type of its own: a bf16 prompt's, with float32 tokens on it, and a scale of the caller's."""
    B, Hq, Hkv, T, D, W = 1, 6, 2, 40, 64, 50
    k, v = normal((B, Hkv, T, D), "bf16", 1), normal((B, Hkv, T, D), "bf16", 2)
    ring = carve.swa_cache_mx(B, Hkv, D, W, bits=8)
    carve.swa_fill_mx(k, v, ring, W)
    q1, k1, v1 = normal((B, Hq, D), "f32", 3), normal((B, Hkv, D), "f32", 4), normal((B, Hkv, D), "f32", 5)
    o = carve.swa_decode_mx(q1, k1, v1, ring, ints([T]), W, scale=0.37)
    assert o.dtype == torch.float32
    live = torch.ones(T + 1, dtype=torch.bool, device="cuda")
    for g in range(Hq):
        kk, vv = (torch.cat([mx_ref.written(x[0, g // 3], 8)[0], mx_ref.written(y[0, g // 3][None], 8)[0]]).cuda() for x, y in ((k, k1), (v, v1)))
        ref.within(o[0, g], mx_ref.rows(q1[0, g], kk, vv, live, 0.37)[:2], f"head {g}")


# ------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_in_a_graph_follows_the_positions(dt):
    """Captured decode steps of both caches, replayed with other inputs and positions and with eager work between, against
    the same steps run eagerly."""
    B, Hq, Hkv, D, window, sinks, C, recent = 2, 8, 2, 64, 30, 2, 20, 5
    q, k, v = normal((B, Hq, D), dt, 61), normal((B, Hkv, D), dt, 62), normal((B, Hkv, D), dt, 63)
    pos = ints([0, 7])
    ring, kept = carve.swa_cache_mx(B, Hkv, D, window, sinks), carve.budget_cache_mx(B, Hkv, D, C, bits=8)

    def step(ring, kept):
        o1 = carve.swa_decode_mx(q, k, v, ring, pos, window, sinks)
        o2, slot = carve.budget_decode_mx(q, k, v, kept, pos, sinks=sinks, recent=recent)
        return o1, o2, slot, carve.mx_dequant(*ring[:2]), carve.mx_quant(q, bits=4)[0]

    step(ring, kept)
    g = torch.cuda.CUDAGraph()
    for x in ring + kept[:5]:
        x.zero_()
    kept[5].fill_(-1)
    with torch.cuda.graph(g):
        got = step(ring, kept)
    mirror = [x.clone() for x in ring], tuple(x.clone() for x in kept)
    for i in range(40):
        for j, x in enumerate((q, k, v)):
            x.copy_(normal(x.shape, dt, 100 + 3 * i + j))
        g.replay()
        want = step(*mirror)
        torch.cuda.synchronize()
        for a, b in zip(list(got) + list(ring) + list(kept), list(want) + list(mirror[0]) + list(mirror[1])):
            assert torch.equal(a, b), i
        pos += 1


def test_joined_ranges_in_two_graphs():
    """Two captured graphs of steps on long caches (a workspace each, of the graph's own memory), replayed in turn with
    positions that go on and eager work between, against the same steps run eagerly."""
    D, C, Hq, Hkv = 128, 5001, 8, 2
    graphs = []
    for seed in (0, 50):
        ring = sum((carve.mx_quant(normal((1, Hkv, C, D), "bf16", seed + i)) for i in range(2)), ())
        kept = tuple(x.clone() for x in ring) + (torch.rand(1, Hkv, C, generator=torch.Generator().manual_seed(seed)).cuda(),
                                                torch.arange(C, dtype=torch.int32, device="cuda").repeat(1, Hkv, 1))
        q, k, v = normal((1, Hq, D), "bf16", seed + 2), normal((1, Hkv, D), "bf16", seed + 3), normal((1, Hkv, D), "bf16", seed + 4)
        pos = ints([C])

        def step(ring, kept, q=q, k=k, v=v, pos=pos):
            return (carve.swa_decode_mx(q, k, v, ring, pos, C), *carve.budget_decode_mx(q, k, v, kept, pos, sinks=2, recent=9))

        mirror = [x.clone() for x in ring], tuple(x.clone() for x in kept)
        g = torch.cuda.CUDAGraph()
        step([x.clone() for x in ring], tuple(x.clone() for x in kept))
        with torch.cuda.graph(g):
            got = step(ring, kept)
        graphs.append((g, step, got, ring, kept, mirror, pos))
    for i in range(4):
        for g, *_ in graphs:
            g.replay()
        torch.zeros(1 << 20, device="cuda").sum()
        for g, step, got, ring, kept, mirror, pos in graphs:
            want = step(*mirror)
            torch.cuda.synchronize()
            for a, b in zip(list(got) + list(ring) + list(kept), list(want) + list(mirror[0]) + list(mirror[1])):
                assert torch.equal(a, b), i
            pos += 1


def test_two_streams_at_once():
    """Calls on two streams, each with caches and workspaces of its own, give the bits of the same calls one after the other."""
    D, window, C, Hq, Hkv = 128, 9000, 9000, 8, 2
    made = []
    for seed in (0, 50):
        ring = carve.mx_quant(normal((1, Hkv, window, D), "bf16", seed)) + carve.mx_quant(normal((1, Hkv, window, D), "bf16", seed + 1))
        kept = tuple(x.clone() for x in ring) + (torch.rand(1, Hkv, C, generator=torch.Generator().manual_seed(seed)).cuda(),
                                                torch.arange(C, dtype=torch.int32, device="cuda").repeat(1, Hkv, 1))
        made.append((normal((1, Hq, D), "bf16", seed + 2), normal((1, Hkv, D), "bf16", seed + 3),
                     normal((1, Hkv, D), "bf16", seed + 4), ring, kept))

    def steps(q, k, v, ring, kept):
        ring, kept, out = [x.clone() for x in ring], tuple(x.clone() for x in kept), []
        for i in range(6):
            pos = torch.full((1,), C + i, dtype=torch.int32, device="cuda")
            out += [carve.swa_decode_mx(q, k, v, ring, pos, window), *carve.budget_decode_mx(q, k, v, kept, pos, sinks=2, recent=9)]
        return out + ring + list(kept)

    want = [steps(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for st, m in zip(streams, made):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(steps(*m))
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_prompt_to_caches_to_tokens():
    """The operators as they are used together: a prompt's attention and weights, both caches made from it in codes, tokens
    decoded on both.  A ring that has held the whole sequence and a budget that has dropped nothing see the same rows."""
    B, Hq, Hkv, T, D = 2, 8, 2, 90, 64
    q, k, v = normal((B, Hq, T, D), "bf16", 1), normal((B, Hkv, T, D), "bf16", 2), normal((B, Hkv, T, D), "bf16", 3)
    lens = ints([90, 47])
    _, lse = carve.swa_fwd(q, k, v, window=T, lens=lens)
    a = carve.budget_weights(q, k, lse, lens=lens)
    for bits in (4, 8):
        ring = carve.swa_cache_mx(B, Hkv, D, 100, sinks=4, bits=bits)
        carve.swa_fill_mx(k, v, ring, 100, sinks=4, lens=lens)
        kept = carve.budget_keep_mx(k, v, a, 104, sinks=4, recent=16, lens=lens, bits=bits)
        whole = [carve.mx_dequant(*kept[i:i + 2]) for i in (0, 2)]
        pos = lens.clone()
        for step in range(5):
            q1, k1, v1 = (normal((B, n, D), "bf16", 20 + 3 * step + i) for i, n in enumerate((Hq, Hkv, Hkv)))
            o1 = carve.swa_decode_mx(q1, k1, v1, ring, pos, 100, sinks=4)
            before = kept[4].double().sum((1, 2))
            o2, slot = carve.budget_decode_mx(q1, k1, v1, kept, pos, sinks=4, recent=16)
            assert torch.equal(slot, pos[:, None].expand(B, Hkv))
            for b in range(B):
                n = int(pos[b]) + 1
                for i in (0, 1, 2, 3):
                    assert torch.equal(ring[i][b, :, :n], kept[i][b, :, :n])
                for h in range(Hq):
                    kk, vv = (mx_ref.values(ring[i][b, h // 4, :n], ring[i + 1][b, h // 4, :n]).cuda() for i in (0, 2))
                    x = mx_ref.rows(q1[b, h], kk, vv, torch.ones(n, dtype=torch.bool, device="cuda"), D ** -0.5)
                    ref.within(o1[b, h], x[:2], f"ring {b} {h}")
                    ref.within(o2[b, h], x[:2], f"kept {b} {h}")
            # a token's weights of all heads sum to one
            assert ((kept[4].double().sum((1, 2)) - before - Hq).abs() <= 1e-4 * Hq).all()
            pos += 1
        assert torch.equal(carve.mx_dequant(*kept[:2])[0, :, :90], whole[0][0, :, :90])
