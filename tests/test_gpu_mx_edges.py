"""Decode steps on caches in codes where results are decided by one rounding or one value: bf16
weights, values that are not finite, scores far below zero (tests/mx_ref.py states the definition and the bounds)."""
import ctypes
import math

import pytest
import torch

from chunk_gated_delta_amd import carve
from tests import attention_ref as ref
from tests import mx_ref
from tests.test_gpu_mx import one_eviction

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ring_of(k, v, bits):
    return carve.mx_quant(k, bits=bits) + carve.mx_quant(v, bits=bits)


def kept_of(k, v, bits, seed=7):
    """A full cache kept by weight: slot j holds position j."""
    B, Hkv, C, _ = k.shape
    w = torch.rand(B, Hkv, C, generator=torch.Generator().manual_seed(seed)).cuda()
    return ring_of(k, v, bits) + (w, torch.arange(C, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1))


def copy_of(cache):
    return tuple(x.clone() for x in cache)


# ------------------------------------------------------------------ roundings
def fine_rows(q, k, v, scale):
    """(o, bound) of one bf16 query over rows k, v [C,D] (float64 values) where the weights enter the product with v as
    two bf16 parts.  The first is a float's upper half, off by less than 2^-7 of it, the second rounds what is left
    by half a step at most: together 2^-7 2^-8.  The sum runs over 2 C products; else as in mx_ref.rows."""
    C, D = k.shape
    s = k @ q.double() * scale
    p = torch.softmax(s, 0)
    A = (k.abs() @ q.double().abs() * scale).amax()
    e = ref.F32 * (2 * (D + 4) * A + 2 * C + 32)
    o = p @ v
    return o, (2 * e + 2.0 ** -15) * (p @ v.abs()) + ref.half_step(torch.bfloat16) * o.abs()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,Hq,Hkv,D,C", [
    (1, 8, 2, 128, 9), (3, 6, 2, 64, 40), (70, 16, 4, 128, 33), (130, 8, 2, 64, 7), (2, 24, 1, 128, 20), (140, 40, 2, 64, 5), (1, 64, 1, 128, 11)])
def test_bf16_outputs_are_rounded_once(B, Hq, Hkv, D, C, bits):
    """With few slots a weight's rounding to bf16 would be as large as the output's: outputs are within half a step."""
    G = Hq // Hkv
    k, v = normal((B, Hkv, C, D), "bf16", 1), normal((B, Hkv, C, D), "bf16", 2)
    kept = kept_of(k, v, bits)
    q, k1, v1 = normal((B, Hq, D), "bf16", 3), normal((B, Hkv, D), "bf16", 4), normal((B, Hkv, D), "bf16", 5)
    ring, pos = copy_of(kept[:4]), ints([C] * B)
    o = carve.swa_decode_mx(q, k1, v1, ring, pos, C)
    o2, slot = carve.budget_decode_mx(q, k1, v1, kept, pos)
    for b in sorted({0, B // 2, B - 1}):
        for g in range(Hq):
            for x, cache, what in ((o, ring, "ring"), (o2, kept, "kept")):
                kk, vv = (mx_ref.values(cache[i][b, g // G], cache[i + 1][b, g // G]).cuda() for i in (0, 2))
                ref.within(x[b, g], fine_rows(q[b, g], kk, vv, D ** -0.5), f"{what} row {b} head {g}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,C", [(64, 2048), (1, 9001)])
def test_a_step_repeats_itself(B, C, dt):
    """The same step on copies of the same caches, in one range and in several: the same bits."""
    Hq, Hkv, D = 16, 4, 128
    kept = kept_of(normal((B, Hkv, C, D), dt, 1), normal((B, Hkv, C, D), dt, 2), 4)
    q, k, v = normal((B, Hq, D), dt, 3), normal((B, Hkv, D), dt, 4), normal((B, Hkv, D), dt, 5)
    pos, want = ints([C] * B), None
    for _ in range(5):
        ring, now = copy_of(kept[:4]), copy_of(kept)
        got = [carve.swa_decode_mx(q, k, v, ring, pos, C), *carve.budget_decode_mx(q, k, v, now, pos, sinks=4, recent=9), *ring, *now]
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ values that are not finite
SIZES = [(1, 6, 2, 128, 1), (2, 6, 2, 64, 70), (1, 40, 2, 128, 33), (2, 8, 2, 128, 9001), (130, 4, 2, 64, 300), (1, 68, 2, 64, 50)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,Hq,Hkv,D,C", SIZES)
def test_query_that_is_not_finite(B, Hq, Hkv, D, C, bits, dt):
    """Its own row is not a number, also where every key has the same sign at the infinite element (all scores are
    then infinite with one sign).  Other key heads keep their bits; heads that share its key head may be scaled anew where
    it is, so they are compared by value: either side is off by less than (2 e + 2^-8) max |v| + 2^-8 |o|, with scores of A < 40
    and 3 C < 2^15 terms e < 2^-24 (2 (3 128 + 4) 40 + 2^15 + 32) < 2^-8, so by less than 2^-5 max |v| together.  In a
    cache kept by weight all slots of its key head weigh not a number from then on, and the next token takes the first that
    may be given up."""
    G, sinks, recent = Hq // Hkv, min(2, C - 1), 1
    k = normal((B, Hkv, C, D), dt, 1).abs() + 0.5
    kept = kept_of(k, normal((B, Hkv, C, D), dt, 2), bits)
    q, k1, v1 = normal((B, Hq, D), dt, 3), normal((B, Hkv, D), dt, 4).abs() + 0.5, normal((B, Hkv, D), dt, 5)
    pos, b, g = ints([C] * B), B - 1, Hq - 1
    h = g // G

    def step(q):
        ring, now = copy_of(kept[:4]), copy_of(kept)
        return carve.swa_decode_mx(q, k1, v1, ring, pos, C), carve.budget_decode_mx(q, k1, v1, now, pos, sinks=sinks, recent=recent), now

    clean, (clean2, slot), held = step(q)
    rest, group = torch.ones(B, Hq, dtype=torch.bool), torch.zeros(B, Hq, dtype=torch.bool)
    rest[b, h * G:h * G + G] = False
    group[b, h * G:g] = True
    others = torch.ones(B, Hkv, dtype=torch.bool)
    others[b, h] = False
    most = 2.0 ** -5 * 6                                      # (of normal values, none is past 6)
    for bad in (-math.inf, math.inf, math.nan):
        q2 = q.clone()
        q2[b, g, 9] = bad
        o, (o2, slot2), now = step(q2)
        assert torch.isnan(o[b, g]).all() and torch.isnan(o2[b, g]).all(), bad
        assert torch.equal(o[rest], clean[rest]) and torch.equal(o2[rest], clean2[rest])
        assert ((o[group] - clean[group]).abs() <= most).all() and ((o2[group] - clean2[group]).abs() <= most).all()
        assert torch.equal(slot2, slot) and all(torch.equal(now[i], held[i]) for i in (0, 1, 2, 3, 5))
        assert torch.isnan(now[4][b, h]).all() and torch.equal(now[4][others], held[4][others])
        at = next(j for j in range(C) if sinks <= int(now[5][b, h, j]) <= C + 1 - recent)
        _, slot3 = carve.budget_decode_mx(q, k1, v1, now, pos + 1, sinks=sinks, recent=recent)
        assert int(slot3[b, h]) == at


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,Hq,Hkv,D,C", SIZES)
def test_key_or_value_that_is_not_finite(B, Hq, Hkv, D, C, bits, dt):
    """A key gives all heads of its group a row that is not a number, and the slots of its key head such weights; a
    value the places of its block, and no weight.  So do a scale byte 255 in the cache and, at its own place, the code of 8
    bits that is not a number."""
    G = Hq // Hkv
    kept = kept_of(normal((B, Hkv, C, D), dt, 1), normal((B, Hkv, C, D), dt, 2), bits)
    if C > 1:
        kept[4][:, :, C // 2] = 2.0 ** 20                     # the slot that is spoilt is not the one that the token takes
    q, k1, v1 = normal((B, Hq, D), dt, 3), normal((B, Hkv, D), dt, 4), normal((B, Hkv, D), dt, 5)
    pos, b, h, recent = ints([C] * B), B - 1, Hkv - 1, 1
    heads = slice(h * G, h * G + G)

    def step(k1, v1, cache=kept):
        ring, now = copy_of(cache[:4]), copy_of(cache)
        return carve.swa_decode_mx(q, k1, v1, ring, pos, C), carve.budget_decode_mx(q, k1, v1, now, pos, recent=recent)[0], now[4]

    clean = step(k1, v1)
    rest = torch.ones(B, Hq, dtype=torch.bool)
    rest[b, heads] = False
    others = torch.ones(B, Hkv, dtype=torch.bool)
    others[b, h] = False

    def spoilt_key(got):
        for o, c in zip(got[:2], clean):
            assert torch.isnan(o[b, heads]).all() and torch.equal(o[rest], c[rest])
        assert torch.isnan(got[2][b, h]).all() and torch.equal(got[2][others], clean[2][others])

    def spoilt_value(got, places):
        for o, c in zip(got[:2], clean):
            assert torch.isnan(o[b, heads][:, places]).all() and torch.equal(o[rest], c[rest])
            keep = torch.ones(D, dtype=torch.bool)
            keep[places] = False
            assert torch.equal(o[b, heads][:, keep], c[b, heads][:, keep])
        assert torch.equal(got[2], clean[2])

    for bad in (math.nan, math.inf, -math.inf):
        k2, v2 = k1.clone(), v1.clone()
        k2[b, h, 5] = bad
        spoilt_key(step(k2, v1))
        v2[b, h, 40] = bad
        spoilt_value(step(k1, v2), slice(32, 64))
    if C > 1:
        for i, check in ((1, spoilt_key), (3, lambda got: spoilt_value(got, slice(32, 64)))):
            cache = copy_of(kept)
            cache[i][b, h, C // 2, 1] = 255
            check(step(k1, v1, cache))
        if bits == 8:
            for i, check in ((0, spoilt_key), (2, lambda got: spoilt_value(got, slice(37, 38)))):
                for code in (0x7f, 0xff):
                    cache = copy_of(kept)
                    cache[i][b, h, C // 2, 37] = code
                    check(step(k1, v1, cache))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,D,C", SIZES)
@pytest.mark.parametrize("bad", [-math.inf, math.inf, math.nan])
def test_infinite_query_on_plain_rows(B, Hq, Hkv, D, C, dt, bad):
    """The same on caches of rows as they are: all scores of a head infinite with one sign give not a number."""
    G, h = Hq // Hkv, Hkv - 1
    k, v = normal((B, Hkv, C, D), dt, 1).abs() + 0.5, normal((B, Hkv, C, D), dt, 2)
    kept = (k, v) + kept_of(k, v, 4)[4:]
    q, k1, v1 = normal((B, Hq, D), dt, 3), normal((B, Hkv, D), dt, 4).abs() + 0.5, normal((B, Hkv, D), dt, 5)
    q[B - 1, Hq - 1, 9] = bad
    now = copy_of(kept)
    o = carve.swa_decode(q, k1, v1, k.clone(), v.clone(), ints([C] * B), C)
    o2, _ = carve.budget_decode(q, k1, v1, now, ints([C] * B))
    keep = torch.ones(B, Hq, dtype=torch.bool)
    keep[B - 1, Hq - 1] = False
    for x in (o, o2):
        assert torch.isnan(x[B - 1, Hq - 1]).all() and torch.isfinite(x[keep]).all()
    assert torch.isnan(now[2][B - 1, h]).all() and int(torch.isnan(now[2]).sum()) == C


# ------------------------------------------------------------------ scores far below zero
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,D,C,have", [(1, 64, 1, 0), (3, 128, 4, 2), (40, 64, 70, 69), (2, 64, 9001, 3), (64, 128, 33, 2)])
def test_scores_below_every_start(Hq, D, C, have, bits, dt):
    """All scores finite and below -10^33: the token nearest to zero has all the weight (scores differ by a
    quarter and more), in one range and in several with nothing in most of them."""
    far = torch.arange(have + 1, 0, -1, dtype=torch.float32).view(1, 1, -1, 1).expand(1, 1, have + 1, D)
    far = (-1e16 * torch.where(far > 4, 4.0, far)).to(DT[dt]).cuda()        # -4 .. -4, -3, -2 and, of the new token, -1
    v = normal((1, 1, have + 1, D), dt, 2)
    q = torch.full((1, Hq, D), 1e16, device="cuda").to(DT[dt])
    ring = carve.swa_cache_mx(1, 1, D, C, bits=bits)
    kept = carve.budget_cache_mx(1, 1, D, C, bits=bits)
    if have:
        prompt = [x[:, :, :have].contiguous() for x in (far, v)]
        carve.swa_fill_mx(*prompt, ring, C)
        carve.budget_keep_mx(*prompt, torch.ones(1, 1, have, device="cuda"), C, cache=kept)
    k1, v1 = (x[:, :, have].contiguous() for x in (far, v))
    o = carve.swa_decode_mx(q, k1, v1, ring, ints([have]), C)
    o2, slot = carve.budget_decode_mx(q, k1, v1, kept, ints([have]))
    want = mx_ref.written(v1, bits)[0].view(D).to(DT[dt]).cuda()         # (a bf16 exactly)
    for x in (o, o2):
        assert all(torch.equal(x[0, g], want) for g in range(Hq))
    assert int(slot) == have and float(kept[4][0, 0, have]) == Hq and (kept[4][0, 0, :have] == 1).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,D,C,have", [(1, 64, 1, 0), (3, 128, 4, 2), (40, 64, 70, 69), (2, 64, 9001, 3)])
def test_scores_below_every_start_on_plain_rows(Hq, D, C, have, dt):
    """The same on caches of rows as they are."""
    far = torch.arange(have + 1, 0, -1, dtype=torch.float32).view(1, 1, -1, 1).expand(1, 1, have + 1, D)
    far = (-1e16 * torch.where(far > 4, 4.0, far)).to(DT[dt]).cuda()
    v = normal((1, 1, have + 1, D), dt, 2)
    q = torch.full((1, Hq, D), 1e16, device="cuda").to(DT[dt])
    ring, kept = carve.swa_cache(1, 1, D, C, dtype=DT[dt]), carve.budget_cache(1, 1, D, C, dtype=DT[dt])
    if have:
        prompt = [x[:, :, :have].contiguous() for x in (far, v)]
        carve.swa_fill(*prompt, *ring, C)
        carve.budget_keep(*prompt, torch.ones(1, 1, have, device="cuda"), C, cache=kept)
    k1, v1 = (x[:, :, have].contiguous() for x in (far, v))
    o = carve.swa_decode(q, k1, v1, *ring, ints([have]), C)
    o2, slot = carve.budget_decode(q, k1, v1, kept, ints([have]))
    for x in (o, o2):
        assert all(torch.equal(x[0, g], v1.view(D)) for g in range(Hq))
    assert int(slot) == have and float(kept[2][0, 0, have]) == Hq and (kept[2][0, 0, :have] == 1).all()


# ------------------------------------------------------------------ where the scores of a step are held
@pytest.mark.parametrize("B,Hq,Hkv,D,C,bits,dt", [
    (65, 8, 2, 128, 5884, 4, "bf16"), (65, 8, 2, 128, 1788, 8, "bf16"), (65, 8, 2, 64, 7996, 4, "f32"), (65, 8, 2, 64, 5948, 8, "bf16"),
    (2, 30, 1, 64, 1064, 4, "f32"), (129, 8, 2, 128, 860, 8, "bf16"), (129, 8, 2, 128, 860, 8, "f32"), (129, 2, 2, 64, 2940, 8, "bf16")])
def test_eviction_with_the_most_scores_in_lds(B, Hq, Hkv, D, C, bits, dt):
    """As many scores as LDS leaves room for, or nearly: a step without a workspace, against the definition."""
    s = carve.carve_budget_shape(B, Hq, Hkv, 1, D, C, 4, 20, D ** -0.5, 1 if dt == "bf16" else 0)
    assert carve.load_library().carve_budget_decode_mx_workspace_size(ctypes.byref(s), bits) == 0
    one_eviction(B, Hq, Hkv, D, C, bits, dt, empty=3)
