"""Decode steps on caches in codes where one rounding decides the result (tests/mx_ref.py states the definition and the
bounds)."""
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
