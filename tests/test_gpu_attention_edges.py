"""Edges of the attention operators on the GPU: values that are not numbers, scores of any size, and
the variants that only some sizes reach, against the definitions in float64 (tests/attention_ref.py
states the bounds)."""
import math

import pytest
import torch

from chunk_gated_delta_amd import carve
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(B, Hq, Hkv, T, D, dt, seed):
    return (normal((B, Hq, T, D), dt, seed), normal((B, Hkv, T, D), dt, seed + 1), normal((B, Hkv, T, D), dt, seed + 2),
            normal((B, Hq, T, D), dt, seed + 3))


def same(x, y):
    """Equal bits."""
    kind = torch.int16 if x.dtype is torch.bfloat16 else torch.int32
    return torch.equal(x.contiguous().view(kind), y.contiguous().view(kind))


# ------------------------------------------------------------------ values that are not numbers
REACH = 192          # a key or value that is not finite stays within this many tokens of those that see it


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,sinks,at", [
    (64, 4, (10, 31, 40, 63)), (128, 1, (1, 20)), (64, 40, (45, 63, 64)), (128, 70, (75, 127))])
def test_not_finite_keys_beside_the_sinks(D, sinks, at, dt):
    """A key and a value beside the sinks that are not finite: past their window (and the tiles
    that see it) every output, gradient of a query, key and value is what it is without them."""
    B, Hq, Hkv, T, window = 1, 4, 2, 900, 100
    q, k, v, dO = inputs(B, Hq, Hkv, T, D, dt, seed=3)

    def step(k, v):
        o, lse = carve.swa_fwd(q, k, v, window, sinks=sinks)
        g = carve.swa_bwd(q, k, v, o, lse, dO, window, sinks=sinks)
        return dict(o=o, lse=lse, dq=g["dq"], dk=g["dk"], dv=g["dv"])

    want = step(k, v)
    for bad in (math.nan, math.inf):
        for which in (0, 1):
            kv = [k.clone(), v.clone()]
            for s in at:
                kv[which][0, 1, s, 5] = bad
            got = step(*kv)
            clean = max(at) + window + REACH         # the first token that none of them reaches
            for name, x in got.items():
                assert same(x[:, :, clean:], want[name][:, :, clean:]), (name, bad, which)
                heads = slice(0, 2 if name in ("o", "lse", "dq") else 1)       # of the other key head
                assert same(x[:, heads], want[name][:, heads]), (name, bad, which)
            # and what sees one that is not a number is not one itself
            if bad is math.nan:
                assert torch.isnan(got["o"][0, 2:, max(at), 5].float()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (50, 3)])
def test_weights_of_a_query_that_is_not_a_number(window, sinks, dt):
    """It gives the keys that its token sees weights that are not, and no other key."""
    T, t = 300, 77
    q, k, v, _ = inputs(1, 4, 2, T, 64, dt, seed=7)

    def weights(q):
        _, lse = carve.swa_fwd(q, k, v, window=window or T, sinks=sinks)
        return carve.budget_weights(q, k, lse, window=window, sinks=sinks)

    want = weights(q)
    q2 = q.clone()
    q2[0, 1, t, 9] = math.nan
    got = weights(q2)
    s = torch.arange(T, device="cuda")
    sees = (s <= t) & ((t - s < (window or T)) | (s < sinks))
    assert torch.isnan(got[0, 0, sees]).all()
    assert same(got[0, 0, ~sees], want[0, 0, ~sees]) and same(got[0, 1], want[0, 1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks,t", [(20, 2, 77), (90, 0, 200), (90, 5, 130)])
def test_gradients_of_an_output_that_is_not_a_number(window, sinks, t, dt):
    """One token's output row that is not a number (its delta is not): its dq, and dk of the keys
    that it sees, are not; everything else is what it is without it."""
    T = 300
    q, k, v, dO = inputs(1, 4, 2, T, 64, dt, seed=13)
    o, lse = carve.swa_fwd(q, k, v, window, sinks=sinks)
    want = carve.swa_bwd(q, k, v, o, lse, dO, window, sinks=sinks)
    o[0, 1, t, 9] = math.nan
    got = carve.swa_bwd(q, k, v, o, lse, dO, window, sinks=sinks)
    s = torch.arange(T, device="cuda")
    sees = (s <= t) & ((t - s < window) | (s < sinks))
    assert torch.isnan(got["dq"][0, 1, t].float()).all()
    got["dq"][0, 1, t] = want["dq"][0, 1, t]
    assert same(got["dq"], want["dq"]) and same(got["dv"], want["dv"])
    assert torch.isnan(got["dk"][0, 0, sees].float()).all()
    assert same(got["dk"][0, 0, ~sees], want["dk"][0, 0, ~sees]) and same(got["dk"][0, 1], want["dk"][0, 1])


# ------------------------------------------------------------------ variants that only some sizes reach
def kept(w, n, C, sinks, recent):
    """Positions that a prompt's cache keeps, from the definition (w without NaN)."""
    safe = set(range(min(sinks, n))) | set(range(max(0, n - recent), n))
    rest = sorted((t for t in range(n) if t not in safe), key=lambda t: (-w[t], t))
    return sorted(list(safe) + rest[:max(0, C - len(safe))])


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("T,C,sinks,recent,lens", [
    (37, 20, 2, 5, [37, 12]),                      # a key a lane
    (4096, 700, 4, 64, [4096, 1]), (4097, 700, 4, 64, [4097, 4096]),       # 4 and 12 keys a lane
    (12288, 900, 4, 64, [12288, 700]), (12289, 900, 4, 64, [12289, 0]),    # 12 and 32
    (20000, 3001, 4, 50, [20000, 300]),            # far more room than the sequence has tokens
    (32768, 1500, 0, 1, [32768, 16385]), (32769, 1500, 7, 1, [32769, 900])])     # 32 and 64
def test_keep_at_every_length(T, C, sinks, recent, lens, dt, D):
    B, Hkv = 2, 2
    k, v = normal((B, Hkv, T, D), dt, 21), normal((B, Hkv, T, D), dt, 22)
    w = torch.exp(2 * torch.randn(B, Hkv, T, generator=torch.Generator().manual_seed(23)))
    w[:, 1] = torch.floor(w[:, 1] * 2)             # many equal weights
    w = w.cuda()
    cache = carve.budget_cache(B, Hkv, D, C, dtype=DT[dt])
    for x in cache[:2]:
        x.fill_(5.0)
    carve.budget_keep(k, v, w, C, sinks=sinks, recent=recent, lens=ints(lens), cache=cache)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            at = kept(w[b, h].tolist(), n, C, sinks, recent)
            m = len(at)
            assert cache[3][b, h].tolist() == at + [-1] * (C - m)
            assert same(cache[2][b, h, :m], w[b, h, at]) and not cache[2][b, h, m:].any()
            for x, y in ((cache[0], k), (cache[1], v)):
                assert same(x[b, h, :m], y[b, h, at]) and (x[b, h, m:] == 5.0).all()


def one_token(B, Hq, Hkv, D, C, sinks, recent, dt, empty, skip, rows=None, seed=31):
    """One step on a cache made for it, against the rule in float64: slots, rows and positions the
    same, outputs and weights within their bounds (a weight is a sum of G + 1 terms).  `empty` slots of every
    key head hold nothing; row `skip` has no token; `rows`: sequences to check."""
    G = Hq // Hkv
    gen = torch.Generator().manual_seed(seed)
    cache = (normal((B, Hkv, C, D), dt, seed + 1), normal((B, Hkv, C, D), dt, seed + 2),
             torch.exp(torch.randn(B, Hkv, C, generator=gen)).cuda(), torch.empty(B, Hkv, C, dtype=torch.int32, device="cuda"))
    p = 3 * C
    # the first and the recent tokens, and positions between in a mixed order
    middle = sinks + torch.randperm(p - recent - sinks, generator=gen)[:C - sinks - recent + 1]
    held = torch.cat([torch.arange(sinks), middle, torch.arange(p - recent + 1, p)]).to(torch.int32)
    cache[3].copy_(held.cuda().expand(B, Hkv, C))
    holes = (torch.arange(C) * 7 % C < empty) & (held >= sinks) & (held <= p - recent)
    for x, y in zip(cache, (math.nan, math.nan, math.nan, -1)):           # an empty slot's rows are not read
        x[:, :, holes.cuda()] = y
    was = [x.clone() for x in cache]
    q, k, v = normal((B, Hq, D), dt, seed + 3), normal((B, Hkv, D), dt, seed + 4), normal((B, Hkv, D), dt, seed + 5)
    pos = [-1 if b == skip else p for b in range(B)]
    o, slot = carve.budget_decode(q, k, v, cache, ints(pos), sinks=sinks, recent=recent)
    for b in range(B) if rows is None else rows:
        if b == skip:
            assert not o[b].any() and (slot[b] == -1).all()
            assert all(same(x[b], y[b]) for x, y in zip(cache, was))
            continue
        for h in range(Hkv):
            w, hold = was[2][b, h].tolist(), was[3][b, h].tolist()
            if holes.any():
                at = hold.index(-1)
            else:
                at = min((j for j in range(C) if sinks <= hold[j] <= p - recent), key=lambda j: (w[j], j))
            assert int(slot[b, h]) == at
            kk, vv, pp, ww = was[0][b, h], was[1][b, h], was[3][b, h], was[2][b, h].double()
            kk[at], vv[at], pp[at], ww[at] = k[b, h], v[b, h], p, 0.0
            assert same(cache[0][b, h], kk) and same(cache[1][b, h], vv) and torch.equal(cache[3][b, h], pp)
            live, tol = pp >= 0, torch.zeros(C, dtype=torch.float64, device="cuda")
            for g in range(h * G, (h + 1) * G):
                x = ref.rows(q[b, g], kk, vv, live, D ** -0.5)
                ref.within(o[b, g], x[:2], f"row {b} head {g}")
                ww, tol = ww + x[2], tol + x[3]
            ref.within(cache[2][b, h][live], (ww[live], (tol + (G + 1) * ref.F32 * ww.abs())[live]), f"weights {b} {h}")
            assert same(cache[2][b, h][~live], was[2][b, h][~live])


@pytest.mark.parametrize("Hq,Hkv,D,C", [
    (16, 2, 128, 512), (16, 2, 128, 516),          # eight waves: 4,096 scores and the first size past it
    (16, 2, 64, 511), (16, 2, 64, 513), (16, 2, 64, 514),                  # slots that four do not divide
    (32, 2, 64, 1021), (4, 4, 64, 4096), (4, 4, 64, 2000)])
@pytest.mark.parametrize("empty", [0, 5])
def test_eviction_by_eight_waves(Hq, Hkv, D, C, empty):
    one_token(2, Hq, Hkv, D, C, 4, 37, "bf16", empty, skip=None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,C", [
    (8, 2, 128, 2500), (20, 1, 64, 5301), (40, 1, 64, 5302), (64, 1, 128, 2603), (5, 1, 128, 1411)])
@pytest.mark.parametrize("empty", [0, 300])
def test_eviction_in_joined_ranges(Hq, Hkv, D, C, empty, dt):
    one_token(3, Hq, Hkv, D, C, 4, 100, dt, empty, skip=1)


@pytest.mark.parametrize("Hq,C", [(4, 500), (8, 2049), (68, 70)])
@pytest.mark.parametrize("D", [64, 128])
def test_eviction_in_batches_of_about_300_key_heads(Hq, C, D):
    one_token(75, Hq, 4, D, C, 4, 20, "bf16", 3, skip=11, rows=(0, 11, 63, 64, 74))


def test_weight_is_conserved_from_prompt_to_tokens():
    """A prompt's weights, the cache kept by them and tokens decoded on it: what a step adds to a
    key head's weights is one for every query head of its group, less what left with the token that gave up
    its slot; outputs are attention over the cache as the step leaves it; positions are distinct.  The sum
    of a token's weights is off by their bound (attention_ref.rows), the cache's sum by one
    rounding of each weight."""
    B, Hq, Hkv, T, D, C, sinks, recent = 2, 8, 2, 400, 64, 96, 4, 16
    G = Hq // Hkv
    q, k, v, _ = inputs(B, Hq, Hkv, T, D, "bf16", seed=41)
    lens = [400, 60]
    _, lse = carve.swa_fwd(q, k, v, window=T, lens=ints(lens))
    w = carve.budget_weights(q, k, lse, lens=ints(lens))
    cache = carve.budget_keep(k, v, w, C, sinks=sinks, recent=recent, lens=ints(lens))
    pos = ints(lens)
    for step in range(50):                         # the second row fills its empty slots, then gives up some
        was = [x.clone() for x in cache]
        q1, k1, v1 = (normal((B, h, D), "bf16", 50 + 3 * step + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        o, slot = carve.budget_decode(q1, k1, v1, cache, pos, sinks=sinks, recent=recent)
        for b in range(B):
            for h in range(Hkv):
                at, live = int(slot[b, h]), cache[3][b, h] >= 0
                held = cache[3][b, h][live].tolist()
                assert len(set(held)) == len(held) and held[int(live[:at].sum())] == int(pos[b])
                assert int(live.sum()) == min(C, int((was[3][b, h] >= 0).sum()) + (int(was[3][b, h, at]) < 0))
                assert set(range(sinks)) | set(range(int(pos[b]) - recent + 1, int(pos[b]) + 1)) <= set(held)
                assert same(cache[0][b, h, at], k1[b, h]) and same(cache[1][b, h, at], v1[b, h])
                tol = ref.F32 * cache[2][b, h].double().abs().sum()
                for g in range(h * G, (h + 1) * G):
                    x = ref.rows(q1[b, g], cache[0][b, h], cache[1][b, h], live, D ** -0.5)
                    ref.within(o[b, g], x[:2], f"step {step} {b} {g}")
                    tol += x[3].sum() + G * ref.F32
                grown = cache[2][b, h].double().sum() - was[2][b, h].double().sum() + was[2][b, h, at].double()
                assert abs(float(grown) - G) <= float(tol), (step, b, h)
        pos += 1


@pytest.mark.parametrize("T,C,lens", [(65536, 2000, [65536, 40000]), (65537, 2000, [65537, 65536])])
def test_keep_of_the_longest_prompts_in_registers(T, C, lens):
    """The largest register variant and the first length that reads its weights again."""
    k = normal((2, 1, T, 64), "bf16", 61)
    w = torch.exp(2 * torch.randn(2, 1, T, generator=torch.Generator().manual_seed(62)))
    w[1] = torch.floor(w[1] * 2)
    w = w.cuda()
    cache = carve.budget_keep(k, k, w, C, sinks=5, recent=100, lens=ints(lens))
    for b, n in enumerate(lens):
        at = kept(w[b, 0].tolist(), n, C, 5, 100)
        assert cache[3][b, 0].tolist() == at
        assert same(cache[2][b, 0], w[b, 0, at]) and same(cache[0][b, 0], k[b, 0, at]) and same(cache[1][b, 0], k[b, 0, at])
