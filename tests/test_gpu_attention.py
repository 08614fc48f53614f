"""Windowed attention with sinks, its ring cache, and the cache kept by attention weight on the GPU,
against their float64 definitions (tests/attention_ref.py states the bounds)."""
import math

import pytest
import torch

from chunk_gated_delta_amd import carve
from chunk_gated_delta_amd.autograd import carve_attention, swa_attention
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(B, Hq, Hkv, T, D, dt, seed=0):
    return (normal((B, Hq, T, D), dt, seed), normal((B, Hkv, T, D), dt, seed + 1), normal((B, Hkv, T, D), dt, seed + 2),
            normal((B, Hq, T, D), dt, seed + 3))


# B, Hq, Hkv, T, D, window, sinks, lens
SWA = [
    (1, 1, 1, 1, 64, 1, 0, None),            # one token
    (2, 2, 1, 2, 128, 8, 1, None),
    (1, 2, 2, 33, 64, 1, 0, None),           # every token sees itself only
    (1, 2, 2, 40, 128, 1, 3, None),          # itself and the sinks
    (1, 4, 2, 127, 64, 16, 4, None),
    (2, 3, 1, 128, 128, 32, 0, None),
    (1, 8, 1, 129, 64, 129, 7, None),        # window = length
    (1, 4, 4, 257, 128, 500, 2, None),       # window past the length
    (3, 6, 2, 200, 64, 50, 3, [0, 1, 200]),  # a row without tokens, with one, a full one
    (2, 2, 1, 300, 128, 64, 200, [299, 130]),   # sinks over two key tiles
    (1, 2, 1, 700, 64, 33, 31, None),        # tokens far behind the sinks
    (1, 1, 1, 500, 128, 100, 500, None),     # every token a sink
    (4, 2, 1, 95, 64, 20, 64, [95, 64, 31, 1000]),   # a length past the end counts as T
]
ids = lambda c: "-".join(str(x).replace(" ", "") for x in c)  # noqa: E731


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", SWA, ids=ids)
def test_swa_forward_and_gradients(case, dt):
    B, Hq, Hkv, T, D, window, sinks, lens = case
    q, k, v, dO = inputs(B, Hq, Hkv, T, D, dt)
    want = ref.swa(q, k, v, window, sinks, None, lens, dO)
    if lens is not None:                      # whatever stands behind a sequence's end stays there
        for b, n in enumerate(lens):
            for x in (q, k, v, dO):
                x[b, :, n:] = math.nan
    at = dict(window=window, sinks=sinks, lens=ints(lens))
    o, lse = carve.swa_fwd(q, k, v, **at)
    g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.within(x, want[name], f"{name} {case} {dt}")


def test_swa_one_visible_key_has_no_score_gradient():
    """A token that sees itself only has o = v and ds = 0 exactly, in either pass."""
    for dt in DT:
        q, k, v, dO = inputs(2, 4, 2, 70, 128, dt, seed=9)
        o, lse = carve.swa_fwd(q, k, v, window=1)
        g = carve.swa_bwd(q, k, v, o, lse, dO, window=1)
        assert torch.equal(o, v.repeat_interleave(2, 1))
        assert not g["dq"].any() and not g["dk"].any()


@pytest.mark.parametrize("dt,window,sinks", [("bf16", 64, 4), ("bf16", 300, 130), ("f32", 40, 1)])
def test_swa_long(dt, window, sinks):
    """Many ranges of tokens behind the sinks' tiles, shared key heads, uneven lengths."""
    q, k, v, dO = inputs(2, 4, 2, 2777, 64, dt, seed=5)
    lens = [2777, 1501]
    want = ref.swa(q, k, v, window, sinks, 0.3, lens, dO)
    at = dict(window=window, sinks=sinks, scale=0.3, lens=ints(lens))
    o, lse = carve.swa_fwd(q, k, v, **at)
    g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.within(x, want[name], f"{name} {dt} {window} {sinks}")


def test_swa_large_scores():
    """Scores of several hundred: the running maximum moves by far more than a weight's range."""
    q, k, v, dO = inputs(1, 2, 1, 400, 64, "bf16", seed=3)
    q *= 16
    k = k * torch.linspace(0.1, 4, 400, device="cuda")[:, None].to(k.dtype)
    want = ref.swa(q, k, v, 150, 2, None, None, dO)
    o, lse = carve.swa_fwd(q, k, v, window=150, sinks=2)
    g = carve.swa_bwd(q, k, v, o, lse, dO, window=150, sinks=2)
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.within(x, want[name], name)


def test_swa_gradient_against_differences():
    """<g, d> against (L(x + h d) - L(x - h d)) / 2h of the float64 loss sum(o dO): the kernel's
    part within its bound, the difference's own error of third derivatives times h^2 / 6 and
    of rounding (1e-16 |L| / h) far below 1e-7 |L| at h = 1e-5."""
    q, k, v, dO = inputs(1, 4, 2, 90, 64, "f32", seed=11)
    at = dict(window=25, sinks=2)
    o, lse = carve.swa_fwd(q, k, v, **at)
    g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
    bounds = ref.swa(q, k, v, 25, 2, None, None, dO)

    def loss(q, k, v):
        return float((ref.swa(q, k, v, 25, 2, None, None)["o"][0] * dO.double()).sum())

    for i, (name, x) in enumerate((("dq", q), ("dk", k), ("dv", v))):
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(20 + i)).double().cuda()
        h = 1e-5
        hi, lo = [q.double(), k.double(), v.double()], [q.double(), k.double(), v.double()]
        hi[i], lo[i] = hi[i] + h * d, lo[i] - h * d
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        got = float((g[name].double() * d).sum())
        room = float((bounds[name][1] * d.abs()).sum()) + 1e-7 * abs(loss(q, k, v)) + 1e-6 * abs(slope)
        assert abs(got - slope) <= room, (name, got, slope, room)


def test_swa_same_bits_and_other_stream():
    q, k, v, dO = inputs(2, 8, 2, 600, 128, "bf16", seed=21)
    at = dict(window=100, sinks=4)

    def both():
        o, lse = carve.swa_fwd(q, k, v, **at)
        g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
        return [o, lse, g["dq"], g["dk"], g["dv"]]

    first = both()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        second = both()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    for x, y in zip(first, second):
        assert torch.equal(x, y)


def test_autograd_in_a_hybrid_block():
    """A delta-rule layer feeding a windowed attention layer: the autograd function's gradients are
    the library's, and they reach the layer below."""
    B, H, T, D = 2, 4, 130, 64
    q, k, v, dO = inputs(B, H, H, T, D, "bf16", seed=31)
    qn = torch.nn.functional.normalize(q.float(), dim=-1).to(q.dtype)
    kn = torch.nn.functional.normalize(k.float(), dim=-1).to(q.dtype)
    log_g = -0.1 * torch.rand(B, H, T, D, device="cuda")
    w = torch.rand(B, H, T, device="cuda")
    x, _ = carve_attention(qn, kn, v, log_g, w)
    leaves = [y.detach().clone().requires_grad_() for y in (q, k, x)]
    o = swa_attention(*leaves, window=40, sinks=2)
    o.backward(dO)
    o2, lse = carve.swa_fwd(*[y.detach() for y in leaves], window=40, sinks=2)
    g = carve.swa_bwd(*[y.detach() for y in leaves], o2, lse, dO, window=40, sinks=2)
    assert torch.equal(o, o2)
    for y, name in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(y.grad, g[name]), name
    vl = v.detach().clone().requires_grad_()
    x, _ = carve_attention(qn, kn, vl, log_g, w)
    swa_attention(q, k, x, window=40, sinks=2).backward(dO)
    assert vl.grad.shape == vl.shape and torch.isfinite(vl.grad.float()).all() and vl.grad.any()


def test_not_a_number_stays_with_its_token():
    """A query that is not a number gives a row that is not, and only that row."""
    for dt in DT:
        q, k, v, _ = inputs(1, 2, 1, 200, 64, dt, seed=33)
        want, lse = carve.swa_fwd(q, k, v, window=50, sinks=2)
        q[0, 1, 77, 5] = math.nan
        o, lse2 = carve.swa_fwd(q, k, v, window=50, sinks=2)
        assert torch.isnan(o[0, 1, 77].float()).all() and torch.isnan(lse2[0, 1, 77])
        rest = torch.ones(1, 2, 200, dtype=torch.bool, device="cuda")
        rest[0, 1, 77] = False
        assert torch.equal(o[rest], want[rest]) and torch.equal(lse2[rest], lse[rest])
        ck, cv = carve.swa_cache(1, 1, 64, 50, 2, dtype=DT[dt])
        o = carve.swa_decode(q[:, :, 77].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), ck, cv, ints([3]), 50, 2)
        assert torch.isnan(o[0, 1].float()).all() and torch.isfinite(o[0, 0].float()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_training_step_in_a_graph(dt):
    """Forward and backward captured and replayed with other inputs, against eager calls."""
    q, k, v, dO = inputs(2, 4, 2, 400, 128, dt, seed=35)
    at = dict(window=60, sinks=3, lens=ints([400, 222]))

    def step():
        o, lse = carve.swa_fwd(q, k, v, **at)
        g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
        return [o, lse, g["dq"], g["dk"], g["dv"]]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(4):
        for j, x in enumerate((q, k, v, dO)):
            x.copy_(normal(x.shape, dt, 500 + 4 * i + j))
        g.replay()
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_streams_at_once(dt):
    """Two training steps on two streams at the same time give what they give one after the other."""
    sets = [inputs(2, 8, 2, 900, 64, dt, seed=37 + 10 * i) for i in range(2)]
    at = dict(window=90, sinks=5)

    def step(q, k, v, dO):
        o, lse = carve.swa_fwd(q, k, v, **at)
        g = carve.swa_bwd(q, k, v, o, lse, dO, **at)
        return [o, g["dq"], g["dk"], g["dv"]]

    want = [step(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for st, x in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(step(*x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_autograd_shapes_of_gradients():
    """An output gradient that is a broadcast number, gradients asked for in part, and a captured
    forward and backward without leaves of an eager graph alive."""
    q, k, v, _ = inputs(2, 4, 2, 90, 64, "bf16", seed=39)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, v)]
    swa_attention(*leaves, window=20, sinks=1).float().sum().backward()
    o, lse = carve.swa_fwd(q, k, v, window=20, sinks=1)
    g = carve.swa_bwd(q, k, v, o, lse, torch.ones_like(o), window=20, sinks=1)
    for x, name in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(x.grad, g[name])
    kk = k.detach().clone().requires_grad_()
    only, = torch.autograd.grad(swa_attention(q, kk, v, window=20, sinks=1).float().sum(), kk)
    assert torch.equal(only, g["dk"])
    del leaves, kk
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = [y.detach().clone().requires_grad_() for y in (q, k, v)]
        for _ in range(2):
            torch.autograd.grad(swa_attention(*x, window=20, sinks=1), x, torch.ones_like(q))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(swa_attention(*x, window=20, sinks=1), x, torch.ones_like(q))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for y, name in zip(got, ("dq", "dk", "dv")):
            assert torch.equal(y, g[name])


def test_gradients_of_gradients_are_refused():
    q, k, v, _ = inputs(1, 2, 1, 20, 64, "f32", seed=49)
    q.requires_grad_()
    with pytest.raises(RuntimeError, match="gradients of gradients"):
        torch.autograd.grad(swa_attention(q, k, v, window=5).sum(), q, create_graph=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_heads_that_parts_do_not_divide(dt):
    """Five and seven heads on one, where a group's heads are cut into parts of two and of four."""
    case = dict(window=60, sinks=3)
    q, k, v, dO = inputs(9, 5, 1, 500, 64, dt, seed=51)
    lens = [500, 0, 1, 64, 65, 499, 333, 130, 500]
    want = ref.swa(q, k, v, 60, 3, None, lens, dO)
    o, lse = carve.swa_fwd(q, k, v, lens=ints(lens), **case)
    g = carve.swa_bwd(q, k, v, o, lse, dO, lens=ints(lens), **case)
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.within(x, want[name], name)
    q, k, v, _ = inputs(1, 7, 1, 1030, 64, dt, seed=53)
    w = carve.budget_weights(q, k, carve.swa_fwd(q, k, v, window=1030)[1])
    ref.within(w, ref.weights(q, k, 1030, 0, None, None), "weights")


def test_most_heads():
    """The largest accepted number of sequences and heads, a few tokens each: sampled rows."""
    B, T, D = 65535, 3, 64
    gen = torch.Generator(device="cuda").manual_seed(45)
    q, k, v, dO = (torch.randn(B, 1, T, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
    o, lse = carve.swa_fwd(q, k, v, window=2, sinks=1)
    g = carve.swa_bwd(q, k, v, o, lse, dO, window=2, sinks=1)
    w = carve.budget_weights(q, k, lse, window=2, sinks=1)
    at = torch.tensor([0, 1, 32767, 32768, 65534], device="cuda")
    want = ref.swa(q[at], k[at], v[at], 2, 1, None, None, dO[at])
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ref.within(x[at], want[name], name)
    ref.within(w[at], ref.weights(q[at], k[at], 2, 1, None, None), "weights")
    cache = carve.budget_keep(k, v, w, 2, sinks=1, recent=1)
    assert (cache[3][:, 0, 0] == 0).all() and (cache[3][:, 0, 1] == 2).all()
    assert torch.equal(cache[0][:, :, 1], k[:, :, 2])
    q1, k1, v1 = (x[:, :, 0].contiguous() for x in (q, k, v))
    pos = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    o1, slot = carve.budget_decode(q1, k1, v1, cache, pos, sinks=1, recent=1)
    assert (slot == 1).all() and torch.equal(cache[0][:, :, 1], k1)
    for b in at.tolist():
        x = ref.rows(q1[b, 0], cache[0][b, 0], cache[1][b, 0], torch.ones(2, dtype=torch.bool, device="cuda"), D ** -0.5)
        ref.within(o1[b, 0], x[:2], f"row {b}")


def test_longest_sequence():
    """2^20 tokens of one head: the last tokens against the definition, the sinks' gradients (which
    come from every token) through sum dq q = sum dk k, both sides sum ds s: each element off by at
    most half a step u twice (as a result, and in ds), so the sums by 2 u (sum |dq q| + sum |dk k|)."""
    T, D, window, sinks = 1 << 20, 64, 40, 3
    gen = torch.Generator(device="cuda").manual_seed(47)
    q, k, v, dO = (torch.randn(1, 1, T, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
    o, lse = carve.swa_fwd(q, k, v, window=window, sinks=sinks)
    g = carve.swa_bwd(q, k, v, o, lse, dO, window=window, sinks=sinks)
    n = 200                                    # tokens that the last n see: the sinks and the n + window last
    at = torch.cat([torch.arange(sinks, device="cuda"), torch.arange(T - n - window, T, device="cuda")])
    qq, kk, vv = q[:, :, at].contiguous(), k[:, :, at].contiguous(), v[:, :, at].contiguous()
    want = ref.swa(qq, kk, vv, window, sinks, None, None, dO[:, :, at].contiguous())
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"])):
        ref.within(x[:, :, T - n:], tuple(y[:, :, -n:] for y in want[name]), name)
    for name in ("dk", "dv"):
        ref.within(g[name][:, :, T - n:], tuple(y[:, :, -n:] for y in want[name]), name)
    a, b = g["dq"].double() * q.double(), g["dk"].double() * k.double()
    room = 2 * ref.half_step(q.dtype) * float(a.abs().sum() + b.abs().sum())
    assert abs(float(a.sum() - b.sum())) <= room
    # the sinks' own share of it is far above what a lost range of tokens could hide in
    s = (q[0, 0].double() @ k[0, 0, :sinks].double().T) * D ** -0.5
    p = torch.exp(s - lse[0, 0, :, None].double())
    t = torch.arange(T, device="cuda")[:, None]
    p = torch.where(t >= torch.arange(sinks, device="cuda"), p, 0.0)
    dv = p.T @ dO[0, 0].double()
    off = (g["dv"][0, 0, :sinks].double() - dv).abs()
    A = float((q[0, 0].double().abs() @ k[0, 0, :sinks].double().abs().T).max()) * D ** -0.5
    # a weight's error with lse as the kernel's; a range of at most T / 64 + 64 tokens summed, then 65 ranges
    e = ref.F32 * (2 * (2 * (D + 4) * A + 64 + 16) + T // 64 + 64 + 65)
    bound = ref.half_step(q.dtype) * dv.abs() + (ref.half_step(q.dtype) + e) * (p.T @ dO[0, 0].double().abs())
    assert (off <= bound).all()


# ------------------------------------------------------------------ ring cache
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,window,sinks,lens", [
    (2, 1, 64, 1500, 4, [1600, 900, 1503]), (24, 2, 128, 700, 0, [700, 699, 2000]),
    (4, 2, 64, 24, 3, [50, 0, 10]), (16, 1, 128, 7, 0, [5, 30, 1]), (6, 2, 64, 130, 64, [70, 300, 64]),
    (40, 1, 64, 50, 1, [20, 3, 90]), (3, 3, 128, 1, 0, [1, 2, 9]), (128, 2, 128, 200, 4, [0, 410, 199])])
def test_ring_cache_follows_the_sequence(Hq, Hkv, D, window, sinks, lens, dt):
    """A prompt's cache, then tokens one by one: each output is the windowed attention of the whole
    sequence at that token.  Row 1 skips a step."""
    B, steps, T = 3, 5, max(lens)
    q, k, v, _ = inputs(B, Hq, Hkv, T + steps, D, dt, seed=41)
    ck, cv = carve.swa_cache(B, Hkv, D, window, sinks, dtype=DT[dt])
    ck.fill_(math.nan)                        # slots without a token are not read
    cv.fill_(math.nan)
    kp, vp = k[:, :, :T].contiguous(), v[:, :, :T].contiguous()
    carve.swa_fill(kp, vp, ck, cv, window, sinks, lens=ints(lens))
    have = list(lens)
    for step in range(steps):
        row = torch.tensor(have, device="cuda")
        b = torch.arange(B, device="cuda")
        pos = [-1 if (i == 1 and step == 2) else n for i, n in enumerate(have)]
        before = ck.clone()
        o = carve.swa_decode(q[b, :, row].contiguous(), k[b, :, row].contiguous(), v[b, :, row].contiguous(), ck, cv,
                             ints(pos), window, sinks)
        for i in range(B):
            if pos[i] < 0:
                assert not o[i].any()
                assert torch.equal(ck[i].view(torch.int16), before[i].view(torch.int16))
                continue
            n = have[i]
            t = torch.arange(n + 1, device="cuda")
            see = (n - t < window) | (t < sinks)
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                x = ref.rows(q[i, h, n], k[i, kv, :n + 1], v[i, kv, :n + 1], see, D ** -0.5)
                ref.within(o[i, h], x[:2], f"step {step} row {i} head {h}")
            have[i] += 1


def test_ring_decode_ranges_agree_with_one_range():
    """A long window cut into slot ranges (one sequence) against the same sequence in a batch that
    needs none: the same rows to the rounding of o."""
    Hq, Hkv, D, window = 8, 2, 128, 3000
    q, k, v, _ = inputs(1, Hq, Hkv, 1, D, "bf16", seed=51)
    ck, cv = normal((1, Hkv, window + 4, D), "bf16", 52), normal((1, Hkv, window + 4, D), "bf16", 53)
    pos = ints([7001])
    one = carve.swa_decode(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(), ck.clone(),
                           cv.clone(), pos, window, 4)
    many = carve.swa_decode(*[x[:, :, 0].repeat(256, 1, 1) for x in (q, k, v)], ck.repeat(256, 1, 1, 1),
                            cv.repeat(256, 1, 1, 1), pos.repeat(256), window, 4)
    at = 4 + (7001 - 4) % window
    kk, vv = ck.clone(), cv.clone()
    kk[:, :, at], vv[:, :, at] = k[:, :, 0], v[:, :, 0]
    live = torch.ones(window + 4, dtype=torch.bool, device="cuda")
    for h in range(Hq):
        x = ref.rows(q[0, h, 0], kk[0, h // 4], vv[0, h // 4], live, D ** -0.5)
        for o in (one[0], many[0], many[255]):
            ref.within(o[h], x[:2], f"head {h}")


def test_decode_in_a_graph_follows_the_positions():
    """Captured decode steps of both caches, replayed with other inputs and positions, against the
    same steps run eagerly."""
    B, Hq, Hkv, D, window, sinks, C, recent = 2, 8, 2, 64, 30, 2, 20, 5
    q, k, v = normal((B, Hq, D), "bf16", 61), normal((B, Hkv, D), "bf16", 62), normal((B, Hkv, D), "bf16", 63)
    pos = ints([0, 7])
    ring = carve.swa_cache(B, Hkv, D, window, sinks)
    budget = carve.budget_cache(B, Hkv, D, C)

    def step(ring, budget):
        o1 = carve.swa_decode(q, k, v, *ring, pos, window, sinks)
        o2, slot = carve.budget_decode(q, k, v, budget, pos, sinks=sinks, recent=recent)
        return o1, o2, slot

    step(ring, budget)
    g = torch.cuda.CUDAGraph()
    for x in ring + budget[:3]:
        x.zero_()
    budget[3].fill_(-1)
    with torch.cuda.graph(g):
        got = step(ring, budget)
    mirror = [x.clone() for x in ring], tuple(x.clone() for x in budget)
    for i in range(40):
        for j, x in enumerate((q, k, v)):
            x.copy_(normal(x.shape, "bf16", 100 + 3 * i + j))
        g.replay()
        want = step(*mirror)
        torch.cuda.synchronize()
        for a, b in zip(list(got) + list(ring) + list(budget), list(want) + list(mirror[0]) + list(mirror[1])):
            assert torch.equal(a, b), i
        pos += 1


# ------------------------------------------------------------------ cache kept by weight
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,T,D,window,sinks,lens", [
    (1, 1, 1, 1, 64, None, 0, None), (2, 6, 2, 77, 128, None, 0, [77, 0]), (1, 14, 2, 11, 128, None, 0, None), (1, 4, 4, 129, 64, 30, 3, None),
    (2, 4, 1, 1030, 64, None, 0, [1030, 515]), (1, 2, 1, 900, 128, 100, 140, None)])
def test_weights(B, Hq, Hkv, T, D, window, sinks, lens, dt):
    q, k, v, _ = inputs(B, Hq, Hkv, T, D, dt, seed=71)
    want = ref.weights(q, k, T if window is None else window, sinks, None, lens)
    if lens is not None:
        for b, n in enumerate(lens):
            for x in (q, k, v):
                x[b, :, n:] = math.nan
    _, lse = carve.swa_fwd(q, k, v, window=window or T, sinks=sinks, lens=ints(lens))
    a = carve.budget_weights(q, k, lse, window=window, sinks=sinks, lens=ints(lens))
    ref.within(a, want, f"weights {dt}")


def keep_ref(w, n, C, sinks, recent):
    """Positions kept, from the definition."""
    safe = set(range(min(sinks, n))) | set(range(max(0, n - recent), n))
    order = lambda t: (0 if math.isnan(w[t]) else 1, 0 if math.isnan(w[t]) else -w[t], t)  # noqa: E731
    rest = sorted((t for t in range(n) if t not in safe), key=order)
    return sorted(list(safe) + rest[:max(0, C - len(safe))])


@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("T,C,sinks,recent,lens", [
    (0, 3, 1, 1, None), (1, 4, 1, 1, None), (10, 16, 2, 3, [10, 0]), (100, 33, 4, 8, [100, 61]), (1500, 200, 0, 1, [1500, 3]),
    (5000, 1024, 7, 100, [5000, 1200]), (64, 12, 4, 8, [64, 64]), (3000, 2999, 1, 5, None),
    (40000, 3001, 4, 50, [40000, 33333]), (50, 12, 4, 8, None)])
def test_keep(T, C, sinks, recent, lens, kind):
    B, Hkv, D = 2, 2, 64
    k, v = normal((B, Hkv, T, D), "bf16", 81), normal((B, Hkv, T, D), "bf16", 82)
    w = torch.rand(B, Hkv, T, generator=torch.Generator().manual_seed(83))
    if kind == "ties":
        w = torch.floor(w * 4)
    elif kind == "special":
        for i, x in enumerate((math.inf, math.nan, 0.0, -0.0, -1.0, 1e-42, -math.inf)):
            w[:, :, i::11] = x
    w = w.cuda()
    cache = carve.budget_cache(B, Hkv, D, C)
    for x in cache[:2]:
        x.fill_(5.0)
    out = carve.budget_keep(k, v, w, C, sinks=sinks, recent=recent, lens=ints(lens), cache=cache)
    assert all(x is y for x, y in zip(out, cache))
    for b in range(B):
        n = T if lens is None else lens[b]
        for h in range(Hkv):
            at = keep_ref(w[b, h].tolist(), n, C, sinks, recent)
            m = len(at)
            assert cache[3][b, h].tolist() == at + [-1] * (C - m)
            assert torch.equal(cache[2][b, h, :m].view(torch.int32), w[b, h, at].view(torch.int32))
            assert not cache[2][b, h, m:].any()
            for x, y in ((cache[0], k), (cache[1], v)):
                assert torch.equal(x[b, h, :m], y[b, h, at])
                assert (x[b, h, m:] == 5.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,C,sinks,recent,steps", [
    (4, 2, 64, 8, 1, 3, 20), (1, 1, 128, 1, 0, 1, 4), (16, 1, 64, 40, 4, 36, 60), (40, 2, 128, 9, 0, 1, 14),
    (6, 2, 64, 300, 2, 10, 6)])
def test_budget_decode_follows_its_rule(Hq, Hkv, D, C, sinks, recent, steps, dt):
    """Token after token from an empty cache (C = 300: from one that is nearly full) against the rule
    in float64: the slots are the same, outputs and weights within their bounds (the weights'
    bounds add up over the steps)."""
    B, G = 2, Hq // Hkv
    cache = carve.budget_cache(B, Hkv, D, C, dtype=DT[dt])
    cache[0].fill_(math.nan)                  # empty slots are not read
    cache[1].fill_(math.nan)
    cache[2].fill_(math.nan)
    start = 0
    if C == 300:
        start = 297
        cache[0][:, :, :start] = normal((B, Hkv, start, D), dt, 91)
        cache[1][:, :, :start] = normal((B, Hkv, start, D), dt, 92)
        cache[2][:, :, :start] = torch.rand(B, Hkv, start, generator=torch.Generator().manual_seed(93)).cuda()
        cache[3][:, :, :start] = torch.arange(start, dtype=torch.int32, device="cuda")
    mk, mv, mp = (cache[0].clone(), cache[1].clone(), cache[3].clone())
    mw, tw = cache[2].double().clone(), torch.zeros_like(cache[2], dtype=torch.float64)
    for step in range(steps):
        p = start + step
        pos = [p, -1 if step == 3 else p - (1 if step > 3 else 0)]
        q, k, v = normal((B, Hq, D), dt, 200 + step), normal((B, Hkv, D), dt, 300 + step), normal((B, Hkv, D), dt, 400 + step)
        o, slot = carve.budget_decode(q, k, v, cache, ints(pos), sinks=sinks, recent=recent)
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
                mk[b, h, at], mv[b, h, at], mp[b, h, at] = k[b, h], v[b, h], pos[b]
                mw[b, h, at], tw[b, h, at] = 0.0, 0.0
                live = mp[b, h] >= 0
                for g in range(h * G, (h + 1) * G):
                    x = ref.rows(q[b, g], mk[b, h], mv[b, h], live, D ** -0.5)
                    ref.within(o[b, g], x[:2], f"step {step} {b} {g}")
                    mw[b, h] += torch.where(live, x[2], 0.0)
                    tw[b, h] += torch.where(live, x[3] + 2 * ref.F32 * (mw[b, h].abs() + 1), 0.0)
        live = mp >= 0
        assert torch.equal(cache[3], mp)
        ref.within(torch.where(live, cache[2], 0.0), (torch.where(live, mw, 0.0), tw + ref.F32 * mw.nan_to_num().abs()), f"weights {step}")
        for x, y in ((cache[0], mk), (cache[1], mv)):
            assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


def test_budget_decode_ties_specials_and_repeats():
    B, Hkv, D, C = 1, 1, 64, 6
    q, k, v = normal((B, 1, D), "bf16", 1), normal((B, 1, D), "bf16", 2), normal((B, 1, D), "bf16", 3)

    def slot_of(w, held, pos, sinks=1, recent=2):
        cache = carve.budget_cache(B, Hkv, D, C)
        cache[2].copy_(torch.tensor(w).view(1, 1, C))
        cache[3].copy_(torch.tensor(held, dtype=torch.int32).view(1, 1, C))
        _, slot = carve.budget_decode(q, k, v, cache, ints([pos]), sinks=sinks, recent=recent)
        assert int(cache[3][0, 0, int(slot)]) == pos
        return int(slot)

    held = [0, 1, 2, 3, 4, 9]
    assert slot_of([0.0, 2.0, 1.0, 1.0, 5.0, 0.0], held, 10) == 2            # the lowest of equal weights
    assert slot_of([0.0, math.nan, 7.0, math.inf, 8.0, 0.0], held, 10) == 2  # not a number is the largest
    assert slot_of([0.0, 2.0, -0.0, 0.0, 5.0, 0.0], held, 10) == 2
    assert slot_of([0.0, 2.0, 1.0, -3.0, 5.0, 0.0], held, 10) == 3
    assert slot_of([9.0, 0.0, 1.0, 1.0, 5.0, 0.0], [0, 1, -1, -7, 4, 9], 10) == 2    # the lowest empty one
    assert slot_of([9.0, 0.0, 1.0, 1.0, 5.0, 0.0], [0, 10, -1, -7, 4, 9], 10) == 1   # repeated: the same slot
    # the call repeated stores the token once
    cache = carve.budget_cache(B, Hkv, D, C)
    for _ in range(3):
        _, slot = carve.budget_decode(q, k, v, cache, ints([0]), sinks=1, recent=2)
        assert int(slot) == 0
    assert cache[3][0, 0].tolist() == [0, -1, -1, -1, -1, -1]
    assert float(cache[2][0, 0, 0]) == 1.0


def test_budget_decode_ranges():
    """One sequence on a large cache (slot ranges joined by a second launch): outputs, weights, slot."""
    Hq, Hkv, D, C = 8, 2, 128, 2500
    cache = (normal((1, Hkv, C, D), "bf16", 5), normal((1, Hkv, C, D), "bf16", 6),
             torch.rand(1, Hkv, C, generator=torch.Generator().manual_seed(7)).cuda(),
             torch.arange(C, dtype=torch.int32, device="cuda").repeat(1, Hkv, 1))
    was = [x.clone() for x in cache]
    q, k, v = normal((1, Hq, D), "bf16", 8), normal((1, Hkv, D), "bf16", 9), normal((1, Hkv, D), "bf16", 10)
    o, slot = carve.budget_decode(q, k, v, cache, ints([C]), sinks=4, recent=100)
    for h in range(Hkv):
        at = 4 + int(was[2][0, h, 4:C - 99].argmin())
        assert int(slot[0, h]) == at
        kk, vv = was[0][0, h].clone(), was[1][0, h].clone()
        kk[at], vv[at] = k[0, h], v[0, h]
        w, tol = was[2][0, h].double(), torch.zeros(C, dtype=torch.float64, device="cuda")
        w[at] = 0.0
        for g in range(h * 4, h * 4 + 4):
            x = ref.rows(q[0, g], kk, vv, torch.ones(C, dtype=torch.bool, device="cuda"), D ** -0.5)
            ref.within(o[0, g], x[:2], f"head {g}")
            w, tol = w + x[2], tol + x[3]
        ref.within(cache[2][0, h], (w, tol + 5 * ref.F32 * w.abs()), "weights")
        assert torch.equal(cache[0][0, h], kk) and torch.equal(cache[1][0, h], vv)
        assert int(cache[3][0, h, at]) == C


def test_prompt_to_budget_cache_to_tokens():
    """The operators as they are used together: a prompt's attention, its weights, the cache kept by
    them, and tokens decoded on it."""
    B, Hq, Hkv, T, D, C, sinks, recent = 2, 8, 2, 400, 64, 96, 4, 16
    q, k, v, _ = inputs(B, Hq, Hkv, T, D, "bf16", seed=111)
    lens = [400, 250]
    _, lse = carve.swa_fwd(q, k, v, window=T, lens=ints(lens))
    a = carve.budget_weights(q, k, lse, lens=ints(lens))
    cache = carve.budget_keep(k, v, a, C, sinks=sinks, recent=recent, lens=ints(lens))
    for b, n in enumerate(lens):
        # every token's weights sum to one
        assert abs(float(a[b].double().sum()) - n * Hq) <= 1e-4 * n * Hq
        for h in range(Hkv):
            assert cache[3][b, h].tolist() == keep_ref(a[b, h].tolist(), n, C, sinks, recent)
    pos = ints(lens)
    for step in range(4):
        q1, k1, v1 = normal((B, Hq, D), "bf16", 120 + step), normal((B, Hkv, D), "bf16", 130 + step), normal((B, Hkv, D), "bf16", 140 + step)
        before = cache[2].double().sum((1, 2))
        o, slot = carve.budget_decode(q1, k1, v1, cache, pos, sinks=sinks, recent=recent)
        assert torch.isfinite(o.float()).all()
        for b in range(B):
            held = cache[3][b].tolist()
            assert all(sorted(h) != [] and set(range(sinks)) <= set(h) for h in held)
            assert all(set(range(int(pos[b]) - recent + 1, int(pos[b]) + 1)) <= set(h) for h in held)
        pos += 1
