"""Timed cases of the attention operators whose memory per sequence is fixed.

The operators (sequence layouts [B, H, T, D], as everywhere in this library):

  swa     attention with a sliding window and sinks: token t sees s when s <= t and
          (t - s < window or s < sinks); the forward pass (a prompt) and the training step
  decode  its form for one new token, on a ring cache of sinks + window slots
  weight  the attention weight every token of a prompt receives, summed over queries and
          over the heads that share its key
  keep    the cache of a fixed number of slots made from a prompt by those weights
  evict   one new token on that cache: it takes an empty slot or that of the least weight,
          attends, and adds its attention weights to the cache's

`run` computes them in plain torch operations in 32 bits, or calls the library (`own`).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt of one conversation: launch latency
        dict(name="swa_prompt_short", op="swa", train=False, B=1, Hq=16, Hkv=4, T=256, D=128, window=128, sinks=4,
             ragged=False, dtype="bf16"),
        # a long document read in one pass
        dict(name="swa_prompt_long", op="swa", train=False, B=1, Hq=16, Hkv=4, T=32768, D=128, window=2048, sinks=4,
             ragged=False, dtype="bf16"),
        # the windowed layer of a training step at the benchmark's batch, heads and length
        dict(name="swa_train", op="swa", train=True, B=4, Hq=16, Hkv=4, T=4096, D=128, window=1024, sinks=4,
             ragged=False, dtype="bf16"),
        # a padded batch of odd lengths in full precision (a small model, or a check of gradients)
        dict(name="swa_train_f32", op="swa", train=True, B=3, Hq=6, Hkv=2, T=777, D=64, window=100, sinks=3,
             ragged=True, dtype="f32"),
        # one conversation, one token: latency
        dict(name="decode_one", op="decode", B=1, Hq=16, Hkv=4, D=128, window=1024, sinks=4, ragged=False, dtype="bf16"),
        # a full serving batch with long windows: the cache's bandwidth
        dict(name="decode_batch", op="decode", B=256, Hq=16, Hkv=4, D=128, window=4096, sinks=4, ragged=True,
             dtype="bf16"),
        # the weights of a padded batch of prompts
        dict(name="weight_batch", op="weight", B=4, Hq=16, Hkv=4, T=1000, D=64, ragged=True, dtype="bf16"),
        # the weights of a long prompt
        dict(name="weight_long", op="weight", B=1, Hq=16, Hkv=4, T=8192, D=128, ragged=False, dtype="bf16"),
        # a short prompt into a small cache, and a long one into a large cache
        dict(name="keep_short", op="keep", B=1, Hkv=4, T=500, D=128, C=256, sinks=4, recent=32, ragged=False,
             dtype="bf16"),
        dict(name="keep_long", op="keep", B=8, Hkv=4, T=32768, D=128, C=4096, sinks=4, recent=1024, ragged=True,
             dtype="bf16"),
        # one conversation on a small cache; a serving batch on large ones, some still filling
        dict(name="evict_one", op="evict", B=1, Hq=16, Hkv=4, D=128, C=512, sinks=4, recent=64, ragged=False,
             dtype="bf16"),
        dict(name="evict_batch", op="evict", B=64, Hq=16, Hkv=4, D=128, C=2048, sinks=4, recent=256, ragged=True,
             dtype="bf16"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["swa", "swa", "decode", "weight", "keep", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, B=log_int(1, 16), Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, D=rng.choice([64, 128]),
             ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "swa":
        c.update(train=rng.random() < 0.6, T=log_int(1, 2048), window=log_int(1, 1024), sinks=rng.choice([0, 1, 4, 7, 64]))
        c["B"] = min(c["B"], 8)
        if c["dtype"] == "f32":
            c["T"] = min(c["T"], 1024)
    elif op == "decode":
        c.update(window=log_int(16, 4096), sinks=rng.choice([0, 1, 4, 7, 64]))
    elif op == "weight":
        c.update(T=log_int(1, 2048), B=min(c["B"], 4))
    elif op == "keep":
        del c["Hq"]
        C = log_int(16, 2048)
        c.update(T=log_int(16, 16384), C=C, sinks=rng.randint(0, C // 8), recent=rng.randint(1, C // 2))
    else:
        C = log_int(16, 2048)
        c.update(C=C, sinks=rng.randint(0, C // 8), recent=rng.randint(1, C // 2))
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    def between(lo, hi, n):       # n whole numbers of [lo, hi]
        return torch.randint(lo, hi + 1, (n,), generator=gen, device=dev, dtype=torch.int32)

    s = dict(case)
    if case["op"] in ("swa", "weight"):
        T, Hq = case["T"], case["Hq"]
        s.update(q=normal(B, Hq, T, D), k=normal(B, Hkv, T, D), v=normal(B, Hkv, T, D))
        s["lens"] = between((T + 1) // 2, T, B) if case["ragged"] else None
        if case.get("train"):
            s["dO"] = normal(B, Hq, T, D)
        if case["op"] == "weight":  # the prompt's forward pass has run: its log-sum-exp is at hand
            s["lse"] = _lse(s["q"], s["k"], s["lens"])
    elif case["op"] == "decode":
        Hq, C = case["Hq"], case["window"] + case["sinks"]
        s.update(q=normal(B, Hq, D), k=normal(B, Hkv, D), v=normal(B, Hkv, D))
        s.update(cache_k=normal(B, Hkv, C, D), cache_v=normal(B, Hkv, C, D))
        # tokens before this one: sequences that fill their window, or (ragged) some that do not
        s["pos"] = between(C // 2 if case["ragged"] else 2 * C, 4 * C, B)
    elif case["op"] == "keep":
        T, C = case["T"], case["C"]
        s.update(k=normal(B, Hkv, T, D), v=normal(B, Hkv, T, D))
        # accumulated weights: positive, a few heavy tokens
        s["weights"] = torch.exp(2 * torch.randn(B, Hkv, T, generator=gen, device=dev))
        s["lens"] = between((T + 1) // 2, T, B) if case["ragged"] else None
        s.update(cache_k=torch.zeros(B, Hkv, C, D, device=dev, dtype=dt),
                 cache_v=torch.zeros(B, Hkv, C, D, device=dev, dtype=dt),
                 cache_w=torch.zeros(B, Hkv, C, device=dev), cache_pos=torch.zeros(B, Hkv, C, device=dev, dtype=torch.int32))
    else:
        Hq, C = case["Hq"], case["C"]
        s.update(q=normal(B, Hq, D), k=normal(B, Hkv, D), v=normal(B, Hkv, D))
        s.update(cache_k=normal(B, Hkv, C, D), cache_v=normal(B, Hkv, C, D))
        s["pos"] = between(C // 2 if case["ragged"] else 2 * C, 4 * C, B)
        # the positions a slot holds: its own index while the cache fills; after that the first
        # tokens, the recent ones, and a share of those between, in order
        slot = torch.arange(C, device=dev)[None, None]
        p = s["pos"].long()[:, None, None]
        old = C - case["sinks"] - (case["recent"] - 1)       # slots of neither kind
        gap = (p - case["recent"] + 1 - case["sinks"]).clamp(min=1)
        middle = case["sinks"] + (slot - case["sinks"]) * gap // max(old, 1)
        held = torch.where(slot < case["sinks"], slot, torch.where(slot < case["sinks"] + old, middle, p - C + slot))
        held = torch.where(p >= C, held, torch.where(slot < p, slot, torch.full_like(slot, -1)))
        s["cache_pos"] = held.expand(B, Hkv, C).to(torch.int32).contiguous()
        s["cache_w"] = torch.where(s["cache_pos"] >= 0, torch.exp(torch.randn(B, Hkv, C, generator=gen, device=dev)), 0.0)
    return s


def _lse(q, k, lens):
    """log-sum-exp of the full causal scores, [B, Hq, T] (-inf past a sequence's end)."""
    B, Hq, T, D = q.shape
    t = torch.arange(T, device=q.device)
    out = torch.empty(B, Hq, T, device=q.device)
    for h in range(Hq):
        s = torch.matmul(q[:, h].double(), k[:, h * k.shape[1] // Hq].double().transpose(-1, -2)) / math.sqrt(D)
        out[:, h] = torch.logsumexp(s.masked_fill(t[None, :] > t[:, None], -math.inf), -1).float()
    if lens is not None:
        out.masked_fill_((t >= lens[:, None])[:, None], -math.inf)
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"swa": _swa, "decode": _decode, "weight": _weight, "keep": _keep, "evict": _evict}[s["op"]](s)


def _own(s):
    from chunk_gated_delta_amd import carve
    if s["op"] == "swa":
        at = dict(window=s["window"], sinks=s["sinks"], lens=s["lens"])
        o, lse = carve.swa_fwd(s["q"], s["k"], s["v"], **at)
        if not s["train"]:
            return o, lse
        g = carve.swa_bwd(s["q"], s["k"], s["v"], o, lse, s["dO"], **at)
        return o, g["dq"], g["dk"], g["dv"]
    if s["op"] == "decode":
        o = carve.swa_decode(s["q"], s["k"], s["v"], s["cache_k"], s["cache_v"], s["pos"], window=s["window"],
                             sinks=s["sinks"])
        return o, s["cache_k"], s["cache_v"]
    if s["op"] == "weight":
        return carve.budget_weights(s["q"], s["k"], s["lse"], lens=s["lens"])
    cache = (s["cache_k"], s["cache_v"], s["cache_w"], s["cache_pos"])
    if s["op"] == "keep":
        return carve.budget_keep(s["k"], s["v"], s["weights"], s["C"], sinks=s["sinks"], recent=s["recent"],
                                 lens=s["lens"], cache=cache)
    o, slot = carve.budget_decode(s["q"], s["k"], s["v"], cache, s["pos"], sinks=s["sinks"], recent=s["recent"])
    return (o, slot) + cache


# ---- plain forms: 32 bits throughout, rounded once at the end
def _softmax(x):
    """Weights and log-sum-exp over the last axis; rows of -inf only give zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m.clamp(min=-1e30))
    z = e.sum(-1, keepdim=True)
    return e / z.clamp(min=1e-30), (m + torch.log(z))[..., 0]


def _swa_forward(q, k, v, window, sinks, lens):
    """o, lse of 32-bit q [B,Hkv,G,T,D], k, v [B,Hkv,T,D].  Blocks of c >= window tokens: the
    queries of a block see keys of their own and of the block before, and the sinks apart."""
    B, Hkv, G, T, D = q.shape
    dev = q.device
    c = min(window, T)
    n = -(-T // c)
    pad = n * c - T
    ns = min(sinks, T)
    tq = torch.arange(n * c, device=dev).view(n, c)
    ts = torch.cat([tq - c, tq], 1)                                        # keys of a block's queries
    see = (ts[:, None] >= 0) & (ts[:, None] <= tq[:, :, None]) & (tq[:, :, None] - ts[:, None] < window)
    first = torch.arange(ns, device=dev)
    see_s = (tq[:, :, None] - first >= window)                             # sinks behind the window
    zero = q.new_zeros(())

    def blocks(x):                                                         # two neighbouring blocks of every block
        x = torch.nn.functional.pad(x, (0, 0, c, pad)).view(B, Hkv, n + 1, c, D)
        return torch.cat([x[:, :, :-1], x[:, :, 1:]], 3)[:, :, None]

    qb = torch.nn.functional.pad(q, (0, 0, 0, pad)).view(B, Hkv, G, n, c, D)
    x = torch.matmul(qb, blocks(k).transpose(-1, -2)) / math.sqrt(D)
    xs = torch.matmul(qb, k[:, :, None, None, :ns].transpose(-1, -2)) / math.sqrt(D)
    x = torch.cat([x.masked_fill(~see, -math.inf), xs.masked_fill(~see_s, -math.inf)], -1)
    p, lse = _softmax(x)
    o = torch.matmul(p[..., :2 * c], blocks(v)) + torch.matmul(p[..., 2 * c:], v[:, :, None, None, :ns])
    o, lse = o.reshape(B, Hkv, G, n * c, D)[..., :T, :], lse.reshape(B, Hkv, G, n * c)[..., :T]
    if lens is not None:
        gone = (torch.arange(T, device=dev) >= lens[:, None])[:, None, None]
        o, lse = torch.where(gone[..., None], zero, o), lse.masked_fill(gone, -math.inf)
    return o, lse


def _swa(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    q5, k4, v4 = q.float().view(B, Hkv, Hq // Hkv, T, D), k.float(), v.float()
    if not s["train"]:
        o, lse = _swa_forward(q5, k4, v4, s["window"], s["sinks"], s["lens"])
        return o.reshape(q.shape).to(q.dtype), lse.reshape(B, Hq, T)
    with torch.enable_grad():
        q5, k4, v4 = (x.detach().requires_grad_() for x in (q5, k4, v4))
        o, _ = _swa_forward(q5, k4, v4, s["window"], s["sinks"], s["lens"])
        dq, dk, dv = torch.autograd.grad(o, (q5, k4, v4), s["dO"].float().view_as(o))
    return tuple(x.detach().reshape(y.shape).to(q.dtype) for x, y in ((o, q), (dq, q), (dk, k), (dv, v)))


def _attend(q, k, v, live):
    """One query per head against cached rows: o [B,Hq,D] and p [B,Hkv,G,C], in 32 bits."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    x = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), k.float().transpose(-1, -2)) / math.sqrt(D)
    p, _ = _softmax(x.masked_fill(~live[:, :, None], -math.inf))
    return torch.matmul(p, v.float()).reshape(B, Hq, D), p


def _decode(s):
    ck, cv, pos, ns, W = s["cache_k"], s["cache_v"], s["pos"].long(), s["sinks"], s["window"]
    B, Hkv, C, D = ck.shape
    slot = torch.where(pos < ns, pos, ns + (pos - ns) % W)
    b = torch.arange(B, device=ck.device)
    ck[b, :, slot] = s["k"]
    cv[b, :, slot] = s["v"]
    live = torch.arange(C, device=ck.device) <= pos[:, None]               # a ring holds its last tokens from slot 0 up
    o, _ = _attend(s["q"], ck, cv, live[:, None].expand(B, Hkv, C))
    return o.to(ck.dtype), ck, cv


def _weight(s):
    q, k, lse = s["q"], s["k"], s["lse"]
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    x = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, T, D), k.float()[:, :, None].transpose(-1, -2)) / math.sqrt(D)
    t = torch.arange(T, device=q.device)
    see = t[None, :] <= t[:, None]
    if s["lens"] is not None:
        see = see & (t < s["lens"][:, None])[:, None, None, :, None]
    p = torch.exp(torch.where(see, x - lse.view(B, Hkv, Hq // Hkv, T, 1), torch.full_like(x, -math.inf)))
    return p.sum((2, 3))


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
    for cache, x in ((s["cache_k"], s["k"]), (s["cache_v"], s["v"])):
        cache[:, :, :m] = torch.where(has[..., None], torch.gather(x, 2, rows), cache[:, :, :m])
    return s["cache_k"], s["cache_v"], s["cache_w"], s["cache_pos"]


def _evict(s):
    ck, cv, cw, cp = s["cache_k"], s["cache_v"], s["cache_w"], s["cache_pos"]
    B, Hkv, C, D = ck.shape
    pos = s["pos"].view(B, 1, 1)
    # the slot: that which holds this position already, else an empty one, else the least
    # weight among those that are neither first nor recent; the lowest of equals
    safe = (cp < s["sinks"]) | (cp > pos - s["recent"])
    key = torch.where(safe, math.inf, cw)
    key = torch.where(cp < 0, -1.0, key)
    key = torch.where(cp == pos, -2.0, key)
    index = torch.arange(C, device=ck.device)
    slot = torch.where(key == key.amin(-1, keepdim=True), index, C).amin(-1)
    at = slot[..., None]
    ck.scatter_(2, at[..., None].expand(B, Hkv, 1, D), s["k"][:, :, None])
    cv.scatter_(2, at[..., None].expand(B, Hkv, 1, D), s["v"][:, :, None])
    cp.scatter_(2, at, pos.expand(B, Hkv, 1))
    cw.scatter_(2, at, 0.0)
    o, p = _attend(s["q"], ck, cv, cp >= 0)
    cw += p.sum(2)
    return o.to(ck.dtype), slot.to(torch.int32), ck, cv, cw, cp


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(T, window, sinks):
    """Visible (token, key) pairs of one sequence and head."""
    n = 0
    w = min(window, T)
    n += w * (w + 1) // 2 + (T - w) * w
    for j in range(min(sinks, T)):           # a sink behind the window: tokens j + window .. T - 1
        n += max(0, T - window - j)
    return n


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    Hq = case.get("Hq", 0)
    share = 0.75 if case["ragged"] else 1.0
    if case["op"] == "swa":
        T = case["T"]
        pairs = B * Hq * _pairs(max(1, int(T * share)), case["window"], case["sinks"])
        qs, ks = B * Hq * T * D * es, B * Hkv * T * D * es
        if case["train"]:                    # q, dO in, o, dq out; k, v in, dk, dv out
            return {"bytes": 4 * qs + 4 * ks, "flops": 14 * D * pairs}
        return {"bytes": 2 * qs + 2 * ks + B * Hq * T * 4, "flops": 4 * D * pairs}
    if case["op"] == "weight":
        T = case["T"]
        pairs = B * Hq * _pairs(max(1, int(T * share)), T, 0)
        return {"bytes": (B * Hq + B * Hkv) * T * D * es + (B * Hq + B * Hkv) * T * 4, "flops": 2 * D * pairs}
    if case["op"] == "keep":
        rows = B * Hkv * min(case["C"], case["T"])
        return {"bytes": B * Hkv * case["T"] * 4 * share + rows * (4 * D * es + 12), "flops": B * Hkv * case["T"]}
    C = case["window"] + case["sinks"] if case["op"] == "decode" else case["C"]
    rows = B * Hkv * C
    return {"bytes": rows * 2 * D * es + (12 * rows if case["op"] == "evict" else 0) + (2 * Hq + 4 * Hkv) * B * D * es,
            "flops": 4 * D * B * Hq * C}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"swa": _exact_swa, "decode": _exact_decode, "weight": _exact_weight, "keep": _exact_keep,
            "evict": _exact_evict}[case["op"]](s)


def _rows(T, r0, r1, window, sinks, n, dev):
    """Which keys the tokens r0 .. r1 - 1 of a sequence of n tokens see."""
    t, u = torch.arange(r0, r1, device=dev)[:, None], torch.arange(T, device=dev)[None]
    return (u <= t) & ((t - u < window) | (u < sinks)) & (t < n)


def _exact_swa(s):
    q, k, v, dev = s["q"], s["k"], s["v"], s["q"].device
    B, Hq, T, D = q.shape
    G = Hq // k.shape[1]
    n = [T] * B if s["lens"] is None else s["lens"].tolist()
    f64 = dict(dtype=torch.float64, device=dev)
    o, lse = torch.zeros(q.shape, **f64), torch.full((B, Hq, T), -math.inf, **f64)
    dq, dk, dv = torch.zeros(q.shape, **f64), torch.zeros(k.shape, **f64), torch.zeros(k.shape, **f64)
    for b in range(B):
        for h in range(Hq):
            kk, vv = k[b, h // G].double(), v[b, h // G].double()
            for r in range(0, n[b], 4096):
                e = min(n[b], r + 4096)
                see = _rows(T, r, e, s["window"], s["sinks"], n[b], dev)
                qq = q[b, h, r:e].double()
                x = (qq @ kk.T * D ** -0.5).masked_fill(~see, -math.inf)
                z = torch.logsumexp(x, -1, keepdim=True)
                p = torch.exp(x - z)
                o[b, h, r:e], lse[b, h, r:e] = p @ vv, z[:, 0]
                if s["train"]:
                    g = s["dO"][b, h, r:e].double()
                    dp = g @ vv.T
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
                    dq[b, h, r:e] = ds @ kk
                    dk[b, h // G] += ds.T @ qq
                    dv[b, h // G] += p.T @ g
    return (o, dq, dk, dv) if s["train"] else (o, lse)


def _exact_rows(q, k, v, live):
    """Attention of one query over the live rows of its cache, with the weights."""
    x = (k.double() @ q.double()) * q.shape[-1] ** -0.5
    p = torch.softmax(x.masked_fill(~live, -math.inf), 0)
    return p @ v.double(), p


def _exact_decode(s):
    ck, cv = s["cache_k"].clone(), s["cache_v"].clone()
    B, Hkv, C, D = ck.shape
    G = s["q"].shape[1] // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=ck.device)
    for b, p in enumerate(s["pos"].tolist()):
        at = p if p < s["sinks"] else s["sinks"] + (p - s["sinks"]) % s["window"]
        ck[b, :, at], cv[b, :, at] = s["k"][b], s["v"][b]
        m = min(p + 1, C)
        for h in range(s["q"].shape[1]):
            o[b, h], _ = _exact_rows(s["q"][b, h], ck[b, h // G, :m], cv[b, h // G, :m],
                                     torch.ones(m, dtype=torch.bool, device=ck.device))
    return o, ck.double(), cv.double()


def _exact_weight(s):
    q, k, dev = s["q"], s["k"], s["q"].device
    B, Hq, T, D = q.shape
    G = Hq // k.shape[1]
    n = [T] * B if s["lens"] is None else s["lens"].tolist()
    a = torch.zeros(B, k.shape[1], T, dtype=torch.float64, device=dev)
    for b in range(B):
        for h in range(Hq):
            x = (q[b, h, :n[b]].double() @ k[b, h // G].double().T) * D ** -0.5
            x = x.masked_fill(~_rows(T, 0, n[b], T, 0, n[b], dev), -math.inf)
            a[b, h // G] += torch.exp(x - s["lse"][b, h, :n[b], None].double()).sum(0)
    return a


def _exact_keep(s):
    B, Hkv, T = s["weights"].shape
    C = s["C"]
    out = [s[x].double().clone() for x in ("cache_k", "cache_v", "cache_w")]
    held = torch.full((B, Hkv, C), -1, dtype=torch.int32, device=out[0].device)
    out[2].zero_()
    for b in range(B):
        n = T if s["lens"] is None else int(s["lens"][b])
        safe = set(range(min(s["sinks"], n))) | set(range(max(0, n - s["recent"]), n))
        for h in range(Hkv):
            w = s["weights"][b, h].tolist()
            rest = sorted((t for t in range(n) if t not in safe), key=lambda t: (-w[t], t))
            at = torch.tensor(sorted(list(safe) + rest[:max(0, C - len(safe))]), device=out[0].device)
            m = len(at)
            out[0][b, h, :m], out[1][b, h, :m] = s["k"][b, h, at].double(), s["v"][b, h, at].double()
            out[2][b, h, :m], held[b, h, :m] = s["weights"][b, h, at].double(), at.to(torch.int32)
    return out[0], out[1], out[2], held


def _exact_evict(s):
    ck, cv, cp = s["cache_k"].clone(), s["cache_v"].clone(), s["cache_pos"].clone()
    cw = s["cache_w"].double()
    B, Hkv, C, D = ck.shape
    G = s["q"].shape[1] // Hkv
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=ck.device)
    slot = torch.zeros(B, Hkv, dtype=torch.int32, device=ck.device)
    for b, p in enumerate(s["pos"].tolist()):
        for h in range(Hkv):
            held, w = cp[b, h].tolist(), cw[b, h].tolist()
            if p in held:
                at = held.index(p)
            elif min(held) < 0:
                at = next(j for j in range(C) if held[j] < 0)
            else:
                at = min((j for j in range(C) if s["sinks"] <= held[j] <= p - s["recent"]), key=lambda j: (w[j], j))
            slot[b, h] = at
            ck[b, h, at], cv[b, h, at], cp[b, h, at], cw[b, h, at] = s["k"][b, h], s["v"][b, h], p, 0.0
            live = cp[b, h] >= 0
            for g in range(h * G, (h + 1) * G):
                o[b, g], pr = _exact_rows(s["q"][b, g], ck[b, h], cv[b, h], live)
                cw[b, h] += pr
    return o, slot, ck.double(), cv.double(), cw, cp
