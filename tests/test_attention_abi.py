"""The attention entry points refuse bad arguments on the host before any launch, answer their
size functions, and the binding refuses tensors that do not fit (CPU only)."""
import ctypes
import math

import pytest
import torch

from chunk_gated_delta_amd import carve

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, ODD = 0x100000, 0x100008  # 16-byte aligned and not; never dereferenced on a rejected call


@pytest.fixture(scope="module")
def lib():
    return carve.load_library()


def swa(B=2, Hq=4, Hkv=2, T=64, D=128, window=16, sinks=2, scale=0.1, dtype=carve.CARVE_BF16):
    return carve.carve_swa_shape(B, Hq, Hkv, T, D, window, sinks, scale, dtype)


def budget(B=2, Hq=4, Hkv=2, T=1, D=128, C=32, sinks=2, recent=4, scale=0.1, dtype=carve.CARVE_BF16):
    return carve.carve_budget_shape(B, Hq, Hkv, T, D, C, sinks, recent, scale, dtype)


# entry point: pointer arguments (16-byte aligned tensors "t", 4-byte ones "f", optional in lower
# case after "?"), whether it takes a workspace
SWA_CALLS = {
    "carve_swa_fwd": ("ttt?ft?f", False, 64),
    "carve_swa_bwd": ("ttt?ftfttt t".replace(" ", ""), True, 64),
    "carve_swa_fill": ("tt?ftt", False, 64),
    "carve_swa_decode": ("tttttft", True, 1),
    "carve_budget_weights": ("ttf?ff", True, 64),
}
BUDGET_CALLS = {
    "carve_budget_keep": ("ttf?fttff", False, 64),
    "carve_budget_decode": ("tttttffftf", True, 1),
}


def parse(spec):
    out, opt = [], False
    for c in spec:
        if c == "?":
            opt = True
        else:
            out.append((c, opt))
            opt = False
    return out


def call(lib, name, s, ptrs, ws=FAKE, ws_bytes=1 << 40):
    table = SWA_CALLS if name in SWA_CALLS else BUDGET_CALLS
    tail = [ws, ws_bytes] if table[name][1] else []
    return getattr(lib, name)(ctypes.byref(s) if s is not None else None, *ptrs, *tail, None)


@pytest.mark.parametrize("name", list(SWA_CALLS) + list(BUDGET_CALLS))
def test_refusals(lib, name):
    table, make = (SWA_CALLS, swa) if name in SWA_CALLS else (BUDGET_CALLS, budget)
    spec, has_ws, T = table[name]
    args = parse(spec)
    good = [FAKE] * len(args)
    assert call(lib, name, None, good) == INVALID
    for kw, want in ((dict(B=-1), INVALID), (dict(Hq=-4), INVALID), (dict(T=-1), INVALID), (dict(Hq=5), INVALID),
                     (dict(Hkv=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
                     (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(dtype=7), INVALID),
                     (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(B=70000), UNSUPPORTED),
                     (dict(sinks=-1), INVALID)):
        assert call(lib, name, make(**{"T": T, **kw}), good) == want, kw
    if make is swa:
        assert call(lib, name, swa(T=T, window=0), good) == INVALID
        assert call(lib, name, swa(T=T, window=1 << 30, sinks=1), good) == UNSUPPORTED
    else:
        assert call(lib, name, budget(T=T, recent=0), good) == INVALID
        assert call(lib, name, budget(T=T, C=0, sinks=0), good) == INVALID
        assert call(lib, name, budget(T=T, C=5, sinks=2, recent=4), good) == INVALID
    if T == 1:
        assert call(lib, name, make(T=2), good) == INVALID
        assert call(lib, name, make(T=1, Hq=130, Hkv=2), good) == UNSUPPORTED
    for i, (kind, opt) in enumerate(args):
        if not opt:
            assert call(lib, name, make(T=T), good[:i] + [None] + good[i + 1:]) == INVALID, i
        assert call(lib, name, make(T=T), good[:i] + [ODD if kind == "t" else FAKE + 2] + good[i + 1:]) == INVALID, i
    if has_ws:
        big = dict(T=T, **(dict(window=5000) if make is swa else dict(C=5000)))
        if name == "carve_budget_weights":
            big = dict(T=4096)
        need = getattr(lib, name + "_workspace_size")(ctypes.byref(make(**big)))
        assert need > 0
        assert call(lib, name, make(**big), good, ws_bytes=need - 1) == WORKSPACE
        assert call(lib, name, make(**big), good, ws=None) == WORKSPACE
    # nothing to do
    assert call(lib, name, make(T=T, B=0), good) == OK
    assert call(lib, name, make(T=T, Hq=0, Hkv=0), good) == OK


def test_sizes(lib):
    size = lambda name, s: getattr(lib, name + "_workspace_size")(ctypes.byref(s))  # noqa: E731
    # a batch that fills the chip needs no joined ranges
    assert size("carve_swa_decode", swa(B=256, Hq=16, Hkv=4, T=1, window=4096)) == 0
    assert size("carve_swa_decode", swa(T=2)) == 0
    assert size("carve_swa_bwd", swa(D=96)) == 0
    # scores of every slot and query head
    assert size("carve_budget_decode", budget(B=256, Hq=16, Hkv=4, C=100, recent=8)) >= 256 * 16 * 100 * 4
    # a small cache of few sequences needs none
    assert size("carve_budget_decode", budget(B=1, Hq=16, Hkv=4, C=1024, recent=8)) == 0
    # sinks behind the window cost partial sums only where tokens are behind the window
    near = size("carve_swa_bwd", swa(T=100, window=100, sinks=4))
    assert near == size("carve_swa_bwd", swa(T=100, window=100, sinks=0))
    assert size("carve_swa_bwd", swa(T=4096, window=100, sinks=4)) > size("carve_swa_bwd", swa(T=4096, window=100, sinks=0))
    # largest accepted head count and a long sequence: sizes past 32 bits
    assert size("carve_swa_bwd", swa(B=65535, Hq=1, Hkv=1, T=1 << 20, window=64, sinks=0)) > 1 << 37


def test_binding_refuses(lib):
    q, k, v = torch.zeros(2, 4, 8, 64), torch.zeros(2, 2, 8, 64), torch.zeros(2, 2, 8, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        carve.swa_fwd(q, k, v, window=4)
    with pytest.raises(ValueError, match="dimensions"):
        carve.swa_fwd(q[0], k, v, window=4)
    with pytest.raises(ValueError, match="contiguous"):
        carve.swa_fwd(q.transpose(1, 2), k, v, window=4)
    with pytest.raises(ValueError, match="dimensions"):
        carve.swa_decode(q, k, v, None, None, None, window=4)
    with pytest.raises(ValueError, match="32 bits"):
        carve.swa_fwd(q, k, v, window=(1 << 32) + 4)
    with pytest.raises(ValueError, match="32 bits"):
        carve.budget_keep(k, v, torch.zeros(2, 2, 8), 1 << 33)


def test_scores_of_small_caches_stay_near_where_one_workgroup_fits(lib):
    """A step of a cache kept by weight keeps its scores in LDS (no workspace) unless that would keep a
    second workgroup off a compute unit: at width 64 from 257 key heads on."""
    size = lambda **kw: lib.carve_budget_decode_workspace_size(ctypes.byref(budget(Hq=16, Hkv=4, C=512, **kw)))  # noqa: E731
    assert size(B=64, D=64) == 0 and size(B=64, D=128) == 0
    assert size(B=75, D=128) == 0
    assert size(B=75, D=64) >= 75 * 16 * 512 * 4 and size(B=65, D=64) > 0
