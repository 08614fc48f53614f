"""Caches in codes of 4 and 8 bits: the definition's own properties, the refusals of the entry points on the
host and of the binding (CPU only)."""
import ctypes
import math

import pytest
import torch

from chunk_gated_delta_amd import carve
from tests import mx_ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, ODD = 0x100000, 0x100008  # 16-byte aligned and not; never dereferenced on a rejected call


@pytest.fixture(scope="module")
def lib():
    return carve.load_library()


def swa(B=2, Hq=4, Hkv=2, T=64, D=128, window=16, sinks=2, scale=0.1, dtype=carve.CARVE_BF16):
    return carve.carve_swa_shape(B, Hq, Hkv, T, D, window, sinks, scale, dtype)


def budget(B=2, Hq=4, Hkv=2, T=1, D=128, C=32, sinks=2, recent=4, scale=0.1, dtype=carve.CARVE_BF16):
    return carve.carve_budget_shape(B, Hq, Hkv, T, D, C, sinks, recent, scale, dtype)


def rows(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, bits=4):
    return carve.carve_mx_rows(k_codes, k_scales, v_codes, v_scales, bits)


# ------------------------------------------------------------------ the definition
@pytest.mark.parametrize("bits", [4, 8])
def test_definition(bits):
    """No value is off by more than half a step of its place on the grid (8 bits: the last step 32, 4 bits: 2),
    writing again changes nothing, and the worked codes are as the header says."""
    gen = torch.Generator().manual_seed(bits)
    x = torch.randn(300, 128, generator=gen).double() * torch.exp(3 * torch.randn(300, 1, generator=gen)).double()
    value, code, scale = mx_ref.written(x, bits)
    assert torch.equal(mx_ref.values(code, scale), value)
    again, code2, scale2 = mx_ref.written(value, bits)
    assert torch.equal(again, value) and torch.equal(code2, code) and torch.equal(scale2, scale)
    assert torch.equal(value.bfloat16().double(), value)
    up = 2.0 ** (scale.double() - 127).repeat_interleave(32, -1)
    size = value.abs() / up
    least = 1.0 if bits == 4 else 2.0 ** -6
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=least)))) * (0.5 if bits == 4 else 0.125)
    assert ((x - value).abs() <= step * up / 2).all()
    # the scale is the least that holds the block: half of it would not
    big = x.abs().unflatten(-1, (-1, 32)).amax(-1) / 2.0 ** (scale.double() - 127)
    most = mx_ref.MOST[bits]
    assert (big <= most).all() and (big > most / 2).all()


def test_worked_codes():
    x = torch.zeros(1, 32).double()
    x[0, :9] = torch.tensor([6.0, -0.25, 0.75, 2.5, -3.5, 5.0, -0.0, 1.25, 7.0])
    value, code, scale = mx_ref.written(x, 4)
    assert scale.tolist() == [[127]]
    assert value[0, :9].tolist() == [6.0, -0.0, 1.0, 2.0, -4.0, 4.0, -0.0, 1.0, 6.0]      # ties to the even code
    assert code[0, :5].tolist() == [7 | 8 << 4, 2 | 4 << 4, 14 | 6 << 4, 8 | 2 << 4, 7]
    x[0, 8] = 7.0 + 2 ** -20
    assert mx_ref.written(x, 4)[2].tolist() == [[128]]
    value, code, scale = mx_ref.written(torch.tensor([[464.0, -1.0625, 2 ** -10, 3 * 2 ** -10] + [0.0] * 28]), 8)
    assert scale.tolist() == [[127]] and value[0, :4].tolist() == [448.0, -1.0, 0.0, 2 ** -8]
    assert code[0, :5].tolist() == [126, 128 + 56, 0, 2, 0]
    for bad in (math.nan, math.inf, -math.inf):
        x[0, 3] = bad
        value, code, scale = mx_ref.written(x, 4)
        assert scale.tolist() == [[255]] and not code.any() and torch.isnan(value).all()


# ------------------------------------------------------------------ refusals of the entry points
CALLS = {   # shape, tokens, arguments before the cache, after it; "t" 16-byte aligned, "f" 4-byte, "?" optional
    "carve_swa_fill_mx": (swa, 64, "tt?f", "", False),
    "carve_swa_decode_mx": (swa, 1, "ttt", "ft", True),
    "carve_budget_keep_mx": (budget, 64, "ttf?f", "ff", False),
    "carve_budget_decode_mx": (budget, 1, "ttt", "fff" + "tf", True),
}


def call(lib, name, s, cache, change=None, ws=FAKE, ws_bytes=1 << 40):
    _, _, before, after, has_ws = CALLS[name]
    before, after = [FAKE] * len(before.replace("?", "")), [FAKE] * len(after)
    if change is not None:
        i, to = change
        if i < len(before):
            before[i] = to
        else:
            after[i - len(before)] = to
    tail = [ws, ws_bytes] if has_ws else []
    return getattr(lib, name)(None if s is None else ctypes.byref(s), *before,
                              None if cache is None else ctypes.byref(cache), *after, *tail, None)


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(lib, name):
    make, T, before, after, has_ws = CALLS[name]
    good = make(T=T)
    assert call(lib, name, None, rows()) == INVALID
    assert call(lib, name, good, None) == INVALID
    for kw, want in ((dict(B=-1), INVALID), (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(scale=math.nan), INVALID),
                     (dict(dtype=7), INVALID), (dict(D=96), UNSUPPORTED), (dict(B=70000), UNSUPPORTED),
                     (dict(sinks=-1), INVALID)):
        assert call(lib, name, make(**{"T": T, **kw}), rows()) == want, kw
    if make is swa:
        assert call(lib, name, swa(T=T, window=0), rows()) == INVALID
    else:
        assert call(lib, name, budget(T=T, C=5, sinks=2, recent=4), rows()) == INVALID
    if T == 1:
        assert call(lib, name, make(T=2), rows()) == INVALID
        assert call(lib, name, make(T=1, Hq=130), rows()) == UNSUPPORTED
    for bits in (0, 2, 16, -4):
        assert call(lib, name, good, rows(bits=bits)) == UNSUPPORTED
    for part in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert call(lib, name, good, rows(**{part: None})) == INVALID
    assert call(lib, name, good, rows(v_codes=ODD)) == INVALID
    assert call(lib, name, good, rows(k_scales=FAKE + 2)) == INVALID
    spec = (before + after).replace("?", "")
    optional = before.index("?") if "?" in before else None
    for i, kind in enumerate(spec):
        if i != optional:
            assert call(lib, name, good, rows(), (i, None)) == INVALID, i
        assert call(lib, name, good, rows(), (i, ODD if kind == "t" else FAKE + 2)) == INVALID, i


def test_empty_calls_do_nothing(lib):
    for name, (make, T, _, _, _) in CALLS.items():
        for kw in (dict(B=0), dict(Hq=0, Hkv=0)):
            assert call(lib, name, make(**{"T": T, **kw}), rows()) == OK
    assert call(lib, "carve_swa_fill_mx", swa(T=0), rows()) == OK
    for fn in (lib.carve_mx_quant, lib.carve_mx_dequant):
        assert fn(0, carve.CARVE_F32, 4, None, None, None, None) == OK


def test_row_refusals(lib):
    for fn in (lib.carve_mx_quant, lib.carve_mx_dequant):
        assert fn(33, carve.CARVE_F32, 4, FAKE, FAKE, FAKE, None) == INVALID
        assert fn(32, 5, 4, FAKE, FAKE, FAKE, None) == INVALID
        assert fn(32, carve.CARVE_F32, 3, FAKE, FAKE, FAKE, None) == UNSUPPORTED
        for i in range(3):
            ptrs = [FAKE] * 3
            ptrs[i] = None
            assert fn(32, carve.CARVE_F32, 4, *ptrs, None) == INVALID
    assert lib.carve_mx_quant(32, carve.CARVE_F32, 4, ODD, FAKE, FAKE, None) == INVALID
    assert lib.carve_mx_dequant(32, carve.CARVE_F32, 4, ODD, FAKE, FAKE, None) == INVALID


def test_workspaces(lib):
    """A long window of one sequence is cut into ranges and needs a workspace; a small one does not.  What the size
    function asks for less one byte is refused."""
    for size, name, s in ((lib.carve_swa_decode_mx_workspace_size, "carve_swa_decode_mx", swa(B=1, T=1, window=200000)),
                          (lib.carve_budget_decode_mx_workspace_size, "carve_budget_decode_mx", budget(B=1, C=200000))):
        for bits in (4, 8):
            need = size(ctypes.byref(s), bits)
            assert need > 0
            assert call(lib, name, s, rows(bits=bits), ws=FAKE, ws_bytes=need - 1) == WORKSPACE
            assert call(lib, name, s, rows(bits=bits), ws=None) == WORKSPACE
        assert size(ctypes.byref(s), 5) == 0
    assert lib.carve_swa_decode_mx_workspace_size(ctypes.byref(swa(B=1, T=1, window=64)), 4) == 0
    assert lib.carve_swa_decode_mx_workspace_size(ctypes.byref(swa(T=2)), 4) == 0


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        carve.mx_quant(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        carve.mx_dequant(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8))
    for codes, scales in (((2, 33), (2, 2)), ((2, 32), (3, 2)), ((2, 16), (2, 2)), ((2, 32), (2, 0)), ((), ())):
        with pytest.raises(ValueError, match="are not rows"):
            carve.mx_dequant(torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8))
    with pytest.raises(ValueError, match="4 or 8"):
        carve.swa_cache_mx(1, 1, 64, 8, bits=6, device="cpu")
    with pytest.raises(ValueError, match="past 32 bits"):
        carve.swa_decode_mx(x, x, x, None, None, window=1 << 40)


def test_cache_shapes():
    for bits in (4, 8):
        ring = carve.swa_cache_mx(2, 3, 128, 20, sinks=4, bits=bits, device="cpu")
        assert [tuple(x.shape) for x in ring] == [(2, 3, 24, 16 * bits), (2, 3, 24, 4)] * 2
        kept = carve.budget_cache_mx(2, 3, 64, 10, bits=bits, device="cpu")
        assert [tuple(x.shape) for x in kept] == [(2, 3, 10, 8 * bits), (2, 3, 10, 2)] * 2 + [(2, 3, 10)] * 2
        assert (kept[5] == -1).all()
