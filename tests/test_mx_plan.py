"""Which decode steps on caches in codes are cut into ranges, as the workspace that they ask for shows (CPU)."""
import ctypes

import pytest

from chunk_gated_delta_amd import carve


def swa_bytes(units, C, bits=4, D=128, dtype=1):
    s = carve.carve_swa_shape(units, 4, 1, 1, D, C, 0, D ** -0.5, dtype)
    return carve.load_library().carve_swa_decode_mx_workspace_size(ctypes.byref(s), bits)


def budget_bytes(units, C, bits=4, D=128, dtype=1):
    s = carve.carve_budget_shape(units, 4, 1, 1, D, C, 0, 1, D ** -0.5, dtype)
    return carve.load_library().carve_budget_decode_mx_workspace_size(ctypes.byref(s), bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [0, 1])
def test_ranges_of_few_key_heads_only(bits, D, dtype):
    """Up to 64 key heads from 1,537 slots on, up to 128 from 3,001 (4,097 with weights); above, one workgroup at any length."""
    for units, most in ((1, 1536), (64, 1536), (65, 3000), (128, 3000)):
        assert swa_bytes(units, most, bits, D, dtype) == 0 and swa_bytes(units, most + 1, bits, D, dtype) > 0
    for units in (129, 192, 255, 256, 4000):
        assert all(swa_bytes(units, C, bits, D, dtype) == 0 for C in (1, 4097, 100000))
    for units, most in ((1, 1536), (64, 1536), (65, 4096), (128, 4096)):
        scores = units * 4 * ((most + 3) // 4 * 4) * 4 + 256
        assert budget_bytes(units, most, bits, D, dtype) in (0, scores)
        assert budget_bytes(units, most + 1, bits, D, dtype) > scores + units * 4 * 16 + 4 * units * D
    for units in (129, 192, 255, 256):
        assert budget_bytes(units, 100000, bits, D, dtype) == units * 4 * 100000 * 4 + 256


def test_kernels_have_names_of_their_own_in_summaries():
    """A summary tells these kernels from each other, and from the delta rule's decode step."""
    from chunk_gated_delta_amd.prof_summary import short_name
    for name in ("mx_decode_kernel", "mx_quant_kernel", "mx_dequant_kernel", "mx_fill_kernel", "decode_kernel", "cache_decode_bf16_kernel"):
        assert short_name(f"_ZN5carve{len(name)}{name}IDF16bLi4EEEvNS_9CacheArgsE") == name
