"""Strides whose offsets pass 63 bits are refused before anything is launched (CPU only)."""
import pytest

from test_cache_host import D, H, append, attend, gather, lib, rope  # noqa: F401

FAR = 1 << 40
N = 1 << 24
APART = (H * N * D, N * D, D)
#: 64 + 2^40 (2^24 - 1) elements of a head wrap to less than nothing in 64 bits
WRAPS = (0, 1 << 43, FAR)


@pytest.mark.parametrize("kw", [
    {"xs": (0, 0, FAR)}, {"xs": (1 << 43, 0, 0), "batch": N, "n": 1, "os_": (H * D, D, D)},
    {"os_": WRAPS, "heads": 2, "batch": 1}, {"os_": (0, 0, 1 << 43), "heads": 1, "batch": 1},
])
def test_rope(lib, kw):  # noqa: F811
    assert rope(lib, **{"n": N, "os_": APART, **kw}) == 1


ONE = {"heads": 1, "r_batch": 1}


@pytest.mark.parametrize("call,kw", [
    (append, {"r_x": (0, 0, FAR)}), (append, {"r_v": (0, 0, FAR)}),
    (append, {"r_out": WRAPS, "heads": 2, "r_batch": 1}),
    (gather, {"r_x": (0, 0, FAR), **ONE}), (gather, {"r_v": (0, 0, FAR), **ONE}),
    (attend, {"r_x": (0, 0, FAR)}), (attend, {"r_out": (0, 0, FAR), **ONE}),
])
def test_cache_calls(lib, call, kw):  # noqa: F811
    assert call(lib, {"r_n": N, "r_max_pages": 1 << 20, "r_x": APART, "r_v": APART, "r_out": APART, **kw}) == 1
