"""Where the calls with MXFP4 on both sides stop taking rows, as the header states
it (CPU only: nothing here reaches a launch)."""
from __future__ import annotations

import ctypes
import os

import pytest

pytest.importorskip("torch")

from moe_layer_route_amd import binding  # noqa: E402

UNSUPPORTED, WORKSPACE = 2, 3
BASE = 1 << 36     # addresses that are never read, 64 GiB apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.library()


def _forward(lib, name, T, H, k, I, E=8):
    p = [ctypes.c_void_p(BASE * (i + 1)) for i in range(11)]
    more = {"moe_forward_w4a4": ((), ()), "moe_forward_padded_w4a4": ((None,), (None,)), "moe_forward_ep_w4a4": ((0, E), ())}
    before, between = more[name]
    return getattr(lib, name)(*p[:9], T, H, E, k, I, *before, p[9], None, None, *between, p[10], 256, 0, None)


@pytest.mark.parametrize("name", ["moe_forward_w4a4", "moe_forward_padded_w4a4", "moe_forward_ep_w4a4"])
def test_bounds_of_x_and_h(lib, name):
    """x below 4 GiB but for 64 bytes, h of fewer than 2^32 values; a workspace too small is looked at behind them."""
    for T, H, k, I, what in ((1 << 26, 32, 1, 32, b"x of"), ((1 << 26) - 1, 32, 1, 32, b"x of"),
                             (1 << 25, 32, 4, 32, b"h of"), (1 << 20, 64, 4, 1024, b"h of")):
        assert _forward(lib, name, T, H, k, I) == UNSUPPORTED and what in lib.moe_last_error(), (T, H, k, I)
    for T, H, k, I in (((1 << 26) - 2, 32, 1, 32), ((1 << 25) - 1, 32, 4, 32), ((1 << 20) - 1, 64, 4, 1024)):
        assert _forward(lib, name, T, H, k, I) == WORKSPACE, (T, H, k, I, lib.moe_last_error())
