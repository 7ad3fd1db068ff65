"""Edges of the block's backward pass that need no GPU: the oracle's reading of
skipped slots, and refusals of the C ABI (nothing here reaches a launch)."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d
import oracle.moe_oracle as orc


@pytest.mark.parametrize("fill", [np.nan, np.inf, -1.0])
def test_oracle_skips_the_weight_of_a_skipped_slot(fill):
    T, E, k, H, I = 6, 3, 2, 16, 8

    def n(i, std, *s):
        return d.normal_bf16(s, std, 51, i, *s)
    a = (n(1, 0.1, T, H), n(2, 1.0, T, H), n(3, 0.1, E, H), n(4, 0.1, E, H * 2 * I).reshape(E, H, 2 * I), n(5, 0.1, E, 2 * I),
         n(6, 0.1, E, I * H).reshape(E, I, H), n(7, 0.1, E, H))
    rng = np.random.default_rng(1)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[1, 0], ids[4] = -1, E
    w = np.full((T, k), 0.5, np.float32)
    skipped = (ids < 0) | (ids >= E)
    want = orc.moe_backward(*a, ids, np.where(skipped, np.float32(0), w))
    got = orc.moe_backward(*a, ids, np.where(skipped, np.float32(fill), w))
    assert all((got[v] == want[v]).all() for v in want) and np.abs(want["dx"]).max() > 0
    assert (want["dx"][4] == 0).all()


# ------------------------------------------------------------------------------------------------ the C ABI
BASE = 1 << 36     # addresses that are never read, 64 GiB apart
NAMES = ("dy", "x", "Wr", "Wgu", "bgu", "Wd", "bd", "topk_ids", "topk_w", "dx", "dWr", "dbr", "dWgu", "dbgu", "dWd", "dbd")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.library()


def _call(lib, T=0, H=64, E=4, k=2, I=32, ws_bytes=0, **add):
    """moe_backward on addresses 64 GiB apart, each moved by add[name] bytes."""
    p = [ctypes.c_void_p(BASE * (i + 1) + add.get(n, 0)) for i, n in enumerate(NAMES)]
    return lib.moe_backward(*p[:9], T, H, E, k, I, *p[9:], ctypes.c_void_p(BASE * 20), ws_bytes, None)


@pytest.mark.parametrize("name,step", [(n, 4 if n in ("bgu", "bd", "dbgu", "dbd", "topk_ids", "topk_w") else
                                        2 if n == "dbr" else 16) for n in NAMES])
def test_alignment(lib, name, step):
    """Biases and their gradients from any word on, as the forward call takes them; everything else as it says."""
    assert _call(lib, **{name: step}) == OK, lib.moe_last_error()
    assert _call(lib, **{name: step // 2}) == INVALID
    assert f"{name} is not {step}-byte aligned" in lib.moe_last_error().decode()


def test_sizes_that_no_launch_holds(lib):
    """Refused before anything is enqueued: rows that 31-bit offsets do not reach, and launches of 2^32 threads (the
    workspace is too small throughout, which is looked at last)."""
    for T, H, k, I in ((1 << 24, 64, 1, 64), (1 << 27, 8, 1, 8), (1 << 17, 8192, 4, 8)):
        assert _call(lib, T=T, H=H, k=k, I=I) == UNSUPPORTED and b"2 GiB" in lib.moe_last_error(), (T, H, k, I)
    for T, k, I in ((1 << 26, 1, 8), ((1 << 26) + 12345, 2, 8), ((1 << 27) - 1, 4, 96), (1 << 25, 4, 2048)):
        assert _call(lib, T=T, H=8, k=k, I=I) == UNSUPPORTED, (T, k, I, lib.moe_last_error())
        assert b"2^32 threads" in lib.moe_last_error()
    for T, H, k, I in ((1 << 25, 8, 4, 8), ((1 << 26) - (1 << 22), 8, 1, 8), ((1 << 25), 8, 4, 1024), (1 << 18, 2880, 4, 2880)):
        assert _call(lib, T=T, H=H, k=k, I=I) == WORKSPACE, (T, H, k, I, lib.moe_last_error())
