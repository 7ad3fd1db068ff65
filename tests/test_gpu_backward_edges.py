"""Calls of the block's backward pass at the edges of what it takes, beside
test_gpu_backward.py, whose inputs and bounds they use (needs an MI355X)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding  # noqa: E402
from checks import bf16_bits, dev  # noqa: E402
from test_gpu_backward import NAMES, _check, _inputs, _need_gpu, _routing, _run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
def test_weight_of_a_skipped_slot(fill):
    """Slots of no expert in the middle of a row, with anything as their weight: the same bits as with 0."""
    _need_gpu()
    T, E, k, H, I = 40, 5, 3, 136, 72
    inputs, (ids, w) = _inputs(T, E, H, I, 41), _routing(T, E, k, 42)
    ids[3, 0], ids[9, 1], ids[17, 2], ids[20:22] = -1, E, 2 ** 31 - 1, -2 ** 31
    skipped = (ids < 0) | (ids >= E)
    w = np.where(skipped, 0.0, w).astype(np.float32)
    want = _run(inputs, ids, w)
    _check(inputs, ids, w, want)
    got = _run(inputs, ids, np.where(skipped, np.float32(fill), w))
    for n in NAMES:
        assert (bf16_bits(got[n]) == bf16_bits(want[n])).all(), n
