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


def _at_word(a):
    """The tensor's values from an address on that is 4 past a multiple of 16."""
    whole = torch.zeros(a.numel() + 8, dtype=a.dtype, device=a.device)
    at = next(i for i in range(8) if (whole.data_ptr() + 2 * i) % 16 == 4)
    part = whole[at:at + a.numel()].view(a.shape)
    part.copy_(a)
    return part


@pytest.mark.parametrize("E,k,H,I", [(5, 2, 136, 72), (3, 3, 8, 8), (2, 1, 1032, 520)])
def test_biases_at_any_word(E, k, H, I):
    """Biases and their gradients that begin at a word, as views into a flat buffer of parameters do."""
    _need_gpu()
    T = 45
    inputs, (ids, w) = _inputs(T, E, H, I, 43), _routing(T, E, k, 44)
    want = _run(inputs, ids, w)
    _check(inputs, ids, w, want)
    a = [dev(v) for v in inputs]
    a[4], a[6] = _at_word(a[4]), _at_word(a[6])
    g = {n: _at_word(torch.full_like(want[n], -1.0)) for n in ("dbgu", "dbd")}
    got = binding.moe_backward(*a, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), **g)
    assert got["dbgu"] is g["dbgu"] and got["dbd"].data_ptr() % 16 == 4
    for n in NAMES:
        assert (bf16_bits(got[n]) == bf16_bits(want[n])).all(), n
