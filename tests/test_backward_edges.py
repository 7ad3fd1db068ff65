"""Edges of the block's backward pass that need no GPU: the oracle's reading of
skipped slots, and refusals of the C ABI (nothing here reaches a launch)."""
from __future__ import annotations

import numpy as np
import pytest

from moe_layer_route_amd import datagen as d
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
