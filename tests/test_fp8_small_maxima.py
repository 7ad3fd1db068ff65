"""FP8 quantisation of rows and experts whose maximum is below 2^-119, where
448 / max is past float32's range: the codes are those of the row times 2^64
(an exact scaling), so no finite input gives the NaN code."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402

LIFT = np.float32(2.0 ** 64)


def _small_rows():
    """float32 rows [R][48] with maxima from 2^-149 (the smallest float32) up to and past 2^-119, zeros of both signs in each."""
    rng = np.random.default_rng(71)
    base = rng.uniform(-1, 1, (10, 48))
    top = 2.0 ** np.array([-149, -148, -140, -133, -126, -121, -119.5, -119, -118.5, -110])
    base[:, 0] = 1.0
    rows = (base * top[:, None]).astype(np.float32)
    rows[:, 1], rows[:, 2] = 0.0, -0.0
    return rows


def test_oracle_codes_do_not_depend_on_a_power_of_two():
    rows = _small_rows()
    codes, s = orc.fp8_quantize_rows(rows)
    want, s_up = orc.fp8_quantize_rows(rows * LIFT)
    assert not (codes == 0x7F).any() and (codes == want).all()
    assert (s == rows.max(axis=1) / np.float32(448)).all() and np.isfinite(s_up).all()
    bits = d.f32_to_bf16_bits(np.ascontiguousarray(rows[:6].T)[None])        # one expert [1][48][6], all of it small
    c, _ = orc.fp8_quantize_weights(bits)
    up, _ = orc.fp8_quantize_weights(d.f32_to_bf16_bits((orc.widen(bits) * 2.0 ** 64).astype(np.float32)))
    assert np.abs(orc.widen(bits)).max() < 2.0 ** -119 and (c == up).all() and not (c == 0x7F).any()


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bf16_rows(K):
    """bf16 bits: rows of subnormals and of small normals, every third value zero, maxima on both sides of 2^-119."""
    rng = np.random.default_rng(72)
    a = np.zeros((8, K), np.uint16)
    a[0, 5] = 1                                               # the smallest subnormal alone
    a[1] = rng.integers(0, 128, K)                            # subnormals
    a[2] = rng.integers(0, 2, K)
    for r, e in ((3, -126), (4, -121), (5, -120), (6, -119), (7, -118)):
        a[r] = d.f32_to_bf16_bits((rng.uniform(-1.9, 1.9, K) * 2.0 ** e).astype(np.float32))
    a[:, ::3] = 0
    a[4, ::3] = 0x8000
    a[0, 5] = 1
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("K", [16, 48, 2880])
def test_quantize_rows(K):
    _need_gpu()
    a = _bf16_rows(K)
    codes, scales = binding.moe_quantize_rows_fp8(dev(a))
    want, s = orc.fp8_quantize_rows(orc.widen(a))
    got = codes.cpu().numpy()
    assert not (got == 0x7F).any() and (got == want).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.gpu
def test_quantize_weights():
    _need_gpu()
    W = np.stack([np.tile(_bf16_rows(48)[r], (16, 1)).T for r in range(8)])     # [8][48][16], one small expert a row
    codes, scales = binding.moe_quantize_fp8(dev(W))
    want, s = orc.fp8_quantize_weights(W)
    got = codes.cpu().numpy()
    assert not (got == 0x7F).any() and (got == want).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [48, 2880, 8208])
def test_norm_rows(H):
    """Small by gamma, and small by the rows themselves (eps is then what 1 / rms comes from)."""
    _need_gpu()
    rng = np.random.default_rng(73)
    for e in (-133, -127, -123, -121, -120, -119, -118):
        gamma = d.f32_to_bf16_bits((rng.uniform(0.5, 1.0, H) * 2.0 ** e).astype(np.float32))
        gamma[::5] = 0
        x = d.normal_bf16((3, H), 1.0, 74, H, 1, 1)
        x[:, ::7] = 0
        x[1, :] = 0
        x[1, 3] = 0x3F80
        y, codes, scales, _ = binding.moe_add_rmsnorm_fp8(dev(x), dev(gamma))
        _, _, v = orc.add_rmsnorm(x, None, gamma, 1e-5)
        want, s = orc.fp8_quantize_rows(v)
        got = codes.cpu().numpy()
        assert not (got == 0x7F).any(), e
        assert (got == want).all() and (scales.cpu().numpy() == s).all(), e
    a = _bf16_rows(H) & 0x80FF                                                  # below 2^-125: the codes of v, about 316 a
    ones = d.f32_to_bf16_bits(np.ones(H, np.float32))
    _, codes, scales, _ = binding.moe_add_rmsnorm_fp8(dev(a), dev(ones))
    want, s = orc.fp8_quantize_rows(orc.add_rmsnorm(a, None, ones, 1e-5)[2])
    got = codes.cpu().numpy()
    assert not (got == 0x7F).any() and (got == want).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.gpu
@pytest.mark.parametrize("path", ["gemv", "gemm"])
def test_blocks_stay_finite(path):
    """A token of subnormals among ordinary ones: its output is the biases' share, not NaN."""
    _need_gpu()
    T, E, H, I, k = 5, 8, 64, 96, 2
    cfg = d.small_config(T=T, E=E, H=H, I=I, k=k)
    Wr, br = d.make_router(cfg, 75)
    w = (Wr, br, *d.make_experts_fp8(cfg, 75, threads=4))
    on = [dev(a) if a.dtype == np.uint16 else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in w]
    x = d.normal_bf16((T, H), 3.0, 76, 1, T, H)
    x[2] = np.arange(H) % 2                                                     # 0 and 2^-133 in turn
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    y = binding.moe_forward_fp8(dev(x), *on, k=k, topk_ids=ids, topk_w=tw, path=path)
    ref = orc.moe_forward_fp8(x, *w, k=k)
    assert_routing(ids.cpu().numpy(), tw.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"])
    gamma = d.f32_to_bf16_bits(np.ones(H, np.float32))
    y, r = binding.moe_forward_norm_fp8(dev(x), dev(gamma), *on, k=k, path=path)
    assert (bf16_bits(r) == x).all()
    assert_y_close(host_f64(y), orc.moe_forward_norm_fp8(x, None, gamma, 1e-5, *w, k=k)["y"])
