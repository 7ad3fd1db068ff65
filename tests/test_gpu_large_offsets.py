"""Rows of the MXFP4 calls and of the backward pass at the far end of what they
take: a second launch of the row quantiser, operands of nearly 2 GiB, gradients'
rows past 4 GiB, and the full model size in both directions (needs an MI355X).

The far rows belong to an expert of their own, behind all others, so that what
they give is compared bit for bit with a call on those rows alone (every sum is
taken in the same order), and that call with the oracle elsewhere."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402
from test_gpu_backward import NAMES, _check, _inputs, _routing, _run  # noqa: E402
from test_gpu_w4a4 import _block, _matrix, _up  # noqa: E402

pytestmark = pytest.mark.gpu


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_rows_of_a_second_launch():
    """More rows than the 2^27 that one launch of the quantiser takes: rows at the border and behind it against the
    oracle, zeros everywhere else, and all of it back."""
    _need_gpu()
    R, K = (1 << 27) + 5, 32
    pick = torch.tensor([0, 1, 17, (1 << 27) - 17, (1 << 27) - 1, 1 << 27, (1 << 27) + 1, R - 1], device="cuda")
    a = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    a[pick] = (torch.randn((len(pick), K), device="cuda") * 3.0).bfloat16()
    codes = torch.full((R, K // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, R, 4), 0x5A, dtype=torch.uint8, device="cuda")
    binding.moe_quantize_rows_mxfp4(a, codes=codes, scales=scales)
    c, s = orc.mxfp4_quantize_rows(host_f64(a[pick]))
    assert (codes[pick].cpu().numpy() == c).all() and (scales[:, pick].cpu().numpy() == s).all()
    back = binding.moe_dequantize_rows_mxfp4(codes, scales)
    assert (host_f64(back[pick]) == orc.mxfp4_dequantize_rows(c, s)).all()
    codes[pick], scales[:, pick], back[pick] = 0, 0, 0
    assert not codes.any() and not scales.any() and not back.view(torch.int16).any()


@pytest.mark.parametrize("T,H,I", [(400000, 64, 2880),       # rows of d, dgu and w h past 2^32 bytes
                                   (372800, 2880, 64)])      # x and dy end just below 2^31 bytes
def test_gradients_of_far_rows(T, H, I):
    """All gradients of an expert whose tokens are the last, alone and behind two experts with all others."""
    _need_gpu()
    n, E, k = 100, 3, 2
    small, (_, w) = _inputs(n, E, H, I, 61), _routing(n, E, k, 62)
    ids = np.full((n, k), -1, np.int32)
    ids[:, 0] = 2
    part = [dev(v) for v in small] + [torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()]
    alone = binding.moe_backward(*part)
    _check(small, ids, w, alone)
    dy, x = (torch.randn((T, H), device="cuda").bfloat16() for _ in range(2))
    ids_all = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(T, 1)
    w_all = torch.full((T, k), 0.5, device="cuda")
    for whole, piece in ((dy, part[0]), (x, part[1]), (ids_all, part[7]), (w_all, part[8])):
        whole[T - n:] = piece
    got = binding.moe_backward(dy, x, *part[2:7], ids_all, w_all)
    assert (bf16_bits(got["dx"][T - n:]) == bf16_bits(alone["dx"])).all()
    for g in NAMES[1:]:
        assert (alone[g][2] != 0).any() and (bf16_bits(got[g][2]) == bf16_bits(alone[g][2])).all(), g


@pytest.mark.parametrize("path", ["gemv", "gemm"])
def test_products_of_far_rows(path):
    """Stage calls whose codes end just below 2^31 bytes: the last rows, alone and behind two experts."""
    _need_gpu()
    T, K, n, E = 1491308, 2880, 70, 3
    assert T * K < 1 << 32
    g = torch.Generator(device="cuda").manual_seed(63)
    xq = torch.randint(0, 256, (T, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sx = torch.randint(121, 124, (-(-K // 128), T, 4), generator=g, device="cuda", dtype=torch.uint8)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % 2).unsqueeze(1)
    ids[T - n:] = 2
    few = torch.full((n, 1), 2, dtype=torch.int32, device="cuda")
    q, s = (_up(a) for a in _matrix(E, K, 64, 64))
    bias = dev(_inputs(1, E, 8, 32, 65)[4])                   # [E][64]
    cnt, off, rows, _ = binding.moe_permute(ids, E)
    cnt1, off1, rows1, _ = binding.moe_permute(few, E)
    tail = xq[T - n:].contiguous(), sx[:, T - n:].contiguous()
    hq, sh = binding.moe_gate_up_w4a4(xq, sx, q, s, bias, cnt, off, rows, k=1, path=path)
    hq1, sh1 = binding.moe_gate_up_w4a4(*tail, q, s, bias, cnt1, off1, rows1, k=1, path=path)
    assert (hq[T - n:] == hq1).all() and (sh[:, T - n:, :1] == sh1[:, :, :1]).all() and hq1.any()
    o = binding.moe_down_w4a4(xq, sx, q, s, bias, cnt, off, T, 1, path=path)
    o1 = binding.moe_down_w4a4(*tail, q, s, bias, cnt1, off1, n, 1, path=path)
    assert (o[T - n:] == o1).all() and o1.any()
    h, W = orc.mxfp4_dequantize_rows(tail[0].cpu().numpy(), tail[1].cpu().numpy()), orc.mxfp4_dequantize(
        q[2].cpu().numpy(), s[2].cpu().numpy()).T
    b = host_f64(bias[2])
    # a matrix instruction is within 2^-23 of its terms' magnitudes; K / 64 of them, the join of eight parts, the bias
    tol = (K / 64 + 9) * 2.0 ** -23 * (np.abs(h) @ np.abs(W) + np.abs(b))
    assert (np.abs(o1.cpu().numpy() - (h @ W + b)) <= tol).all()


# ------------------------------------------------------------------------------------------------ the model's own size
@pytest.mark.parametrize("T,E,k,H,I", [(150, 2, 1, 2880, 2880), (40, 3, 2, 2880, 2880), (2000, 40, 4, 264, 200),
                                       (300, 256, 8, 72, 40)])
def test_gradients_at_full_size(T, E, k, H, I):
    """Both dimensions of the model at once, and many experts with many tokens or many picks."""
    _need_gpu()
    inputs, (ids, w) = _inputs(T, E, H, I, 66), _routing(T, E, k, 67)
    _check(inputs, ids, w, _run(inputs, ids, w))


@pytest.mark.parametrize("path", ["auto", "gemv", "gemm"])
@pytest.mark.parametrize("T,E,k", [(60, 4, 2), (300, 4, 2)])
def test_w4a4_block_at_full_size(T, E, k, path):
    _need_gpu()
    args = _block(T, E, k, 2880, 2880, 68)
    ref = orc.moe_forward_w4a4(*args, k)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    y = binding.moe_forward_w4a4(*[_up(a) for a in args], k=k, topk_ids=ids, topk_w=w, path=path)
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"])
    assert_y_close(host_f64(y), ref["y"])
