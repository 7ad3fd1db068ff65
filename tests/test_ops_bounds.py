"""Sizes just inside the limits of the int4 and norm calls get past every size
check (a missing workspace ends them there), and outputs that would take the
place of the residual stream are refused (CPU only: nothing is launched)."""
import ctypes
import os

import pytest
import torch

from moe_layer_route_amd import binding

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.library()


def _p(i):
    return ctypes.c_void_p((1 << 34) * (i + 1))     # addresses that are never read, 16 GiB apart


# T, k, H, I: the last size that is taken and the first that is not, by x and by h (2^32 - 64 bytes)
EDGES = [((2 ** 32 - 65) // (2 * 2880), 1, 2880, 32), (2 ** 20 - 1, 2, 32, 1024), ((2 ** 32 - 65) // (2 * 32), 1, 32, 32)]


@pytest.mark.parametrize("T,k,H,I", EDGES)
@pytest.mark.parametrize("call", ["forward", "padded", "rank", "norm"])
def test_largest_sizes(lib, call, T, k, H, I):
    p = [_p(i) for i in range(20)]
    p[5] = p[9] = None                              # no zero points

    def run(T):
        int4 = (*p[:11], T, H, 8, k, I, 32)
        end = (None, None, None, 0, 0, None)        # ids, weights, workspace, its bytes, path, stream
        if call == "forward":
            return lib.moe_forward_int4_ex(*int4, p[11], *end)
        if call == "padded":
            return lib.moe_forward_padded_int4(*int4, None, p[11], None, None, None, None, 0, 0, None)
        if call == "rank":
            return lib.moe_forward_ep_int4(*int4, 2, 3, p[11], *end)
        return lib.moe_forward_norm_fp8(p[0], p[1], p[2], 1e-5, *p[3:5], *p[10:16], T, H, 8, k, I, p[17], p[18], *end)

    assert run(T) == WORKSPACE, lib.moe_last_error()
    assert run(T + 1) == UNSUPPORTED, lib.moe_last_error()


# ---------------------------------------------------------------------------
# without a residual x is the residual stream: nothing may take its place
# ---------------------------------------------------------------------------
def _forward_norm(lib, residual, residual_out, y):
    p = [_p(i) for i in range(20)]
    return lib.moe_forward_norm_fp8(p[0], residual, p[2], 1e-5, *p[3:11], 4, 64, 8, 2, 32, residual_out, y, None, None, None,
                                    0, 0, None)


def test_block_output_does_not_replace_the_stream(lib):
    x = _p(0).value
    for y in (x, x + 16, x + 4 * 64 * 2 - 16, x - 4 * 64 * 2 + 16):
        assert _forward_norm(lib, None, None, ctypes.c_void_p(y)) == INVALID
        assert b"y overlaps x" in lib.moe_last_error()
    assert _forward_norm(lib, None, None, ctypes.c_void_p(x + 4 * 64 * 2)) == WORKSPACE
    # with a residual the stream is in residual_out, and x may be written over
    assert _forward_norm(lib, _p(1), _p(12), _p(0)) == WORKSPACE
    assert _forward_norm(lib, _p(1), _p(12), _p(1)) == WORKSPACE
    assert _forward_norm(lib, _p(1), _p(0), _p(1)) == WORKSPACE


def test_fp8_norm_does_not_replace_the_stream_it_returns():
    x, gamma = torch.zeros((5, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    buf = torch.zeros((9, 64), dtype=torch.bfloat16)
    for rows, y in ((x, x), (buf[:5], buf[2:7]), (buf[2:7], buf[:5])):
        with pytest.raises(binding.MoEError, match="y overlaps x"):
            binding.moe_add_rmsnorm_fp8(rows, gamma, y=y)
    for rows, kw in ((x, {}), (x, dict(y=x, residual=x.clone())), (buf[:4], dict(y=buf[4:8]))):   # these end at the device check
        with pytest.raises(binding.MoEError, match="must be on the GPU"):
            binding.moe_add_rmsnorm_fp8(rows, gamma, **kw)


def test_eps_is_any_finite_value_above_zero(lib):
    x, gamma, y = _p(0), _p(1), _p(2)
    for eps, want in ((3.4028234663852886e38, 0), (1e-45, 0), (float("inf"), INVALID), (float("nan"), INVALID), (0.0, INVALID)):
        assert lib.moe_add_rmsnorm(x, None, gamma, 0, 64, eps, None, y, None) == want, eps
