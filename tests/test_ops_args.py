"""Refusals of the norm's and the int4 calls, in the C ABI and in the binding
(CPU only: nothing here reaches a launch), and the oracle's int4 format
against a scalar reading of it."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.moe_oracle as orc
from moe_layer_route_amd import binding

OK, INVALID, WORKSPACE = 0, 1, 3
BASE = 1 << 32     # addresses that are never read, one 4 GiB stretch each


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.library()


def _p(i, add=0):
    return ctypes.c_void_p(BASE * (i + 1) + add)


def _norm(lib, T=4, H=64, eps=1e-5, x=_p(0), res=_p(1), gamma=_p(2), r=_p(3), y=_p(4)):
    return lib.moe_add_rmsnorm(x, res, gamma, T, H, eps, r, y, None)


def _norm8(lib, T=4, H=64, eps=1e-5, x=_p(0), res=_p(1), gamma=_p(2), r=_p(3), y=_p(4), codes=_p(5), scales=_p(6)):
    return lib.moe_add_rmsnorm_fp8(x, res, gamma, T, H, eps, r, y, codes, scales, None)


@pytest.mark.parametrize("kw,err", [
    (dict(T=-1), "T=-1"), (dict(T=1 << 31), "T="), (dict(H=0), "H=0"), (dict(H=60), "H=60"), (dict(H=16392), "H=16392"),
    (dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(x=None), "x is NULL"), (dict(gamma=None), "gamma is NULL"), (dict(y=None), "y is NULL"),
    (dict(res=None), "both"), (dict(r=None), "both"), (dict(x=_p(0, 8)), "x is not"), (dict(y=_p(4, 2)), "y is not"),
    (dict(y=_p(0, 16)), "y overlaps x"), (dict(y=_p(3)), "y overlaps residual_out"), (dict(r=_p(1, 64)), "overlaps residual"),
    (dict(y=_p(2)), "overlaps gamma"), (dict(r=_p(0), y=_p(0)), "y overlaps residual_out"),
])
def test_norm_refuses(lib, kw, err):
    assert _norm(lib, **kw) == INVALID
    assert err in lib.moe_last_error().decode(), lib.moe_last_error()


@pytest.mark.parametrize("kw,err", [
    (dict(H=72), "H=72"), (dict(codes=None), "codes is NULL"), (dict(scales=None), "scales is NULL"),
    (dict(codes=_p(5, 8)), "codes is not"), (dict(scales=_p(6, 2)), "scales is not"), (dict(codes=_p(0)), "codes overlaps x"),
    (dict(scales=_p(5, 16)), "scales overlaps codes"), (dict(y=_p(5)), "codes overlaps y"), (dict(eps=0.0), "eps"),
])
def test_norm_fp8_refuses(lib, kw, err):
    assert _norm8(lib, **kw) == INVALID
    assert err in lib.moe_last_error().decode(), lib.moe_last_error()


def test_norm_takes_no_tokens_and_buffers_in_place(lib):
    assert _norm(lib, T=0) == OK and _norm8(lib, T=0) == OK and lib.moe_last_error() == b""
    assert _norm8(lib, T=0, y=None, res=None, r=None) == OK
    assert _norm(lib, T=0, r=_p(1), y=_p(0)) == OK


def _fwd_norm(lib, T=4, H=64, E=8, k=2, I=64, eps=1e-5, r=_p(3), y=_p(4), ws=_p(20), ws_bytes=1 << 30, path=0, res=_p(1)):
    return lib.moe_forward_norm_fp8(_p(0), res, _p(2), eps, *[_p(10 + i) for i in range(8)], T, H, E, k, I, r, y, None,
                                    None, ws, ws_bytes, path, None)


@pytest.mark.parametrize("kw,err", [
    (dict(T=-1), "T=-1"), (dict(H=72), "H=72"), (dict(k=9), "k=9"), (dict(eps=0.0), "eps"), (dict(y=None), "y is NULL"),
    (dict(y=_p(3)), "y overlaps residual_out"), (dict(path=4), "path 4"), (dict(r=None), "both"), (dict(r=_p(0, 16)), "overlaps x"),
    (dict(I=24), "I=24")])
def test_forward_norm_refuses(lib, kw, err):
    assert _fwd_norm(lib, **kw) == INVALID
    assert err in lib.moe_last_error().decode(), lib.moe_last_error()


def test_forward_norm_workspace(lib):
    need = lib.moe_workspace_bytes_norm_fp8(4, 64, 8, 2, 64)
    assert need >= lib.moe_workspace_bytes_fp8(4, 64, 8, 2, 64) + 4 * 64 * 2 and need % 256 == 0
    assert _fwd_norm(lib, ws_bytes=need - 1) == WORKSPACE and _fwd_norm(lib, ws=None) == WORKSPACE
    assert _fwd_norm(lib, T=0, ws=None, ws_bytes=0) == OK
    assert lib.moe_workspace_bytes_norm_fp8(0, 64, 8, 2, 64) == 0 and lib.moe_workspace_bytes_norm_fp8(4, 64, 1, 2, 64) == 0


def test_forward_norm_refuses_what_its_kernels_cannot_address(lib):
    """Before the norm is enqueued."""
    UNSUPPORTED = 2
    assert _fwd_norm(lib, T=(1 << 31) // 64, r=_p(60), res=_p(50), y=_p(70), ws=_p(90), ws_bytes=1 << 60) == UNSUPPORTED
    assert b"x of" in lib.moe_last_error()
    assert _fwd_norm(lib, T=1 << 20, I=1024, ws_bytes=1 << 60) == UNSUPPORTED and b"h of" in lib.moe_last_error()


def _fwd4(lib, T=8, H=64, E=8, k=2, I=64, G=32, ptr=None, z=(None, None), ws=_p(20), ws_bytes=1 << 30, path=0):
    p = [_p(i) for i in range(12)]
    for i, v in (ptr or {}).items():
        p[i] = v
    p[5], p[9] = z
    return lib.moe_forward_int4_ex(*p[:11], T, H, E, k, I, G, p[11], None, None, ws, ws_bytes, path, None)


@pytest.mark.parametrize("kw,err", [
    (dict(G=16), "G=16"), (dict(G=0), "G=0"), (dict(G=256), "G=256"), (dict(H=48), "H=48"), (dict(I=40), "I=40"),
    (dict(E=257), "E=257"), (dict(k=9), "k=9"), (dict(path=3), "path 3"), (dict(T=-2), "T=-2"),
    (dict(ptr={0: None}), "x is NULL"), (dict(ptr={3: None}), "Wgu_q is NULL"), (dict(ptr={4: _p(4, 8)}), "Wgu_s is not"),
    (dict(ptr={7: _p(7, 4)}), "Wd_q is not"), (dict(ptr={11: _p(11, 8)}), "y is not"), (dict(z=(_p(5, 4), None)), "Wgu_z"),
    (dict(z=(None, _p(9, 2))), "Wd_z"), (dict(ws=_p(20, 64)), "workspace")])
def test_forward_int4_refuses(lib, kw, err):
    assert _fwd4(lib, **kw) == INVALID
    assert err in lib.moe_last_error().decode(), lib.moe_last_error()


def test_forward_int4_workspace_and_no_tokens(lib):
    need = lib.moe_workspace_bytes(8, 64, 8, 2, 64)
    assert _fwd4(lib, ws_bytes=need - 1) == WORKSPACE and _fwd4(lib, ws=None) == WORKSPACE
    assert _fwd4(lib, T=0, ws=None, ws_bytes=0) == OK


def test_int4_rows_from_four_gib_on_are_refused(lib):
    """Before anything is enqueued; one row less is taken (T = 0 stands in for it here)."""
    UNSUPPORTED = 2
    T = (1 << 32) // (2 * 2880) + 1
    assert _fwd4(lib, T=T, H=2880, ws_bytes=1 << 60) == UNSUPPORTED and b"x of" in lib.moe_last_error()
    assert _fwd4(lib, T=1 << 20, k=2, I=1024, H=32, ws_bytes=1 << 60) == UNSUPPORTED and b"h of" in lib.moe_last_error()
    v = _p
    assert lib.moe_gate_up_int4(v(0), v(1), v(2), None, *[v(i) for i in range(4, 8)], T, 2880, 8, 2, 64, 32, v(9), 0, None) == UNSUPPORTED
    assert lib.moe_down_int4(v(0), v(1), v(2), None, *[v(i) for i in range(4, 7)], T, 64, 8, 1, 2880, 32, v(9), 0, None) == UNSUPPORTED


def test_int4_stages_quantizer_and_packer_refuse(lib):
    v = _p
    gate_up = lambda **kw: lib.moe_gate_up_int4(*[v(i) for i in range(3)], kw.get("z"), *[v(i) for i in range(4, 8)],  # noqa: E731
                                                4, kw.get("H", 64), 8, 2, 64, kw.get("G", 32), v(9), kw.get("path", 0), None)
    down = lambda **kw: lib.moe_down_int4(*[v(i) for i in range(3)], kw.get("z"), *[v(i) for i in range(4, 7)],  # noqa: E731
                                          4, 64, 8, 2, kw.get("I", 64), kw.get("G", 32), kw.get("o", v(9)), kw.get("path", 0), None)
    for call in (gate_up, down):
        assert call(G=33) == INVALID and call(path=9) == INVALID and call(z=_p(3, 4)) == INVALID
    assert gate_up(H=40) == INVALID and down(I=40) == INVALID and down(o=None) == INVALID
    for E, K, N, G in ((0, 64, 64, 32), (2, 48, 64, 32), (2, 64, 60, 32), (2, 64, 64, 48), (2, 0, 64, 32), (2, 64, 40000, 32)):
        assert lib.moe_quantize_int4(v(0), E, K, N, G, v(1), v(2), None, None) == INVALID
    for E, K, N in ((0, 64, 64), (2, 48, 64), (2, 64, 60)):
        assert lib.moe_pack_int4(v(0), E, K, N, v(1), None) == INVALID
    assert lib.moe_pack_int4(v(0), 2, 64, 64, v(0), None) == INVALID and lib.moe_pack_int4(None, 2, 64, 64, v(1), None) == INVALID
    assert lib.moe_quantize_int4(v(0), 2, 64, 64, 32, v(1), None, None, None) == INVALID


@pytest.mark.parametrize("e_begin,n_local", [(-1, 2), (0, 0), (7, 2), (0, 9)])
def test_int4_rank_range(lib, e_begin, n_local):
    st = lib.moe_forward_ep_int4(*[_p(i) for i in range(5)], None, *[_p(i) for i in range(6, 9)], None, _p(10), 8, 64, 8, 2, 64, 32,
                                 e_begin, n_local, _p(11), None, None, _p(20), 1 << 30, 0, None)
    assert st == INVALID and b"local experts" in lib.moe_last_error()


# ---------------------------------------------------------------------------
# the binding: shapes, dtypes, groups (CPU tensors end at the device check)
# ---------------------------------------------------------------------------
T, H, E, I, k = 5, 96, 4, 64, 2


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _int4(G=32):
    ng = lambda K: -(-K // G)  # noqa: E731
    return dict(x=_bf(T, H), Wr=_bf(E, H), br=_bf(E), Wgu_q=_u8(E, 2, H // 32, 1024), Wgu_s=_bf(E, ng(H), 2 * I),
                bgu=_bf(E, 2 * I), Wd_q=_u8(E, 2, I // 32, 1024), Wd_s=_bf(E, ng(I), H), bd=_bf(E, H),
                Wgu_z=_u8(E, ng(H), 2 * I), Wd_z=_u8(E, ng(I), H))


def _raises(call, word):
    with pytest.raises(binding.MoEError) as ei:
        call()
    assert word in str(ei.value), str(ei.value)


@pytest.mark.parametrize("G", [32, 64, 128])
def test_well_formed_int4_arguments_reach_the_device_check(G):
    _raises(lambda: binding.moe_forward_int4(**_int4(G), k=k), "must be on the GPU")


@pytest.mark.parametrize("name,bad,word", [
    ("Wgu_q", _u8(E, 1, H // 32, 1024), "Wgu_q"), ("Wgu_q", _bf(E, 2, H // 32, 1024), "Wgu_q"), ("Wd_q", _u8(E, 2, 1, 1024), "Wd_q"),
    ("Wgu_s", _bf(E, 3, 2 * I - 8), "I=60"), ("Wgu_s", _bf(E, 3, 2 * I + 64), "Wgu_q"), ("Wd_s", torch.zeros(E, 2, H), "Wd_s"), ("Wgu_s", _bf(E, 5, 2 * I), "Wgu_z"),
    ("Wgu_z", _u8(E, 3, 2 * I - 1), "Wgu_z"), ("Wd_z", _bf(E, 2, H), "Wd_z"), ("bgu", _bf(E, I), "bgu"), ("bd", _bf(E - 1, H), "bd"),
    ("br", _bf(E + 1), "br")])
def test_int4_argument_shapes(name, bad, word):
    _raises(lambda: binding.moe_forward_int4(**(_int4() | {name: bad}), k=k), word)


def test_int4_group_follows_from_the_scales():
    assert binding._int4_group((2880, 90)) == 32 and binding._int4_group((2880, 45)) == 64
    assert binding._int4_group((2880, 23), (64, 1)) == 128 and binding._int4_group((32, 1)) == 32
    _raises(lambda: binding._int4_group((2880, 90), (2880, 45)), "90 scales")
    _raises(lambda: binding._int4_group((2880, 22)), "22 scales")
    a = _int4(32)
    b = _int4(64)
    a.update(Wd_s=b["Wd_s"], Wd_z=b["Wd_z"])
    _raises(lambda: binding.moe_forward_int4(**a, k=k), "scales")


def test_norm_argument_shapes():
    x, g = _bf(T, H), _bf(H)
    _raises(lambda: binding.moe_add_rmsnorm(x, g), "must be on the GPU")
    _raises(lambda: binding.moe_add_rmsnorm(x, _bf(H - 8)), "gamma")
    _raises(lambda: binding.moe_add_rmsnorm(x.float(), g), "x: expected")
    _raises(lambda: binding.moe_add_rmsnorm(x, g, residual=_bf(T + 1, H)), "residual")
    _raises(lambda: binding.moe_add_rmsnorm(x, g, residual_out=_bf(T, H)), "without a residual")
    _raises(lambda: binding.moe_add_rmsnorm(x, g, y=torch.zeros(T, H)), "y: expected")
    _raises(lambda: binding.moe_add_rmsnorm_fp8(x, g, codes=_bf(T, H)), "codes")
    _raises(lambda: binding.moe_add_rmsnorm_fp8(x, g, scales=torch.zeros(T + 1)), "scales")
    _raises(lambda: binding.moe_add_rmsnorm(_bf(H), g), "x: expected 2")


def test_int4_format_by_hand():
    """The packed bytes of a small matrix, value by value from the documented bit positions, and the dequantiser."""
    rng = np.random.default_rng(1)
    E_, K_, N_ = 2, 64, 72
    q = rng.integers(0, 16, (E_, K_, N_), dtype=np.uint8)
    words = orc.int4_pack(q).view("<u4").reshape(E_, 2, K_ // 32, 256)
    for e, kk, n in ((0, 0, 0), (1, 63, 71), (0, 37, 5), (1, 15, 66), (0, 31, 63), (1, 7, 64)):
        g, i, c, j = kk % 32 // 8, kk % 8, n % 64 // 4, n % 4
        w = int(words[e, n // 64, kk // 32, 4 * (16 * g + c) + j])
        bits = [w >> ((3 + 4 * (i // 2) + 16 * (i % 2) + b) % 32) & 1 for b in range(4)]
        assert sum(v << b for b, v in enumerate(bits)) == q[e, kk, n]
    s = np.full((3, N_), 0x3F80, np.uint16)
    s[1] = 0x4000
    z = rng.integers(0, 16, (3, N_), dtype=np.uint8)
    W = orc.int4_dequantize(q[0][:64], s[:2], z[:2], 32)
    assert W[40, 9] == (int(q[0, 40, 9]) - int(z[1, 9])) * 2.0 and W[31, 3] == int(q[0, 31, 3]) - int(z[0, 3])
    assert orc.int4_dequantize(q[0], s[:1], None, 64)[63, 7] == int(q[0, 63, 7]) - 8


def test_int4_quantizer_error_is_at_most_half_a_step():
    """Every weight comes back within half a step of its group's scale (and the clipping that a scale rounded down to
    bf16 can add: 7 or 15 steps times 2^-8)."""
    rng = np.random.default_rng(2)
    W = rng.standard_normal((1, 96, 24)).astype(np.float32)
    bits = (W.view(np.uint32) >> 16).astype(np.uint16)
    for zeros, steps in ((False, 7), (True, 15)):
        q, s, z = orc.int4_quantize(bits, 64, zeros)
        back = orc.int4_dequantize(q[0], s[0], None if z is None else z[0], 64)
        step = orc.widen(s[0])[np.arange(96) // 64]
        # the zero point's own rounding can add another half step at either end
        assert (np.abs(back - orc.widen(bits[0])) <= step * (0.5 + (0.5 if zeros else 0.0) + steps * 2.0 ** -8)).all()
