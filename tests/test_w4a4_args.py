"""Refusals of the calls with MXFP4 rows, in the C ABI and in the binding (CPU
only: nothing here reaches a launch), and the oracle's row format against a
scalar reading of it."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle.moe_oracle as orc
from moe_layer_route_amd import binding

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BASE = 1 << 36     # addresses that are never read, 64 GiB apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.library()


def _p(i, add=0):
    return ctypes.c_void_p(BASE * (i + 1) + add)


def _q(lib, R=4, K=64, a=_p(0), codes=_p(1), scales=_p(2)):
    return lib.moe_quantize_rows_mxfp4(a, R, K, codes, scales, None)


def _dq(lib, R=4, K=64, a=_p(0), codes=_p(1), scales=_p(2)):
    return lib.moe_dequantize_rows_mxfp4(codes, scales, R, K, a, None)


@pytest.mark.parametrize("call,name", [(_q, "a"), (_dq, "out")])
def test_rows_refuse(lib, call, name):
    for kw, err in [(dict(R=-1), "R=-1"), (dict(R=1 << 31), "R="), (dict(K=0), "K=0"), (dict(K=48), "K=48"),
                    (dict(K=16416), "K=16416"), (dict(a=None), f"{name} is NULL"), (dict(codes=None), "codes is NULL"),
                    (dict(scales=None), "scales is NULL"), (dict(a=_p(0, 8)), f"{name} is not"),
                    (dict(codes=_p(1, 8)), "codes is not"), (dict(scales=_p(2, 2)), "scales is not"),
                    (dict(codes=_p(0, 16)), f"codes overlaps {name}"), (dict(scales=_p(0, 508)), f"scales overlaps {name}"),
                    (dict(scales=_p(1, 124)), "scales overlaps codes")]:
        assert call(lib, **kw) == INVALID, kw
        assert err in lib.moe_last_error().decode(), (kw, lib.moe_last_error())
    assert call(lib, R=0) == OK


def _fwd(lib, T=4, H=64, E=8, k=2, I=64, ptrs=None, ids=None, w=None, ws=_p(30), ws_bytes=1 << 40, path=0):
    p = ptrs or [_p(i) for i in range(10)]
    return lib.moe_forward_w4a4(*p[:9], T, H, E, k, I, p[9], ids, w, ws, ws_bytes, path, None)


def test_forward_refuses(lib):
    for kw, err in [(dict(H=48), "multiples of 32"), (dict(I=40), "multiples of 32"), (dict(T=-1), "T=-1"),
                    (dict(k=9), "k=9"), (dict(E=257), "E=257"), (dict(path=3), "unknown path"), (dict(path=-1), "unknown path"),
                    (dict(ids=_p(11, 2)), "topk_ids_out"), (dict(w=_p(11, 2)), "topk_w_out")]:
        assert _fwd(lib, **kw) == INVALID, kw
        assert err in lib.moe_last_error().decode(), (kw, lib.moe_last_error())
    for i in range(10):
        ptrs = [_p(j) for j in range(10)]
        ptrs[i] = None
        assert _fwd(lib, ptrs=ptrs) == INVALID and b"is NULL" in lib.moe_last_error()
    need = lib.moe_workspace_bytes_w4a4(4, 64, 8, 2, 64)
    assert need > 0 and _fwd(lib, ws_bytes=need - 1) == WORKSPACE and _fwd(lib, ws=None) == WORKSPACE
    assert _fwd(lib, ws=_p(30, 16)) == INVALID and b"256-byte" in lib.moe_last_error()
    assert _fwd(lib, T=0) == OK
    # rows past what the kernels address: refused before anything is enqueued
    assert _fwd(lib, T=1 << 20, H=16384, k=1) == UNSUPPORTED and b"x of" in lib.moe_last_error()
    assert _fwd(lib, T=1 << 18, H=32, I=16384, k=1) == UNSUPPORTED and b"h of" in lib.moe_last_error()
    assert lib.moe_workspace_bytes_w4a4(4, 64, 0, 2, 64) == 0 and lib.moe_workspace_bytes_w4a4(4, 40, 8, 2, 64) == 0
    assert lib.moe_workspace_bytes_w4a4(0, 64, 8, 2, 64) == 0


def test_variants_refuse(lib):
    p = [_p(i) for i in range(9)]

    def padded(n_valid=None, counts=None, path=0, T=4, ws_bytes=1 << 40):
        return lib.moe_forward_padded_w4a4(*p, T, 64, 8, 2, 64, n_valid, _p(9), None, None, counts, _p(30), ws_bytes, path, None)

    def ep(lo=0, n=8, T=4):
        return lib.moe_forward_ep_w4a4(*p, T, 64, 8, 2, 64, lo, n, _p(9), None, None, _p(30), 1 << 40, 0, None)
    assert padded(n_valid=_p(11, 2)) == INVALID and b"n_valid" in lib.moe_last_error()
    assert padded(counts=_p(11, 1)) == INVALID and b"expert_counts_out" in lib.moe_last_error()
    assert padded(ws_bytes=16) == WORKSPACE and padded(T=0) == OK and padded(path=9) == INVALID
    for lo, n in ((-1, 4), (0, 0), (0, 9), (5, 4)):
        assert ep(lo, n) == INVALID and b"local experts" in lib.moe_last_error()
    assert ep(T=0) == OK


def test_stages_refuse(lib):
    def gate_up(T=4, H=64, E=8, k=2, I=64, path=0, **at):
        names = ("xq", "sx", "Wgu_q", "Wgu_s", "bgu", "cnt", "off", "rows", "hq", "sh")
        a = [at.get(n, _p(i)) for i, n in enumerate(names)]
        return lib.moe_gate_up_w4a4(*a[:8], T, H, E, k, I, a[8], a[9], path, None)

    def down(T=4, H=64, E=8, k=2, I=64, path=0, **at):
        names = ("hq", "sh", "Wd_q", "Wd_s", "bd", "cnt", "off", "o")
        a = [at.get(n, _p(i)) for i, n in enumerate(names)]
        return lib.moe_down_w4a4(*a[:7], T, H, E, k, I, a[7], path, None)
    for call, names in ((gate_up, ("xq", "sx", "Wgu_q", "Wgu_s", "bgu", "cnt", "off", "rows", "hq", "sh")),
                        (down, ("hq", "sh", "Wd_q", "Wd_s", "bd", "cnt", "off", "o"))):
        for n in names:
            assert call(**{n: None}) == INVALID and f"{n} is NULL" in lib.moe_last_error().decode()
            assert call(**{n: _p(3, 2)}) == INVALID and f"{n} is not" in lib.moe_last_error().decode()
        for kw in (dict(H=40), dict(I=48), dict(T=-1), dict(path=3), dict(k=0)):
            assert call(**kw) == INVALID, kw
        assert call(T=0) == OK
    assert gate_up(T=1 << 27, H=64, k=1, I=32) == UNSUPPORTED and b"x of" in lib.moe_last_error()
    assert gate_up(T=1 << 25, H=32, k=4, I=32) == UNSUPPORTED and b"h of" in lib.moe_last_error()
    assert down(T=1 << 25, H=32, k=4, I=32) == UNSUPPORTED


# ------------------------------------------------------------------------------------------------ the binding
def _t(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_shapes():
    bf = torch.bfloat16
    E, T, k, H, I = 4, 6, 2, 64, 96
    gu = (_t(E, 2 * I, H // 2), _t(E, H // 32, 2 * I), _t(E, 2 * I, dtype=bf))
    dn = (_t(E, H, I // 2), _t(E, I // 32, H), _t(E, H, dtype=bf))
    cnt, off, rows = _t(E, dtype=torch.int32), _t(E + 1, dtype=torch.int32), _t(T * k, dtype=torch.int32)
    xq, sx, hq, sh = _t(T, H // 2), _t(1, T, 4), _t(T * k, I // 2), _t(1, T * k, 4)

    def refused(match, f, *a, **kw):
        with pytest.raises(binding.MoEError, match=match):
            f(*a, **kw)
    q, dq = binding.moe_quantize_rows_mxfp4, binding.moe_dequantize_rows_mxfp4
    refused("a: expected torch.bfloat16", q, _t(T, H, dtype=torch.float16))
    refused("2 dimensions", q, _t(T, 2, H, dtype=bf))
    refused("codes: expected shape", q, _t(T, H, dtype=bf), codes=_t(T, H))
    refused("scales: expected shape", q, _t(T, H, dtype=bf), scales=_t(T, 4))
    refused("GPU", q, _t(T, H, dtype=bf))
    refused("scales: expected shape", dq, xq, _t(2, T, 4))
    refused("out: expected", dq, xq, sx, out=_t(T, H, dtype=torch.float32))
    refused("codes: expected torch.uint8", dq, xq.to(torch.int8), sx)
    g, dd = binding.moe_gate_up_w4a4, binding.moe_down_w4a4
    refused("sx: expected shape", g, xq, _t(1, T + 1, 4), *gu, cnt, off, rows, k)
    refused("Wgu_s: expected shape", g, xq, sx, gu[0], _t(E, 2 * I, H // 32), gu[2], cnt, off, rows, k)
    refused("Wgu_q: expected", g, xq, sx, _t(E, 2 * I, H), gu[1], gu[2], cnt, off, rows, k)
    refused("bgu: expected", g, xq, sx, gu[0], gu[1], _t(E, 2 * I), cnt, off, rows, k)
    refused("rows: expected", g, xq, sx, *gu, cnt, off, rows[:-1], k)
    refused("hq: expected shape", g, xq, sx, *gu, cnt, off, rows, k, hq=_t(T * k + 1, I // 2))
    refused("sh: expected shape", g, xq, sx, *gu, cnt, off, rows, k, sh=_t(1, T, 4))
    refused("GPU", g, xq, sx, *gu, cnt, off, rows, k)
    refused("hq: expected shape", dd, hq[:-1], sh, *dn, cnt, off, T, k)
    refused("cnt: expected", dd, hq, sh, *dn, cnt.long(), off, T, k)
    refused("o: expected shape", dd, hq, sh, *dn, cnt, off, T, k, o=_t(T * k - 1, H, dtype=torch.float32))
    x, Wr, br = _t(T, H, dtype=bf), _t(E, H, dtype=bf), _t(E, dtype=bf)
    f = binding.moe_forward_w4a4
    refused("y: expected", f, x, Wr, br, *gu, *dn, k=k, y=_t(T, H, dtype=torch.float32))
    refused("Wd_s: expected", f, x, Wr, br, *gu, dn[0], _t(E, H, I // 32), dn[2], k=k)
    refused("GPU", f, x, Wr, br, *gu, *dn, k=k)
    refused("n_valid", binding.moe_forward_padded_w4a4, x, Wr, br, *gu, *dn, k=k, n_valid=_t(1, dtype=torch.int64))
    refused("expert range", binding.moe_forward_ep_w4a4, x, Wr, br, *gu, *dn, e_begin=1, k=k)


# ------------------------------------------------------------------------------------------------ the format
def test_row_format_by_hand():
    """A row of five blocks: scales side by side in fours, codes low nibble first, a block that is not finite."""
    a = np.zeros((2, 160))
    a[1, :4] = 6.0, -0.5, 0.25, 5.0          # max 6: floor(log2) - 2 = 0; ties to the even code: 0.25 -> 0, 5 -> 4
    a[1, 32] = 1.0                           # 2^-2: the code of 4
    a[1, 96] = np.inf
    a[1, 128:131] = 2.0 ** -140, 0.0, -(2.0 ** -128)   # below the smallest unit
    codes, scales = orc.mxfp4_quantize_rows(a)
    assert scales.shape == (2, 2, 4)
    assert scales[:, 0].tolist() == [[0, 0, 0, 0], [0, 0, 0, 0]] and scales[:, 1].tolist() == [[127, 125, 0, 255], [0, 0, 0, 0]]
    assert codes[1, :2].tolist() == [7 | 9 << 4, 0 | 6 << 4] and codes[1, 16] == 6 and (codes[1, 48:64] == 0).all()
    assert codes[1, 64:66].tolist() == [0, 1 | 8]
    v = orc.mxfp4_dequantize_rows(codes, scales)
    assert v[1, :4].tolist() == [6.0, -0.5, 0.0, 4.0] and v[1, 32] == 1.0 and np.isnan(v[1, 96:128]).all()
    assert v[1, 130] == -(2.0 ** -128) and (v[0] == 0).all()
