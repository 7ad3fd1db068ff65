"""Residual addition and RMS norm (bf16 rows and FP8 codes), and the block that
runs behind it, against the oracle (needs an MI355X).

The norm's definition fixes every float32 rounding and takes its sum of exact
squares in float64, so the kernel and the oracle can only part where two
orders of a float64 sum (2^-52) fall on two sides of a float32 border (2^-24):
about one row in 10^8.  The comparisons are therefore bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rows(T, H, seed, std=3.0):
    return d.normal_bf16((T, H), std, seed, 91, T, H)


def _gamma(H, seed):
    return d.f32_to_bf16_bits(1.0 + 0.3 * np.random.default_rng(seed + 5).standard_normal(H).astype(np.float32))


def _bits(v):
    """float64 values of bf16 -> bits."""
    return (np.asarray(v, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _same_bits(got, want, what):
    """Equal bits; any NaN matches any NaN."""
    nan = np.isnan(orc.widen(want))
    bad = np.argwhere(np.where(nan, ~np.isnan(orc.widen(got)), got != want))
    assert bad.size == 0, f"{what} differs at {bad[:5].tolist()} ({len(bad)} values)"


def _check(x, res, gamma, eps, y, r, codes=None, scales=None):
    with np.errstate(all="ignore"):
        y_ref, r_ref, v = orc.add_rmsnorm(x, res, gamma, eps)
    _same_bits(bf16_bits(r), _bits(r_ref), "r")
    _same_bits(bf16_bits(y), _bits(y_ref), "y")
    if codes is not None:
        with np.errstate(all="ignore"):
            c_ref, s_ref = orc.fp8_quantize_rows(v)
        s = scales.cpu().numpy()
        assert ((s == s_ref) | (np.isnan(s) & np.isnan(s_ref))).all(), np.argwhere(s != s_ref)[:5].tolist()
        bad = np.argwhere(codes.cpu().numpy() != c_ref)
        assert bad.size == 0, f"codes differ at {bad[:5].tolist()} ({len(bad)} values)"


SIZES = [(1, 16), (1, 2880), (2, 512), (7, 528), (64, 2880), (33, 4096), (3, 16384), (5, 8208), (300, 64), (130, 1040),
         (2500, 2880), (9000, 496)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_fp8_matches_oracle(T, H, residual):
    _need_gpu()
    x, res, gamma = _rows(T, H, 1), _rows(T, H, 2, 8.0) if residual else None, _gamma(H, 3)
    y, codes, scales, r = binding.moe_add_rmsnorm_fp8(dev(x), dev(gamma), None if res is None else dev(res), eps=EPS)
    _check(x, res, gamma, EPS, y, r, codes, scales)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H", SIZES + [(1, 8), (5, 24), (40, 2888), (70000, 8)])
def test_norm_bf16_matches_oracle(T, H, residual):
    _need_gpu()
    x, res, gamma = _rows(T, H, 4), _rows(T, H, 5, 0.5) if residual else None, _gamma(H, 6)
    y, r = binding.moe_add_rmsnorm(dev(x), dev(gamma), None if res is None else dev(res), eps=1e-6)
    _check(x, res, gamma, 1e-6, y, r)


def test_unusual_rows():
    """Zero rows, NaN and infinite values, subnormal and huge rows, rows whose 448 / max overflows: each row by itself."""
    _need_gpu()
    T, H = 14, 2880
    f = d.f32_to_bf16_bits
    x = _rows(T, H, 7)
    x[0] = 0
    x[1] = 0x8000                                     # -0
    x[2, 17] = 0x7FC0                                 # NaN
    x[3, 2879] = 0x7F80                               # +inf
    x[4, 0], x[4, 1] = 0x7F80, 0xFF80                 # both infinities
    x[5] = np.arange(H, dtype=np.uint16) % 120        # subnormals
    x[6] = f(np.full(H, 3.0e38, np.float32))          # squares past float32
    x[7] = 0
    x[7, 5] = 0x4000                                  # one value
    x[8] = f(np.linspace(-1e-30, 1e-30, H, dtype=np.float32))
    x[9] = f((2.0 ** (np.arange(H) % 30 - 20)).astype(np.float32))
    x[10, :] = 0x3F80                                 # all equal
    res = np.zeros_like(x)
    res[11] = x[11] ^ 0x8000                          # the sum cancels
    res[12, 3] = 0xFFC0
    res[13] = f(np.full(H, 3.3e38, np.float32))
    x[13] = res[13]                                   # the sum overflows
    gamma = _gamma(H, 8)
    gamma[100], gamma[101] = 0, 0x8000
    for r_in in (None, res):
        y, codes, scales, r = binding.moe_add_rmsnorm_fp8(dev(x), dev(gamma), None if r_in is None else dev(r_in), eps=EPS)
        _check(x[:13] if r_in is not None else x, None if r_in is None else r_in[:13], gamma, EPS,
               *(t[:13] if r_in is not None else t for t in (y, r, codes, scales)))
        if r_in is not None:                          # bf16(x + residual) past the largest finite: infinite, then NaN
            assert np.isinf(host_f64(r)[13]).all() and np.isnan(host_f64(y)[13]).all()
            assert (codes.cpu().numpy()[13] == 0x7F).all()
    tiny = f(np.full(H, 1e-38, np.float32))           # normalised rows near 1e-38: 448 / max is infinite
    tiny[7] = 0
    y, codes, scales, r = binding.moe_add_rmsnorm_fp8(dev(x[9:12]), dev(tiny), eps=EPS)
    _check(x[9:12], None, tiny, EPS, y, r, codes, scales)


def test_code_borders():
    """Rows whose normalised values are the midpoints between codes: a row of +-1 has 1 / rms within rounding of 1, so
    gamma sets the values."""
    _need_gpu()
    mids = np.array([0.5 * (a + b) for a, b in zip(orc.E4M3_VALUES[:126], orc.E4M3_VALUES[1:127])])
    vals = np.concatenate([mids, orc.E4M3_VALUES[:127], [448.0]])
    H = -(-len(vals) // 16) * 16
    gamma = np.zeros(H, np.float32)
    gamma[:len(vals)] = vals
    gamma = d.f32_to_bf16_bits(gamma)
    x = np.full((3, H), 0x3F80, np.uint16)
    x[1, ::2] = 0xBF80
    x[2] = _rows(1, H, 9)[0]
    y, codes, scales, r = binding.moe_add_rmsnorm_fp8(dev(x), dev(gamma), eps=1e-30)
    _check(x, None, gamma, 1e-30, y, r, codes, scales)


def test_row_results_do_not_depend_on_the_batch():
    _need_gpu()
    H, T = 2880, 5000
    x, res, gamma = dev(_rows(T, H, 10)), dev(_rows(T, H, 11)), dev(_gamma(H, 12))
    big = binding.moe_add_rmsnorm_fp8(x, gamma, res)
    for lo, n in ((0, 1), (1, 2), (17, 64), (4000, 700)):
        part = binding.moe_add_rmsnorm_fp8(x[lo:lo + n], gamma, res[lo:lo + n])
        for a, b in zip(big, part):
            assert torch.equal(a[lo:lo + n].view(torch.uint8), b.view(torch.uint8)), (lo, n)


@pytest.mark.parametrize("T", [1, 3000])
def test_in_place(T):
    _need_gpu()
    H = 2880
    x, res, gamma = dev(_rows(T, H, 13)), dev(_rows(T, H, 14)), dev(_gamma(H, 15))
    y, r = binding.moe_add_rmsnorm(x, gamma, res)
    for r_at, y_at in (("res", "x"), ("x", "res"), ("x", None), (None, "x"), ("res", None)):
        b = {"x": x.clone(), "res": res.clone(), None: None}
        y2, r2 = binding.moe_add_rmsnorm(b["x"], gamma, b["res"], residual_out=b[r_at], y=b[y_at])
        assert torch.equal(y, y2) and torch.equal(r, r2), (r_at, y_at)
    x2 = x.clone()
    y3, r3 = binding.moe_add_rmsnorm(x2, gamma, y=x2)
    assert r3 is x2 and torch.equal(y3, binding.moe_add_rmsnorm(x, gamma)[0])


def test_offsets_past_32_bits():
    """5 GB of rows: the last ones as by themselves."""
    _need_gpu()
    T, H = 320000, 8192
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).fill_(0x3F80)
    tail = dev(_rows(5, H, 16))
    x[-5:] = tail
    gamma = dev(_gamma(H, 17))
    y, codes, scales, r = binding.moe_add_rmsnorm_fp8(x, gamma)
    y2, codes2, scales2, _ = binding.moe_add_rmsnorm_fp8(tail, gamma)
    assert torch.equal(y[-5:], y2) and torch.equal(codes[-5:], codes2) and torch.equal(scales[-5:], scales2)


@pytest.mark.parametrize("H", [8, 1040])
def test_more_rows_than_workgroups(H):
    """2^21 rows and more: a workgroup takes several, one after the other."""
    _need_gpu()
    T = (1 << 21) + 5 if H == 8 else (1 << 22) + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = dev(_gamma(H, 34))
    n = H if H % 16 == 0 else None                                   # FP8 rows come in sixteens
    y = torch.empty_like(x)
    codes = torch.empty((T, H), dtype=torch.uint8, device="cuda") if n else None
    scales = torch.empty((T,), device="cuda") if n else None
    if n:
        binding.moe_add_rmsnorm_fp8(x, gamma, y=y, codes=codes, scales=scales)
    else:
        binding.moe_add_rmsnorm(x, gamma, y=y)
    for lo in (0, (1 << 21) - 4, T - 9):
        part = binding.moe_add_rmsnorm_fp8(x[lo:lo + 9], gamma) if n else binding.moe_add_rmsnorm(x[lo:lo + 9], gamma)
        m = len(part[0])
        assert torch.equal(y[lo:lo + m], part[0]), lo
        if n:
            assert torch.equal(codes[lo:lo + m], part[1]) and torch.equal(scales[lo:lo + m], part[2]), lo


def test_no_tokens():
    _need_gpu()
    x, gamma = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), dev(_gamma(64, 18))
    y, r = binding.moe_add_rmsnorm(x, gamma, x.clone())
    assert y.shape == (0, 64) and r.shape == (0, 64)
    y, codes, scales, r = binding.moe_add_rmsnorm_fp8(x, gamma)
    assert codes.shape == (0, 64) and scales.shape == (0,)


def test_other_stream():
    """On a stream that is not the current one, with outputs that the call allocates."""
    _need_gpu()
    T, H = 2000, 2880
    x, res, gamma = dev(_rows(T, H, 19)), dev(_rows(T, H, 20)), dev(_gamma(H, 21))
    want = binding.moe_add_rmsnorm_fp8(x, gamma, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = binding.moe_add_rmsnorm_fp8(x, gamma, res, stream=stream)
        s.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _block(T, E, H, I, k, seed):
    cfg = d.small_config(T=T, E=E, H=H, I=I, k=k)
    Wr, br = d.make_router(cfg, seed)
    return (Wr, br, *d.make_experts_fp8(cfg, seed, threads=4))


def _dev_any(a):
    return dev(a) if a.dtype == np.uint16 else torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("path", ["gemv", "gemm"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,E,H,I,k", [(1, 4, 32, 32, 1), (5, 8, 64, 96, 2), (70, 4, 160, 32, 2), (200, 16, 256, 160, 4),
                                       (17, 8, 2880, 2880, 4)])
def test_forward_norm_fp8(T, E, H, I, k, residual, path):
    _need_gpu()
    x, res, gamma = _rows(T, H, 22), _rows(T, H, 23) if residual else None, _gamma(H, 24)
    w = _block(T, E, H, I, k, 25)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    y, r = binding.moe_forward_norm_fp8(dev(x), dev(gamma), *[_dev_any(a) for a in w], k=k,
                                        residual=None if res is None else dev(res), eps=EPS, topk_ids=ids, topk_w=tw,
                                        path=path)
    ref = orc.moe_forward_norm_fp8(x, res, gamma, EPS, *w, k=k)
    _same_bits(bf16_bits(r), _bits(ref["residual"]), "r")
    assert_routing(ids.cpu().numpy(), tw.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"], f"y T{T} E{E} H{H}")


@pytest.mark.parametrize("path", ["gemv", "gemm"])
def test_norm_and_stages_match_the_whole_call(path):
    """The pieces as a caller would chain them (norm, route, permute, gate_up from the norm's codes, quantised h, down,
    combine) give the whole call's bits."""
    _need_gpu()
    T, E, H, I, k = 96, 8, 256, 160, 4
    x, res, gamma = dev(_rows(T, H, 26)), dev(_rows(T, H, 27)), dev(_gamma(H, 28))
    Wr, br, gq, gs, bgu, dq, ds, bd = [_dev_any(a) for a in _block(T, E, H, I, k, 29)]
    y, r = binding.moe_forward_norm_fp8(x, gamma, Wr, br, gq, gs, bgu, dq, ds, bd, k=k, residual=res, path=path)
    n, xq, sx, r2 = binding.moe_add_rmsnorm_fp8(x, gamma, res)
    ids, w = binding.moe_route(n, Wr, br, k)
    cnt, off, rows, pos = binding.moe_permute(ids, E)
    h = binding.moe_gate_up_fp8(xq, sx, gq, gs, bgu, cnt, off, rows, k, path=path)
    o = binding.moe_down_fp8(*binding.moe_quantize_rows_fp8(h), dq, ds, bd, cnt, off, T, k, path=path)
    assert torch.equal(r, r2) and torch.equal(y, binding.moe_combine(o, pos, w))


def test_forward_norm_fp8_in_a_graph():
    """Captured and replayed between eager calls on the same buffers, in place on the residual stream."""
    _need_gpu()
    T, E, H, I, k = 48, 8, 256, 160, 4
    x0, res0, gamma = dev(_rows(T, H, 30)), dev(_rows(T, H, 31)), dev(_gamma(H, 32))
    w = [_dev_any(a) for a in _block(T, E, H, I, k, 33)]
    ws = binding.alloc_workspace_norm_fp8(T, H, E, k, I)
    x, res, y = x0.clone(), res0.clone(), torch.empty_like(x0)

    def step():
        binding.moe_forward_norm_fp8(x, gamma, *w, k=k, residual=res, residual_out=res, y=y, workspace=ws)

    y_ref, r_ref = binding.moe_forward_norm_fp8(x0, gamma, *w, k=k, residual=res0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(x0), res.copy_(res0), y.fill_(-1.0), ws.fill_(0xAB if i % 2 else 0x11)
        binding.moe_forward_norm_fp8(x0, gamma, *w, k=k, residual=res0)   # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y_ref) and torch.equal(res, r_ref), i
