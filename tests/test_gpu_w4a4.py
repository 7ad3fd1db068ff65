"""MXFP4 rows and the block with MXFP4 on both sides against the float64 oracle
(needs an MI355X).  Every call goes through the C ABI.

Rows: bit for bit (the scale is read off an exponent and the codes are exact
comparisons).

Products, derived: products of two E2M1 values and powers of two are exact in
float32.  A matrix instruction adds 64 or 128 of them to the accumulator; its
result is within 2^-23 of the sum of the terms' magnitudes A (an ulp, the
instruction may truncate), so K/64 instructions and the joining of at most
eight parts and the bias stay within (K / 64 + 9) 2^-23 (A + |bias|).
h: the GLU's slopes are at most 8.8 in gate and 7 in up, the hardware
exponential and reciprocal within 2^-20 of h; rounding to bf16 and to MXFP4 are
monotonic, so with the block scale that was chosen, the code lies between those
of h - tol and h + tol, and the scale between those of the blocks' maxima.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402

pytestmark = pytest.mark.gpu
PATHS = ["gemv", "gemm"]
ULP = 2.0 ** -23


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _up(a):
    return dev(a) if a.dtype == np.uint16 else torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------------------------------------ rows
def _check_rows(a, codes, scales):
    c, s = orc.mxfp4_quantize_rows(orc.widen(a))
    got = scales.cpu().numpy()
    assert (got == s).all(), f"scales differ at {np.argwhere(got != s)[:5].tolist()}"
    bad = np.argwhere(codes.cpu().numpy() != c)
    assert bad.size == 0, f"codes differ at {bad[:5].tolist()} ({len(bad)} bytes)"


@pytest.mark.parametrize("R,K", [(1, 32), (1, 2880), (3, 96), (15, 128), (16, 160), (17, 2880), (64, 2880), (2, 16384),
                                 (1000, 64), (257, 1056)])
def test_rows_match_oracle(R, K):
    _need_gpu()
    a = d.normal_bf16((R, K), 3.0, 7, 1, R, K)
    a[:, K // 2] = d.f32_to_bf16_bits(np.full(R, 1e4, np.float32))
    codes, scales = binding.moe_quantize_rows_mxfp4(dev(a))
    _check_rows(a, codes, scales)
    back = binding.moe_dequantize_rows_mxfp4(codes, scales)
    want = orc.mxfp4_dequantize_rows(codes.cpu().numpy(), scales.cpu().numpy())
    assert (host_f64(back) == want).all() and (np.signbit(host_f64(back)) == np.signbit(want)).all()


def test_rows_every_bf16():
    """Every bf16 with every leading value of its block: the block's maximum is the row's index among the powers."""
    _need_gpu()
    v = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(2048, 32)
    for lead in (0x0000, 0x0001, 0x0080, 0x3F80, 0x4048, 0x7F7F, 0x7F80, 0x7FC0, 0xFF80):
        a = v.copy()
        a[:, 5] = np.where(np.arange(2048) % 2, lead, a[:, 5])
        codes, scales = binding.moe_quantize_rows_mxfp4(dev(a))
        _check_rows(a, codes, scales)


def test_rows_borders():
    """Midpoints of the codes and their neighbours under every power of two that a block can have, subnormals too."""
    _need_gpu()
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    rows = []
    for e in list(range(-126, 125)) + [-130]:
        with np.errstate(all="ignore"):
            b = d.f32_to_bf16_bits(np.ldexp(mids, e).astype(np.float32)).astype(np.int32)
        row = np.zeros(32, np.int32)
        row[:9], row[9:18], row[18:27] = b, np.maximum(b - 1, 0), np.minimum(b + 1, 0x7F7F)
        row[27] = d.f32_to_bf16_bits(np.ldexp(np.float32(4.0), e).astype(np.float32).reshape(1))[0]
        rows.append(row | (np.arange(32) % 2 << 15))
    a = np.array(rows).astype(np.uint16)
    codes, scales = binding.moe_quantize_rows_mxfp4(dev(a))
    _check_rows(a, codes, scales)


def test_dequantize_every_code_and_scale():
    _need_gpu()
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))      # 256 rows of 32 values
    scales = np.zeros((1, 256, 4), np.uint8)
    for s0 in range(0, 256, 16):
        scales[0, :, 0] = s0 + np.arange(256) // 16
        got = host_f64(binding.moe_dequantize_rows_mxfp4(_up(codes), _up(scales)))
        want = orc.mxfp4_dequantize_rows(codes, scales)
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()


def test_rows_many():
    """More rows than one launch of 2^16 workgroups along y would hold, ragged."""
    _need_gpu()
    R = (1 << 20) + 5
    a = torch.randn((R, 32), device="cuda").bfloat16()
    codes, scales = binding.moe_quantize_rows_mxfp4(a)
    back = binding.moe_dequantize_rows_mxfp4(codes, scales)
    pick = np.r_[0:64, R - 64:R]
    assert (host_f64(back)[pick] == orc.mxfp4_dequantize_rows(*orc.mxfp4_quantize_rows(host_f64(a)[pick]))).all()


# ------------------------------------------------------------------------------------------------ products
def _matrix(E, K, N, seed):
    rng = np.random.default_rng([seed, E, K, N])
    q = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    s = rng.integers(116, 123, (E, K // 32, N), dtype=np.uint8)
    s[:, -1, 0] = 0                                            # 2^-127
    s[0, 0, N - 1] = 140
    return q, s


def _rows(R, K, seed, std=3.0):
    return orc.mxfp4_quantize_rows(orc.widen(d.normal_bf16((R, K), std, seed, 3, R, K)))


def _routing(T, E, k, seed, live=None):
    """ids [T][k], all different in a row, among the first `live` experts."""
    rng = np.random.default_rng([seed, T, E])
    return np.stack([rng.permutation(live or E)[:k] for _ in range(T)]).astype(np.int32)


def _within(got, want, tol, what):
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} off, first {bad[0].tolist()}: {got[tuple(bad[0])]} for "
                           f"{want[tuple(bad[0])]} +- {tol[tuple(bad[0])]}")


# T, E, k, K (H or I), columns / 32, live experts
STAGES = [
    (1, 4, 1, 32, 1, None),        # one token, one block of K
    (1, 8, 4, 2880, 90, None),     # one token, fewer slots than experts
    (3, 8, 2, 96, 3, None),        # three blocks of K, columns that end inside a tile
    (16, 2, 1, 160, 2, None),      # about eight rows an expert, a lone block in the second step
    (17, 1, 1, 288, 4, None),      # 17 rows: one past a 16-row operand
    (33, 3, 2, 2880, 3, 2),        # full K, 33 rows: a third chunk; an expert without rows
    (100, 4, 2, 352, 7, None),     # 50 rows an expert
    (70, 2, 2, 64, 90, None),      # full width, 70 rows
    (300, 1, 1, 128, 3, None),     # 300 rows of one expert: past one 256-row tile
    (40, 40, 8, 224, 5, 30),       # many experts, k = 8
    (129, 5, 4, 1440, 9, None),    # 103 rows an expert
    (257, 1, 1, 544, 17, None),    # one row past a tile of rows, K and columns past a tile too
]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,k,K,n32,live", STAGES)
def test_down(T, E, k, K, n32, live, path):
    _need_gpu()
    N, S = 32 * n32, T * k
    q, s = _matrix(E, K, N, 1)
    bd = d.normal_bf16((E, N), 0.5, 2, 1, E, N)
    cnt, off, rows, pos = binding.moe_permute(_up(_routing(T, E, k, 3, live)), E)
    hq, sh = _rows(S, K, 4)
    sh[0, S // 2, 0] = 127 + 9                                  # a loud block
    if K % 128:
        sh[-1, :, (K // 32) % 4:] = 255                         # the bytes past K are nobody's
    o = binding.moe_down_w4a4(_up(hq), _up(sh), _up(q), _up(s), dev(bd), cnt, off, T, k, path=path)
    o, at = o.cpu().numpy().astype(np.float64), off.cpu().numpy()
    h = orc.mxfp4_dequantize_rows(hq, sh)
    for e in range(E):
        part = slice(at[e], at[e + 1])
        W, b = orc.mxfp4_dequantize(q[e], s[e]).T, orc.widen(bd[e])
        tol = (K / 64 + 9) * ULP * (np.abs(h[part]) @ np.abs(W) + np.abs(b))
        _within(o[part], h[part] @ W + b, tol, f"o of expert {e}")


def _values(v, s):
    """Nearest E2M1 values of float64 v under the scale bytes s."""
    unit = np.ldexp(1.0, s.astype(np.int64) - 127)
    m = np.abs(v) / unit
    step = 2.0 ** (np.floor(np.log2(np.maximum(m, 1.0))) - 1)
    return np.sign(v) * np.minimum(np.rint(m / step) * step, 6.0) * unit


def _scale(amax):
    return np.clip(np.floor(np.log2(np.maximum(amax, 2.0 ** -125))) - 2, -127, 127).astype(np.int64) + 127


def _check_h(hq, sh, want, tol, what):
    """Rows of codes and scales against float64 h within tol (see the module's docstring)."""
    got, nb = orc.mxfp4_dequantize_rows(hq, sh), want.shape[1] // 32
    s = sh.transpose(0, 2, 1).reshape(-1, hq.shape[0])[:nb].T                    # [rows][blocks]
    lo, hi = orc.bf16_round(want - tol), orc.bf16_round(want + tol)
    big = np.maximum(np.abs(lo), np.abs(hi)).reshape(-1, nb, 32).max(axis=2)
    small = np.where(np.sign(lo) == np.sign(hi), np.minimum(np.abs(lo), np.abs(hi)), 0.0).reshape(-1, nb, 32).max(axis=2)
    assert ((s >= _scale(small)) & (s <= _scale(big))).all(), f"{what}: a block scale is off"
    s = np.repeat(s, 32, axis=1)
    bad = np.argwhere((got < _values(lo, s)) | (got > _values(hi, s)))
    assert bad.size == 0, f"{what}: {len(bad)} values off, first {bad[0].tolist()}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,k,K,n32,live", STAGES)
def test_gate_up(T, E, k, K, n32, live, path):
    _need_gpu()
    I, S = 32 * n32, T * k
    q, s = _matrix(E, K, 2 * I, 5)
    bgu = d.normal_bf16((E, 2 * I), 0.5, 6, 1, E, I)
    cnt, off, rows, pos = binding.moe_permute(_up(_routing(T, E, k, 7, live)), E)
    xq, sx = _rows(T, K, 8, 60.0 / np.sqrt(K))                  # gates of deviation about 4: the clamps are reached
    if K % 128:
        sx[-1, :, (K // 32) % 4:] = 255
    hq = torch.full((S, I // 2), 0x5A, dtype=torch.uint8, device="cuda")
    sh = torch.full((-(-I // 128), S, 4), 0x5A, dtype=torch.uint8, device="cuda")
    binding.moe_gate_up_w4a4(_up(xq), _up(sx), _up(q), _up(s), dev(bgu), cnt, off, rows, k=k, hq=hq, sh=sh, path=path)
    hq, sh, at, rows = hq.cpu().numpy(), sh.cpu().numpy(), off.cpu().numpy(), rows.cpu().numpy()
    if I % 128:
        assert (sh[-1, :, (I // 32) % 4:] == 0x5A).all(), "a byte past the last block was written"
    x = orc.mxfp4_dequantize_rows(xq, sx)
    for e in range(E):
        part = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        W, b, a = orc.mxfp4_dequantize(q[e], s[e]).T, orc.widen(bgu[e]), x[rows[part] // k]
        u = (K / 64 + 9) * ULP * (np.abs(a) @ np.abs(W) + np.abs(b))
        h = orc.clamped_glu(a @ W + b)
        tol = 8.8 * u[:, 0::2] + 7.0 * u[:, 1::2] + 2.0 ** -20 * np.abs(h)
        _check_h(hq[part], sh[:, part], h, tol, f"h of expert {e}")


@pytest.mark.parametrize("path", PATHS)
def test_skipped_slots_are_left_alone(path):
    """Slots of no expert (id -1) come behind the others: their rows are neither read nor written."""
    _need_gpu()
    T, E, k, H, I = 21, 4, 2, 160, 96
    ids = _routing(T, E, k, 1)
    ids[3], ids[7, 1], ids[20, 0] = -1, -1, E
    cnt, off, rows, pos = binding.moe_permute(_up(ids), E)
    n = int(off[-1])
    assert n == T * k - 4
    q, s = _matrix(E, H, 2 * I, 2)
    xq, sx = _rows(T, H, 3)
    hq = torch.full((T * k, I // 2), 0x5A, dtype=torch.uint8, device="cuda")
    sh = torch.full((1, T * k, 4), 0xFF, dtype=torch.uint8, device="cuda")
    b = torch.zeros((E, 2 * I), dtype=torch.bfloat16, device="cuda")
    binding.moe_gate_up_w4a4(_up(xq), _up(sx), _up(q), _up(s), b, cnt, off, rows, k=k, hq=hq, sh=sh, path=path)
    assert (hq[n:] == 0x5A).all() and (sh[:, n:] == 0xFF).all() and (sh[:, :n, :3] != 0xFF).all()
    q, s = _matrix(E, I, H, 4)
    o = torch.full((T * k, H), 7.0, device="cuda")
    binding.moe_down_w4a4(hq, sh, _up(q), _up(s), torch.zeros((E, H), dtype=torch.bfloat16, device="cuda"), cnt, off, T,
                          k, o=o, path=path)
    assert (o[n:] == 7.0).all() and torch.isfinite(o).all()


@pytest.mark.parametrize("path", PATHS)
def test_extreme_scales(path):
    """Scales far apart: subnormal and huge products, a NaN block, codes of zero under a large scale."""
    _need_gpu()
    T, K, N = 20, 192, 64
    rng = np.random.default_rng(5)
    hq, q = rng.integers(0, 256, (T, K // 2), dtype=np.uint8), rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    sh, s = np.full((2, T, 4), 127, np.uint8), np.full((1, K // 32, N), 127, np.uint8)
    sh[0, 0], s[0, :, 0] = 60, 60                    # products near 2^-134
    sh[:, 1] = 0                                     # rows of 2^-127
    sh[0, 2, 1] = 250                                # overflows against the next
    s[0, 1, 5] = 250
    sh[0, 3, 2] = 255                                # NaN
    hq[4, 16:32], sh[0, 4, 1] = 0, 254               # zeros under 2^127
    s[0, 3, 9] = 255
    cnt, off, rows, pos = binding.moe_permute(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1)
    bd = torch.zeros((1, N), dtype=torch.bfloat16, device="cuda")
    o = binding.moe_down_w4a4(_up(hq), _up(sh), _up(q), _up(s), bd, cnt, off, T, 1, path=path).cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        h, W = orc.mxfp4_dequantize_rows(hq, sh), orc.mxfp4_dequantize(q[0], s[0]).T
        want, mag = h @ W, np.abs(h) @ np.abs(W)
    nan = np.isnan(want)
    assert nan[3].all() and nan[:, 9].all() and np.isnan(o[nan]).all()
    over = ~nan & (mag >= 2.0 ** 127)                # infinite, NaN or huge: outside the format's float32 sums
    fine = ~nan & ~over
    assert np.isfinite(o[fine]).all() and over.any() and fine.sum() > T * N * 0.9 - T - 2 * N
    _within(np.where(fine, o, 0), np.where(fine, want, 0), (K / 64 + 9) * ULP * np.where(fine, mag, 0) + 2.0 ** -126, "o")


# ------------------------------------------------------------------------------------------------ the block
def _block(T, E, k, H, I, seed):
    rng = np.random.default_rng([seed, T, H])
    x = d.normal_bf16((T, H), 190.85 / np.sqrt(H), seed, 1, T, H)
    Wr, br = d.normal_bf16((E, H), 0.02, seed, 2, E, H), d.normal_bf16((E,), 0.1, seed, 3, E, 1)
    def w(K, N):
        return rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8), rng.integers(119, 121, (E, K // 32, N), dtype=np.uint8)
    gu, dn = w(H, 2 * I), w(I, H)
    return x, Wr, br, *gu, d.normal_bf16((E, 2 * I), 0.01, seed, 4, E, I), *dn, d.normal_bf16((E, H), 0.01, seed, 5, E, H)


BLOCKS = [(1, 32, 4, 320, 96), (7, 8, 2, 96, 160), (64, 8, 4, 352, 224), (200, 4, 1, 288, 544), (90, 60, 8, 160, 64),
          (700, 4, 2, 544, 288), (1, 1, 1, 32, 32), (2, 4, 4, 2880, 2880), (5, 100, 4, 288, 96), (3, 64, 5, 160, 64),
          (8, 256, 8, 96, 32)]


@pytest.mark.parametrize("path", ["auto"] + PATHS)
@pytest.mark.parametrize("T,E,k,H,I", BLOCKS)
def test_forward_matches_oracle_and_stages(T, E, k, H, I, path):
    """y against the oracle; and bit for bit what the public stage calls give one after the other."""
    _need_gpu()
    args = _block(T, E, k, H, I, 11)
    ref = orc.moe_forward_w4a4(*args, k)
    g = [_up(a) for a in args]
    x, Wr, br, gq, gs, bgu, dq, ds, bd = g
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    y = binding.moe_forward_w4a4(*g, k=k, topk_ids=ids, topk_w=w, path=path)
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"])
    # a code of h on a border may fall to either side: half a step of 4 bits (1/4 of it at most) in one of I terms
    assert_y_close(host_f64(y), ref["y"])
    xq, sx = binding.moe_quantize_rows_mxfp4(x)
    cnt, off, rows, pos = binding.moe_permute(ids, E)
    stage = binding.moe_gate_up_w4a4(xq, sx, gq, gs, bgu, cnt, off, rows, k=k, path=path)
    o = binding.moe_down_w4a4(*stage, dq, ds, bd, cnt, off, T, k, path=path)
    assert (bf16_bits(binding.moe_combine(o, pos, w)) == bf16_bits(y)).all()
    # again, other bytes in the workspace
    ws = binding.alloc_workspace_w4a4(T, H, E, k, I).fill_(0xFF)
    assert (bf16_bits(binding.moe_forward_w4a4(*g, k=k, workspace=ws, path=path)) == bf16_bits(y)).all()


@pytest.mark.parametrize("path", ["auto"] + PATHS)
@pytest.mark.parametrize("T,n_valid", [(40, 0), (40, 1), (40, 29), (40, 40), (40, 99), (300, 133)])
def test_padded(T, n_valid, path):
    _need_gpu()
    E, k, H, I = 8, 2, 160, 96
    g = [_up(a) for a in _block(T, E, k, H, I, 12)]
    n = min(n_valid, T)
    counts = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    y = binding.moe_forward_padded_w4a4(*g, k=k, n_valid=torch.tensor([n_valid], dtype=torch.int32, device="cuda"),
                                        topk_ids=ids, topk_w=w, expert_counts=counts, path=path)
    assert (y[n:] == 0).all() and (ids[n:] == -1).all() and (w[n:] == 0).all() and int(counts.sum()) == n * k
    if n:
        ref = orc.moe_forward_w4a4(*_block(T, E, k, H, I, 12), k)
        assert_y_close(host_f64(y)[:n], ref["y"][:n])
    whole = binding.moe_forward_padded_w4a4(*g, k=k, path=path)
    assert (bf16_bits(whole) == bf16_bits(binding.moe_forward_w4a4(*g, k=k, path=path))).all()


@pytest.mark.parametrize("path", PATHS)
def test_ep_shares_sum_to_the_block(path):
    _need_gpu()
    T, E, k, H, I = 50, 7, 3, 224, 128
    args = _block(T, E, k, H, I, 13)
    g = [_up(a) for a in args]
    total = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for lo, hi in ((0, 1), (1, 5), (5, 7)):
        part = binding.moe_forward_ep_w4a4(*g[:3], *(t[lo:hi] for t in g[3:]), e_begin=lo, k=k, path=path)
        ref = orc.moe_forward_w4a4(*args[:3], *(a[lo:hi] for a in args[3:]), k, experts=range(lo, hi))
        assert_y_close(host_f64(part), ref["y"], f"the share of experts {lo} to {hi}")
        total += part.double()
    assert_y_close(total.cpu().numpy(), orc.moe_forward_w4a4(*args, k)["y"])


def test_nan_and_infinite_tokens_stay_their_own():
    _need_gpu()
    T, E, k, H, I = 12, 4, 2, 160, 96
    args = list(_block(T, E, k, H, I, 14))
    clean = binding.moe_forward_w4a4(*[_up(a) for a in args], k=k)
    args[0] = args[0].copy()
    args[0][3, 40], args[0][9, 0] = 0x7FC0, 0x7F80
    y = binding.moe_forward_w4a4(*[_up(a) for a in args], k=k)
    keep = [t for t in range(T) if t not in (3, 9)]
    assert torch.isnan(y[3]).all() and torch.isnan(y[9]).all()
    assert (bf16_bits(y)[keep] == bf16_bits(clean)[keep]).all()


@pytest.mark.parametrize("path", PATHS)
def test_graph_replays_match_eager(path):
    _need_gpu()
    T, E, k, H, I = 96, 8, 4, 256, 160
    g = [_up(a) for a in _block(T, E, k, H, I, 15)]
    ws, y = binding.alloc_workspace_w4a4(T, H, E, k, I), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    codes, scales = binding.moe_quantize_rows_mxfp4(g[0])
    back = torch.empty_like(g[0])

    def run():
        binding.moe_forward_w4a4(*g, k=k, y=y, workspace=ws, path=path)
        binding.moe_quantize_rows_mxfp4(g[0], codes=codes, scales=scales)
        binding.moe_dequantize_rows_mxfp4(codes, scales, out=back)
    run()
    eager = bf16_bits(y).copy(), bf16_bits(back).copy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        for t in (y, back):
            t.view(torch.int16).fill_(-1)
        codes.fill_(i), scales.fill_(255)
        ws.fill_(0xAB if i % 2 else 0x11)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (bf16_bits(y) == eager[0]).all() and (bf16_bits(back) == eager[1]).all()


def test_other_stream():
    """Calls on a stream of their own, which is not the current one, wait for nothing else and give the same."""
    _need_gpu()
    T, E, k, H, I = 33, 4, 2, 160, 96
    g = [_up(a) for a in _block(T, E, k, H, I, 16)]
    want = bf16_bits(binding.moe_forward_w4a4(*g, k=k))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = binding.moe_forward_w4a4(*g, k=k, stream=s)
    y2 = binding.moe_forward_w4a4(*g, k=k, stream=s.cuda_stream)
    codes, scales = binding.moe_quantize_rows_mxfp4(g[0], stream=s)
    back = binding.moe_dequantize_rows_mxfp4(codes, scales, stream=s)
    s.synchronize()
    assert (bf16_bits(y) == want).all() and (bf16_bits(y2) == want).all()
    assert (host_f64(back) == orc.mxfp4_dequantize_rows(*orc.mxfp4_quantize_rows(host_f64(g[0])))).all()


@pytest.mark.parametrize("T,K", [(4096, 32), (4096, 672), (1500, 352)])
def test_products_of_many_tiles(T, K):
    """So many tiles and rows that the GEMM takes its large ones (of gate_up: at the fewer tokens): ragged experts, some
    of one row, against 64 bits."""
    _need_gpu()
    E, k, N = 32, 4, 2880
    rng = np.random.default_rng(K)
    # experts of very different size: the first few take most of the tokens
    p = 1.0 / (1.0 + np.arange(E)) ** 1.5
    ids = np.argsort(rng.gumbel(size=(T, E)) + np.log(p), axis=1)[:, -k:].astype(np.int32)
    ids[ids == E - 1] = -1
    ids[5, 0] = E - 1                                          # one row
    cnt, off, rows, pos = binding.moe_permute(_up(ids), E)
    at, rows_h = off.cpu().numpy(), rows.cpu().numpy()
    q, s = _matrix(E, K, N, 9)
    b = d.normal_bf16((E, N), 0.5, 9, 1, E, N)
    W = [torch.from_numpy(orc.mxfp4_dequantize(q[e], s[e]).T.copy()).cuda() for e in range(E)]
    bias = torch.from_numpy(orc.widen(b)).cuda()
    hq, sh = binding.moe_quantize_rows_mxfp4(torch.randn((T * k, K), device="cuda").bfloat16() * 3)
    o = binding.moe_down_w4a4(hq, sh, _up(q), _up(s), dev(b), cnt, off, T, k, path="gemm").double()
    h = torch.from_numpy(orc.mxfp4_dequantize_rows(hq.cpu().numpy(), sh.cpu().numpy())).cuda()
    for e in range(E):
        part = slice(int(at[e]), int(at[e + 1]))
        tol = (K / 64 + 9) * ULP * (h[part].abs() @ W[e].abs() + bias[e].abs())
        assert bool(((o[part] - (h[part] @ W[e] + bias[e])).abs() <= tol).all()), f"o of expert {e}"
    xq, sx = binding.moe_quantize_rows_mxfp4(torch.randn((T, K), device="cuda").bfloat16() * float(60.0 / np.sqrt(K)))
    gq, gs = binding.moe_gate_up_w4a4(xq, sx, _up(q), _up(s), dev(b), cnt, off, rows, k=k, path="gemm")
    gq, gs = gq.cpu().numpy(), gs.cpu().numpy()
    x = torch.from_numpy(orc.mxfp4_dequantize_rows(xq.cpu().numpy(), sx.cpu().numpy())).cuda()
    for e in list(range(0, E, 5)) + [E - 1]:
        part = slice(int(at[e]), int(at[e + 1]))
        a = x[torch.from_numpy(rows_h[part] // k).cuda().long()]
        u = ((K / 64 + 9) * ULP * (a.abs() @ W[e].abs() + bias[e].abs())).cpu().numpy()
        want = orc.clamped_glu((a @ W[e] + bias[e]).cpu().numpy())
        tol = 8.8 * u[:, 0::2] + 7.0 * u[:, 1::2] + 2.0 ** -20 * np.abs(want)
        _check_h(gq[part], gs[:, part], want, tol, f"h of expert {e}")


@pytest.mark.parametrize("path", PATHS)
def test_outputs_past_four_gib(path):
    """Rows of o that lie beyond 2^32 bytes."""
    _need_gpu()
    S, K, N = 400000, 64, 2880
    q, s = _matrix(1, K, N, 10)
    bd = d.normal_bf16((1, N), 0.5, 10, 1, 1, N)
    hq, sh = binding.moe_quantize_rows_mxfp4(torch.randn((S, K), device="cuda").bfloat16())
    cnt, off, rows, pos = binding.moe_permute(torch.zeros((S, 1), dtype=torch.int32, device="cuda"), 1)
    o = binding.moe_down_w4a4(hq, sh, _up(q), _up(s), dev(bd), cnt, off, S, 1, path=path)
    pick = np.r_[0:3, 372820:372840, S - 70:S]
    h = orc.mxfp4_dequantize_rows(hq.cpu().numpy()[pick], sh.cpu().numpy()[:, pick])
    W, b = orc.mxfp4_dequantize(q[0], s[0]).T, orc.widen(bd[0])
    got = o[torch.from_numpy(pick).cuda()].cpu().numpy().astype(np.float64)
    _within(got, h @ W + b, (K / 64 + 9) * ULP * (np.abs(h) @ np.abs(W) + np.abs(b)), "o")


@pytest.mark.parametrize("path", PATHS)
def test_two_calls_at_once(path):
    """Two streams, each with its own workspace, in turn without a wait between them."""
    _need_gpu()
    E, k, H, I = 8, 4, 352, 224
    sets = [[_up(a) for a in _block(T, E, k, H, I, 17)] for T in (64, 301)]
    want = [bf16_bits(binding.moe_forward_w4a4(*g, k=k, path=path)) for g in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [binding.alloc_workspace_w4a4(g[0].shape[0], H, E, k, I) for g in sets]
    torch.cuda.synchronize()
    ys = [[binding.moe_forward_w4a4(*g, k=k, workspace=w, path=path, stream=s)
           for g, w, s in zip(sets, spaces, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in ys:
        for y, bits in zip(pair, want):
            assert (bf16_bits(y) == bits).all()


def test_same_expert_twice_in_a_row():
    """Stage calls with an expert that a token names twice: two slots, two rows of h and of o."""
    _need_gpu()
    T, E, k, H, I = 40, 4, 3, 160, 96
    ids = _routing(T, E, k, 18)
    ids[:, 2] = ids[:, 0]
    cnt, off, rows, pos = binding.moe_permute(_up(ids), E)
    gq, gs = _matrix(E, H, 2 * I, 19)
    dq, ds = _matrix(E, I, H, 20)
    z = torch.zeros((E, 2 * I), dtype=torch.bfloat16, device="cuda"), torch.zeros((E, H), dtype=torch.bfloat16, device="cuda")
    xq, sx = _rows(T, H, 21)
    for path in PATHS:
        hq, sh = binding.moe_gate_up_w4a4(_up(xq), _up(sx), _up(gq), _up(gs), z[0], cnt, off, rows, k=k, path=path)
        o = binding.moe_down_w4a4(hq, sh, _up(dq), _up(ds), z[1], cnt, off, T, k, path=path)
        at = pos.view(T, k).long()
        assert (hq[at[:, 0]] == hq[at[:, 2]]).all() and (o[at[:, 0]] == o[at[:, 2]]).all()
        assert (at[:, 0] != at[:, 2]).all()


def test_graph_replays_of_few_tokens():
    """One workgroup column a slot: captured, and replayed over other bytes in the workspace."""
    _need_gpu()
    T, E, k, H, I = 2, 40, 4, 288, 96
    g = [_up(a) for a in _block(T, E, k, H, I, 22)]
    ws, y = binding.alloc_workspace_w4a4(T, H, E, k, I), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    binding.moe_forward_w4a4(*g, k=k, y=y, workspace=ws)
    eager = bf16_bits(y).copy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        binding.moe_forward_w4a4(*g, k=k, y=y, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_forward_w4a4(*g, k=k, y=y, workspace=ws)
    for i in range(4):
        y.view(torch.int16).fill_(-1)
        ws.fill_(0xAB if i % 2 else 0x11)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (bf16_bits(y) == eager).all()


@pytest.mark.parametrize("T", [1, 40, 600])
def test_ep_rank_of_many(T):
    """One rank of eight by itself, at sizes that take different variants, against the oracle."""
    _need_gpu()
    E, k, H, I = 32, 4, 160, 96
    args = _block(T, E, k, H, I, 23)
    g = [_up(a) for a in args]
    for lo in (0, 28):
        part = binding.moe_forward_ep_w4a4(*g[:3], *(t[lo:lo + 4].contiguous() for t in g[3:]), e_begin=lo, k=k)
        ref = orc.moe_forward_w4a4(*args[:3], *(a[lo:lo + 4] for a in args[3:]), k, experts=range(lo, lo + 4))
        assert_y_close(host_f64(part), ref["y"], f"the share of experts from {lo}")


@pytest.mark.parametrize("K", [64, 352])
def test_products_of_many_experts(K):
    """Many tiles of few rows each (the GEMM's tiles of 128 x 256): against 64 bits."""
    _need_gpu()
    T, E, k, N = 900, 150, 4, 2880
    ids = _routing(T, E, k, 24, 140)
    cnt, off, rows, pos = binding.moe_permute(_up(ids), E)
    at, rows_h = off.cpu().numpy(), rows.cpu().numpy()
    q, s = _matrix(E, K, N, 25)
    b = d.normal_bf16((E, N), 0.5, 25, 1, E, N)
    hq, sh = binding.moe_quantize_rows_mxfp4(torch.randn((T * k, K), device="cuda").bfloat16() * 3)
    o = binding.moe_down_w4a4(hq, sh, _up(q), _up(s), dev(b), cnt, off, T, k, path="gemm").cpu().numpy().astype(np.float64)
    h = orc.mxfp4_dequantize_rows(hq.cpu().numpy(), sh.cpu().numpy())
    xq, sx = binding.moe_quantize_rows_mxfp4(torch.randn((T, K), device="cuda").bfloat16() * float(60.0 / np.sqrt(K)))
    gq, gs = binding.moe_gate_up_w4a4(xq, sx, _up(q), _up(s), dev(b), cnt, off, rows, k=k, path="gemm")
    gq, gs, x = gq.cpu().numpy(), gs.cpu().numpy(), orc.mxfp4_dequantize_rows(xq.cpu().numpy(), sx.cpu().numpy())
    for e in range(0, 140, 9):
        part = slice(at[e], at[e + 1])
        W, bias = orc.mxfp4_dequantize(q[e], s[e]).T, orc.widen(b[e])
        tol = (K / 64 + 9) * ULP * (np.abs(h[part]) @ np.abs(W) + np.abs(bias))
        _within(o[part], h[part] @ W + bias, tol, f"o of expert {e}")
        a = x[rows_h[part] // k]
        u = (K / 64 + 9) * ULP * (np.abs(a) @ np.abs(W) + np.abs(bias))
        want = orc.clamped_glu(a @ W + bias)
        _check_h(gq[part], gs[:, part], want, 8.8 * u[:, 0::2] + 7.0 * u[:, 1::2] + 2.0 ** -20 * np.abs(want), f"h of expert {e}")
