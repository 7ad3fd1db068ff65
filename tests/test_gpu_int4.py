"""Expert products with 4-bit integer weights and group scales against the
float64 oracle (needs an MI355X).  Every call goes through the C ABI.

Tolerance of a product (before bias and GLU), derived: the integers, zero
points and bf16 activations are exact operands, so the errors are float32
accumulation, in two places.
 - Inside a group of G values, sums whose terms are at most
   |a| (16 + q) + |a| (16 + z) in total (the operands are 16 + q, and
   (16 + z) times the sum of a is taken off).  One v_mfma_f32_16x16x32 step
   accumulates within 128 / 90 u of the sum of its terms' magnitudes (the
   bound the MFMA router rests on, which tests/test_gpu_router_bound.py
   measures), u = 2^-24; a group is at most 4 steps and as many for the sum
   of a, and its parts meet in at most 4 more operations: 16 u.
 - Over groups: at most ceil(K/G) + 8 float32 operations on partial sums that
   the sum of |a w| bounds, each off by u.
A GLU with gate <= 7 and |up + 1| <= 8 has slopes of at most 8.8 in gate (1.1,
the largest slope of g sigmoid(1.702 g), times 8) and 7 in up; the hardware
exponential and reciprocal are within 2^-20 of h; h is rounded to bf16, half a
step of which is 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_nan_rows, assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PATHS = ["gemv", "gemm"]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if a.dtype != np.uint16 else dev(a)


def _matrix(E, K, N, G, zeros, seed):
    """Plain codes [E][K][N], scales (bf16 bits) and zero points; a few groups with scale 0 and codes at the ends."""
    rng = np.random.default_rng([seed, E, K, N, G])
    ng = -(-K // G)
    q = rng.integers(0, 16, (E, K, N), dtype=np.uint8)
    q[:, :, 0], q[:, :, 1] = 15, 0
    s = d.f32_to_bf16_bits((0.02 / 4.6 * 2.0 ** rng.uniform(-1, 1, (E, ng, N))).astype(np.float32))
    s[:, -1, 2] = 0
    z = rng.integers(0, 16, (E, ng, N), dtype=np.uint8) if zeros else None
    return q, s, z


def _gpu(m):
    q, s, z = m
    return torch.from_numpy(orc.int4_pack(q)).cuda(), dev(s), None if z is None else torch.from_numpy(z).cuda()


def _bound(a, m, e, G):
    """Error bound of a @ W[e] as derived above, and the exact product."""
    q, s, z = m
    W = orc.int4_dequantize(q[e], s[e], None if z is None else z[e], G)
    group = np.arange(q.shape[1]) // G
    big = (32.0 + q[e] + (8.0 if z is None else z[e].astype(np.float64)[group])) * np.abs(orc.widen(s[e]))[group]
    return a @ W, 16 * U * (np.abs(a) @ big) + (len(s[e]) + 8) * U * (np.abs(a) @ np.abs(W))


def _assert_within(got, want, tol, what):
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} off, first {bad[0].tolist()}: {got[tuple(bad[0])]} for "
                           f"{want[tuple(bad[0])]} +- {tol[tuple(bad[0])]}")


def _routing(T, E, k, seed, live=None):
    """ids [T][k], all different in a row, among the first `live` experts."""
    rng = np.random.default_rng([seed, T, E])
    return np.stack([rng.permutation(live or E)[:k] for _ in range(T)]).astype(np.int32)


# T, E, k, K (H or I), columns (2I or H), live experts
STAGES = [
    (1, 4, 1, 32, 16, None),       # one token, one tile of K, a quarter of a tile of columns
    (3, 8, 2, 96, 80, None),       # three tiles of K: a ragged group of 64, a lone one of 128
    (16, 2, 1, 160, 64, None),     # about eight rows an expert
    (17, 1, 1, 288, 128, None),    # 17 rows: one past a 16-row operand
    (33, 3, 2, 2880, 72, 2),       # full K, 33 rows: a third chunk; an expert without rows
    (100, 4, 2, 352, 208, None),   # 50 rows an expert
    (70, 2, 2, 64, 2880, None),    # full width, 70 rows
    (300, 1, 1, 128, 96, None),    # 300 rows of one expert
    (40, 40, 8, 224, 136, 30),     # many experts, k = 8
    (129, 5, 4, 1440, 144, None),  # 103 rows an expert, K = 11.25 groups of 128
]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,K,N,live", STAGES)
def test_down(T, E, k, K, N, live, G, zeros, path):
    _need_gpu()
    m = _matrix(E, K, N, G, zeros, 1)
    q, s, z = _gpu(m)
    bd = d.normal_bf16((E, N), 0.5, 2, 1, E, N)
    ids = _routing(T, E, k, 3, live)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    h = d.normal_bf16((T * k, K), 3.0, 4, 1, T, K)
    o = torch.full((T * k, N), float("nan"), device="cuda")
    binding.moe_down_int4(dev(h), q, s, dev(bd), cnt, off, T, k, Wd_z=z, o=o, path=path)
    got, off = host_f64(o), off.cpu().numpy()
    for e in range(E):
        a = orc.widen(h[off[e]:off[e + 1]])
        want, tol = _bound(a, m, e, G)
        b = orc.widen(bd[e])
        _assert_within(got[off[e]:off[e + 1]], want + b, tol + U * np.abs(want + b), f"expert {e}")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,K,N,live", STAGES)
def test_gate_up(T, E, k, K, N, live, G, zeros, path):
    _need_gpu()
    N = -(-N // 16) * 16                                              # I % 8 == 0
    m = _matrix(E, K, N, G, zeros, 5)
    q, s, z = _gpu(m)
    bgu = d.normal_bf16((E, N), 0.5, 6, 1, E, N)
    ids = _routing(T, E, k, 7, live)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    x = d.normal_bf16((T, K), 60.0 / np.sqrt(K) / 0.3, 8, 1, T, K)   # some gates and ups reach the clamps
    h = torch.full((T * k, N // 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.moe_gate_up_int4(dev(x), q, s, dev(bgu), cnt, off, rows, k, Wgu_z=z, h=h, path=path)
    got, off, rows = host_f64(h), off.cpu().numpy(), rows.cpu().numpy()
    for e in range(E):
        a = orc.widen(x[rows[off[e]:off[e + 1]] // k])
        u, tol = _bound(a, m, e, G)
        u = u + orc.widen(bgu[e])
        tol = tol + U * np.abs(u)
        want = orc.clamped_glu(u)
        _assert_within(got[off[e]:off[e + 1]], want,
                       (8.8 * tol[:, 0::2] + 7 * tol[:, 1::2]) * (1 + 2.0 ** -8) + np.abs(want) * (2.0 ** -8 + 2.0 ** -20)
                       + 2.0 ** -134, f"expert {e}")


@pytest.mark.parametrize("G,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("counts", [
    (0, 1, 63, 64, 65, 127, 128, 129, 1100), (1,) * 256, (0,) * 255 + (300,), (16, 17, 31, 33, 80, 81, 96, 97, 112, 113),
    (1300, 1290, 0, 5)])
def test_gemm_takes_every_tile(counts, G, zeros):
    """Long and short last M tiles, whole and cut N tiles, in every mix; each row of every expert is written once."""
    _need_gpu()
    E, T, K, N = len(counts), sum(counts), 96, 1160 if len(counts) < 16 else 584
    m = _matrix(E, K, N, G, zeros, 35)
    q, s, z = _gpu(m)
    ids = np.random.default_rng(36).permutation(np.repeat(np.arange(E, dtype=np.int32), counts)).reshape(T, 1)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    h = d.normal_bf16((T, K), 3.0, 37, 1, T, K)
    bd = d.normal_bf16((E, N), 0.5, 38, 1, E, N)
    o = torch.full((T, N), float("nan"), device="cuda")
    binding.moe_down_int4(dev(h), q, s, dev(bd), cnt, off, T, 1, Wd_z=z, o=o, path="gemm")
    got, off = host_f64(o), off.cpu().numpy()
    for e in range(E):
        if counts[e]:
            want, tol = _bound(orc.widen(h[off[e]:off[e + 1]]), m, e, G)
            b = orc.widen(bd[e])
            _assert_within(got[off[e]:off[e + 1]], want + b, tol + U * np.abs(want + b), f"expert {e}")


# 48 experts x 10 column tiles of 256: more small tiles than the card runs at once, so the large ones (128 x 512) run.
LARGE = (0, 1, 15, 16, 17, 33, 63, 64, 65, 80, 96, 97, 112, 127, 128, 129, 145, 191, 192, 193, 255, 256, 257, 300) * 2


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K", [32, 160, 288])
def test_gemm_large_tiles(K, zeros, G):
    """Both products, every count of 16-row chunks, first and last rounds, one to nine tiles of K."""
    _need_gpu()
    E, T, N = len(LARGE), sum(LARGE), 2320
    m = _matrix(E, K, N, G, zeros, 39)
    q, s, z = _gpu(m)
    ids = np.random.default_rng(40).permutation(np.repeat(np.arange(E, dtype=np.int32), LARGE)).reshape(T, 1)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    x = d.normal_bf16((T, K), 60.0 / np.sqrt(K) / 0.3, 41, 1, T, K)
    b = d.normal_bf16((E, N), 0.5, 42, 1, E, N)
    o = torch.full((T, N), float("nan"), device="cuda")
    h = torch.full((T, N // 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.moe_down_int4(dev(x), q, s, dev(b), cnt, off, T, 1, Wd_z=z, o=o, path="gemm")
    binding.moe_gate_up_int4(dev(x), q, s, dev(b), cnt, off, rows, 1, Wgu_z=z, h=h, path="gemm")
    o, h, off, rows = host_f64(o), host_f64(h), off.cpu().numpy(), rows.cpu().numpy()
    for e in range(E):
        if LARGE[e]:
            r = slice(off[e], off[e + 1])
            bias = orc.widen(b[e])
            want, tol = _bound(orc.widen(x[r]), m, e, G)
            _assert_within(o[r], want + bias, tol + U * np.abs(want + bias), f"down, expert {e}")
            u, tol = _bound(orc.widen(x[rows[r]]), m, e, G)
            u = u + bias
            tol = tol + U * np.abs(u)
            want = orc.clamped_glu(u)
            _assert_within(h[r], want, (8.8 * tol[:, 0::2] + 7 * tol[:, 1::2]) * (1 + 2.0 ** -8)
                           + np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -134, f"gate_up, expert {e}")


@pytest.mark.parametrize("T,E,k,N,G,path", [
    (64, 2, 1, 64, 64, "gemv"), (65, 2, 1, 64, 64, "gemv"), (256, 2, 1, 64, 32, "gemv"), (257, 2, 1, 64, 32, "gemm"),
    (1023, 8, 1, 2048, 64, "gemv"), (1024, 8, 1, 2048, 64, "gemm"), (1024, 8, 1, 2048, 32, "gemv"),
    (1536, 12, 1, 2048, 32, "gemm"), (1024, 32, 1, 4096, 64, "gemv"), (1025, 32, 1, 4096, 64, "gemm")])
def test_auto_takes_the_documented_path(T, E, k, N, G, path):
    """The paths are told apart by their bits: streaming sums four parts of K, the GEMM goes through K in one sequence
    (at K = 64, one part, they are equal)."""
    _need_gpu()
    K = 1024
    q, s, z = _gpu(_matrix(E, K, N, G, True, 43))
    ids = _routing(T, E, k, 44)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    h, b = dev(d.normal_bf16((T * k, K), 3.0, 45, 1, T, K)), dev(d.normal_bf16((E, N), 0.5, 46, 1, E, N))
    got = {p: binding.moe_down_int4(h, q, s, b, cnt, off, T, k, Wd_z=z, path=p) for p in ("auto", "gemv", "gemm")}
    assert not torch.equal(got["gemv"], got["gemm"]) and torch.equal(got["auto"], got[path])


def _block(T, E, H, I, k, G, zeros, seed=0, router_bias="normal"):
    cfg = d.small_config(T=T, E=E, H=H, I=I, k=k, x_scale=d.scale_for_hidden(H), router_bias=router_bias)
    x = d.make_activations(cfg, seed)
    Wr, br = d.make_router(cfg, seed)
    gu, down = _matrix(E, H, 2 * I, G, zeros, seed + 1), _matrix(E, I, H, G, zeros, seed + 2)
    bgu, bd = d.normal_bf16((E, 2 * I), 0.01, seed, 5, E, I), d.normal_bf16((E, H), 0.01, seed, 7, E, H)
    return x, Wr, br, gu, bgu, down, bd


def _gpu_args(b):
    x, Wr, br, gu, bgu, down, bd = b
    gq, gs, gz = _gpu(gu)
    dq, ds, dz = _gpu(down)
    return (dev(x), dev(Wr), dev(br), gq, gs, dev(bgu), dq, ds, dev(bd)), {"Wgu_z": gz, "Wd_z": dz}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,H,I,k,G,zeros", [
    (1, 4, 32, 32, 1, 32, False), (5, 8, 64, 96, 2, 64, True), (33, 8, 96, 64, 4, 128, False),
    (200, 16, 256, 160, 4, 32, True), (17, 8, 2880, 2880, 4, 128, True), (300, 4, 160, 608, 4, 64, False),
    (60, 256, 128, 96, 8, 64, True), (257, 4, 1440, 2880, 2, 32, False)])
def test_forward(T, E, H, I, k, G, zeros, path):
    _need_gpu()
    b = _block(T, E, H, I, k, G, zeros, seed=T)
    args, z = _gpu_args(b)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), dtype=torch.float32, device="cuda")
    y = binding.moe_forward_int4(*args, k=k, topk_ids=ids, topk_w=w, path=path, **z)
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"], f"y T{T} E{E}")


# Up to a quarter as many slots as experts run one by one, more of them in groups; a padded batch without padding
# always runs in groups.
@pytest.mark.parametrize("T,E,H,I,k,G,zeros", [
    (1, 4, 32, 32, 1, 32, True), (1, 32, 2880, 2880, 4, 32, False), (2, 32, 96, 160, 4, 64, True),
    (3, 32, 96, 160, 4, 64, True), (4, 64, 1440, 96, 4, 128, False), (5, 128, 608, 2880, 3, 128, True),
    (8, 256, 256, 64, 8, 32, True), (64, 256, 64, 96, 1, 64, False), (1, 256, 32, 32, 1, 32, False),
    (1, 20, 32, 5760, 5, 64, True)])
def test_few_slots(T, E, H, I, k, G, zeros):
    """The decision is the groups' (weights within one float step of each other), and so are the rows."""
    _need_gpu()
    b = _block(T, E, H, I, k, G, zeros, seed=T + E)
    args, z = _gpu_args(b)
    out = []
    for call in (binding.moe_forward_int4, binding.moe_forward_padded_int4):
        ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), -1.0, dtype=torch.float32, device="cuda")
        out.append((call(*args, k=k, topk_ids=ids, topk_w=w, **z), ids, w))
    (y, ids, w), (y2, ids2, w2) = out
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"], f"y T{T} E{E}")
    assert torch.equal(ids, ids2)
    torch.testing.assert_close(w, w2, rtol=2 ** -23, atol=0)
    if torch.equal(w, w2):
        assert torch.equal(y, y2)
    assert torch.equal(binding.moe_forward_int4(*args, k=k, **z), y)   # and with ids and weights in the workspace


def test_few_slots_ties():
    """Equal logits go to the lower index, -0 and 0 are equal, and NaN logits still pick k experts."""
    _need_gpu()
    T, E, H, I, k, G = 2, 64, 64, 64, 8, 64
    b = list(_block(T, E, H, I, k, G, False, seed=3))
    b[1][:] = b[1][0]
    b[2][:] = 0
    args, z = _gpu_args(tuple(b))
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), dtype=torch.float32, device="cuda")
    binding.moe_forward_int4(*args, k=k, topk_ids=ids, topk_w=w, **z)
    assert ids.tolist() == [list(range(k))] * T and (w == 1 / k).all()
    x = args[0].clone()
    x[0] = 0
    x[1, 5] = float("nan")
    args[1][:, 0] = -args[1][:, 0]
    y = binding.moe_forward_int4(x, *args[1:], k=k, topk_ids=ids, topk_w=w, **z)
    assert ids[0].tolist() == list(range(k)) and torch.isfinite(y[0]).all()
    assert len(set(ids[1].tolist())) == k and 0 <= ids[1].min() and ids[1].max() < E and torch.isnan(y[1]).all()


def test_few_slots_of_a_rank_with_every_expert():
    _need_gpu()
    T, E, H, I, k, G = 3, 64, 128, 96, 4, 32
    args, z = _gpu_args(_block(T, E, H, I, k, G, True, seed=29))
    y = binding.moe_forward_int4(*args, k=k, **z)
    part = binding.moe_forward_ep_int4(*args, 0, k=k, Wgu_z_local=z["Wgu_z"], Wd_z_local=z["Wd_z"])
    assert torch.equal(part.to(torch.bfloat16), y)


@pytest.mark.parametrize("T", [1, 40])
def test_infinity_in_a_row_of_h_gives_nan_there(T):
    _need_gpu()
    E, H, I, k, G = 16, 64, 128, 1, 64
    args, z = _gpu_args(_block(T, E, H, I, k, G, True, seed=31))
    h = dev(d.normal_bf16((T, I), 1.0, 33, 1, T, I))
    h[T // 2, 3] = float("inf")
    cnt = torch.zeros(E, dtype=torch.int32, device="cuda")
    cnt[5] = T
    off = torch.cat([cnt.new_zeros(1), cnt.cumsum(0).to(torch.int32)])
    o = binding.moe_down_int4(h, args[6], args[7], args[8], cnt, off, T, k, Wd_z=z["Wd_z"])
    bad = torch.arange(T, device="cuda") == T // 2
    assert torch.isnan(o[bad]).all() and torch.isfinite(o[~bad]).all()


def test_few_slots_graph_replays():
    """Two captured calls that share a workspace, replayed in turn with eager calls between."""
    _need_gpu()
    T, E, H, I, k, G = 2, 64, 256, 160, 4, 64
    args, z = _gpu_args(_block(T, E, H, I, k, G, True, seed=23))
    xs = (args[0], args[0].flip(0).contiguous())
    ws = binding.alloc_workspace(T, H, E, k, I)
    ys = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [binding.moe_forward_int4(x, *args[1:], k=k, **z) for x in xs]
    torch.cuda.synchronize()
    graphs = []
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.moe_forward_int4(x, *args[1:], k=k, y=y, workspace=ws, **z)
        graphs.append(g)
    for i in range(3):
        for y in ys:
            y.fill_(-1.0)
        ws.fill_(0xFF if i % 2 else 0x11)
        eager = binding.moe_forward_int4(xs[1], *args[1:], k=k, **z)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, want[1])
        assert all(torch.equal(y, w) for y, w in zip(ys, want)), i


@pytest.mark.parametrize("E,K,N,G", [(2, 96, 40, 64), (1, 2880, 72, 128), (3, 32, 8, 32), (1, 160, 200, 32), (2, 128, 64, 64)])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantizer_matches_oracle(E, K, N, G, zeros):
    """Codes, scales and zero points bit for bit; columns of zeros, of one sign, of exact halves, tiny and huge."""
    _need_gpu()
    W = d.normal_bf16((E, K, N), 0.02, 9, 1, K, N)
    W[:, :, 0] = 0
    W[:, :, 1] &= 0x7FFF
    W[:, :, 2] |= 0x8000
    W[:, :, 3] = d.f32_to_bf16_bits((np.arange(K) % 15 * 0.5 - 3.5).astype(np.float32))
    W[:, :, 4] = np.arange(K) % 100                                   # subnormals
    W[:, :, 5] = d.f32_to_bf16_bits(np.where(np.arange(K) % 2, 3e38, -3e38).astype(np.float32))
    q, s, z = binding.moe_quantize_int4(dev(W), G=G, zeros=zeros)
    q_ref, s_ref, z_ref = orc.int4_quantize(W, G, zeros)
    assert (bf16_bits(s) == s_ref).all(), np.argwhere(bf16_bits(s) != s_ref)[:5].tolist()
    assert (z is None) == (z_ref is None) and (z is None or (z.cpu().numpy() == z_ref).all())
    want = orc.int4_pack(q_ref)
    assert (q.cpu().numpy() == want).all(), np.argwhere(q.cpu().numpy() != want)[:5].tolist()


@pytest.mark.parametrize("E,K,N", [(2, 96, 40), (1, 32, 64), (3, 224, 136)])
def test_pack_matches_oracle(E, K, N):
    _need_gpu()
    q = np.random.default_rng(10).integers(0, 16, (E, K, N), dtype=np.uint8)
    kn = np.swapaxes(q, 1, 2)
    got = binding.moe_pack_int4(torch.from_numpy(np.ascontiguousarray(kn[:, :, 0::2] | (kn[:, :, 1::2] << 4))).cuda())
    assert (got.cpu().numpy() == orc.int4_pack(q)).all()


@pytest.mark.parametrize("path", PATHS)
def test_columns_past_the_width_are_ignored(path):
    """Whatever the codes of a tile's columns past N hold, the results are the same bits."""
    _need_gpu()
    T, E, H, I, k, G = 40, 4, 96, 64, 2, 64
    b = _block(T, E, H, I, k, G, True, seed=11)
    args, z = _gpu_args(b)
    ref = binding.moe_forward_int4(*args, k=k, path=path, **z)
    dq = args[6].clone()                                               # down: N = 96, the second tile half used
    v = dq.view(E, 2, I // 32, 64, 4, 4)
    v[:, 1].view(E, I // 32, 4, 16, 16)[:, :, :, 8:] = 0xFF            # lanes c = 8..15 of the last tile: columns 96..127
    y = binding.moe_forward_int4(*args[:6], dq, *args[7:], k=k, path=path, **z)
    assert torch.equal(ref, y)


@pytest.mark.parametrize("path", PATHS)
def test_nan_stays_in_its_rows(path):
    """A token with NaN or infinite values spoils its own rows alone: every other row keeps its bits."""
    _need_gpu()
    T, E, H, I, k, G = 50, 4, 160, 96, 2, 64
    b = _block(T, E, H, I, k, G, False, seed=12)
    ids = _routing(T, E, k, 13)
    args, z = _gpu_args(b)
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(ids).cuda(), E)
    x = args[0].clone()
    h0 = binding.moe_gate_up_int4(x, args[3], args[4], args[5], cnt, off, rows, k, path=path)
    x[7, 3], x[31, 150], x[49, 0] = float("nan"), float("inf"), float("-inf")
    h1 = binding.moe_gate_up_int4(x, args[3], args[4], args[5], cnt, off, rows, k, path=path)
    tok = rows.cpu().numpy() // k
    clean = ~np.isin(tok, (7, 31, 49))
    assert (bf16_bits(h0)[clean] == bf16_bits(h1)[clean]).all()
    assert np.isnan(host_f64(h1)[tok == 7]).all()
    o0 = binding.moe_down_int4(h0, args[6], args[7], args[8], cnt, off, T, k, path=path)
    o1 = binding.moe_down_int4(h1, args[6], args[7], args[8], cnt, off, T, k, path=path)
    assert torch.equal(o0[torch.from_numpy(clean).cuda()], o1[torch.from_numpy(clean).cuda()])


@pytest.mark.parametrize("path", PATHS)
def test_nan_scale(path):
    """A NaN scale makes its column NaN, for its expert's rows alone."""
    _need_gpu()
    T, E, H, I, k, G = 30, 4, 96, 64, 2, 32
    x, Wr, br, gu, bgu, down, bd = _block(T, E, H, I, k, G, False, seed=14)
    down[1][2, 1, 17] = 0x7FC0
    b = (x, Wr, br, gu, bgu, down, bd)
    args, z = _gpu_args(b)
    y = binding.moe_forward_int4(*args, k=k, path=path, **z)
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    got, want = np.isnan(host_f64(y)), np.isnan(ref["y"])
    assert want.any() and not want.all() and (got == want).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("n", [0, 1, 37, 64, 90])
def test_padded(n, path):
    _need_gpu()
    T, E, H, I, k, G = 64, 8, 96, 64, 2, 32
    b = _block(T, E, H, I, k, G, True, seed=15)
    args, z = _gpu_args(b)
    counts = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    y = binding.moe_forward_padded_int4(*args, k=k, n_valid=torch.tensor([n], dtype=torch.int32, device="cuda"),
                                        expert_counts=counts, topk_ids=ids, path=path, **z)
    m = min(n, T)
    assert (host_f64(y)[m:] == 0).all() and (ids[m:] == -1).all()
    if m:
        ref = orc.moe_forward_int4(b[0][:m], *b[1:], k=k, G=G)
        assert_y_close(host_f64(y)[:m], ref["y"])
        assert (counts.cpu().numpy() == orc.expert_loads(ref["ids"], E)).all()
    else:
        assert (counts == 0).all()


# Up to 64 tokens the router and the permutation take two launches of their own.
@pytest.mark.parametrize("T,E,k,n,ranks", [
    (2, 4, 1, 1, 2), (3, 5, 4, 3, 1), (4, 8, 8, 2, 3), (5, 64, 8, 0, 4), (7, 65, 3, 7, 2), (33, 32, 4, 20, 4),
    (63, 128, 5, 62, 5), (64, 256, 8, 64, 3), (64, 3, 2, 50, 3), (65, 16, 4, 64, 2)])
def test_few_tokens_route_and_permute(T, E, k, n, ranks):
    """Ids, weights, loads and rows of padded batches and of expert-parallel ranks, against the router's own call."""
    _need_gpu()
    H, I, G = 256, 64, 64
    b = _block(T, E, H, I, k, G, False, seed=T * E)
    args, z = _gpu_args(b)
    want_ids, want_w = binding.moe_route(*args[:3], k, method="exact")
    ids, w = torch.full_like(want_ids, -7), torch.full_like(want_w, -7.0)
    counts = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    valid = torch.tensor([n], dtype=torch.int32, device="cuda")
    y = binding.moe_forward_padded_int4(*args, k=k, n_valid=valid, expert_counts=counts, topk_ids=ids, topk_w=w, **z)
    assert torch.equal(ids[:n], want_ids[:n]) and (ids[n:] == -1).all()
    torch.testing.assert_close(w[:n], want_w[:n], rtol=2 ** -23, atol=0)
    assert (w[n:] == 0).all() and (y[n:] == 0).all()
    assert counts.tolist() == np.bincount(want_ids[:n].cpu().numpy().ravel(), minlength=E).tolist()
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    if n:
        assert_y_close(host_f64(y)[:n], ref["y"][:n])
    cuts = np.linspace(0, E, ranks + 1).astype(int)
    parts = []
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        c = slice(int(lo), int(hi))
        parts.append(binding.moe_forward_ep_int4(*args[:3], *[a[c].contiguous() for a in args[3:]], int(lo), k=k))
    assert_y_close(sum(p.double() for p in parts).to(torch.bfloat16).double().cpu().numpy(), ref["y"])


@pytest.mark.parametrize("path", PATHS)
def test_expert_parallel_ranks_sum_to_the_whole(path):
    _need_gpu()
    T, E, H, I, k, G = 70, 8, 96, 64, 4, 64
    b = _block(T, E, H, I, k, G, True, seed=16)
    (x, Wr, br, gq, gs, bgu, dq, ds, bd), z = _gpu_args(b)
    total = torch.zeros((T, H), device="cuda")
    for lo, n in ((0, 3), (3, 1), (4, 4)):
        c = slice(lo, lo + n)
        part = binding.moe_forward_ep_int4(x, Wr, br, gq[c], gs[c], bgu[c], dq[c], ds[c], bd[c], e_begin=lo, k=k,
                                           Wgu_z_local=z["Wgu_z"][c], Wd_z_local=z["Wd_z"][c], path=path)
        ref = orc.moe_forward_int4(*b, k=k, G=G, experts=(lo, lo + n))
        assert_y_close(host_f64(part), ref["y"], f"experts {lo}..{lo + n - 1}")
        total += part
    assert_y_close(host_f64(total), orc.moe_forward_int4(*b, k=k, G=G)["y"])


def test_norm_then_int4_block():
    """A decode step as served: norm with the residual's addition, then the block on its rows."""
    _need_gpu()
    T, E, H, I, k, G = 9, 8, 288, 160, 4, 64
    b = _block(T, E, H, I, k, G, False, seed=17)
    args, z = _gpu_args(b)
    res = d.normal_bf16((T, H), 2.0, 18, 3, T, H)
    gamma = d.f32_to_bf16_bits(np.full(H, 3.0, np.float32))
    n, r = binding.moe_add_rmsnorm(args[0], dev(gamma), dev(res))
    y = binding.moe_forward_int4(n, *args[1:], k=k, **z)
    n_ref, _, _ = orc.add_rmsnorm(b[0], res, gamma, 1e-5)
    bits = (n_ref.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    assert_y_close(host_f64(y), orc.moe_forward_int4(bits, *b[1:], k=k, G=G)["y"])


@pytest.mark.parametrize("path", PATHS)
def test_rows_past_two_gib(path):
    """Token rows up to just below 4 GiB, gathered (gate_up) and in place (down): the last rows as in a small call."""
    _need_gpu()
    T, K, E, G = 524000, 4096, 2, 128
    m = _matrix(E, K, 64, G, False, 22)
    q, s, _ = _gpu(m)
    bias = dev(d.normal_bf16((E, 64), 0.5, 23, 1, E, 64))
    a = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    tail = dev(d.normal_bf16((40, K), 1.0, 24, 1, 40, K))
    a[-40:] = tail
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[-17:] = 1                                                     # both experts have rows in the tail
    cnt, off, rows, pos = binding.moe_permute(ids, E)
    small = binding.moe_permute(ids[-40:].contiguous(), E)
    h = binding.moe_gate_up_int4(a, q, s, bias, cnt, off, rows, 1, path=path)
    want = binding.moe_gate_up_int4(tail, q, s, bias, small[0], small[1], small[2], 1, path=path)
    assert torch.equal(h[pos[-40:].long()], want[small[3].long()])
    o = binding.moe_down_int4(a, q, s, bias, cnt, off, T, 1, path=path)   # rows in permuted order already
    want = binding.moe_down_int4(tail, q, s, bias, small[0], small[1], 40, 1, path=path)
    assert torch.equal(o[-40:], want)


@pytest.mark.parametrize("path", PATHS)
def test_graph_replays(path):
    """Two captured forwards that share a workspace and a stream, replayed in turn with eager calls between."""
    _need_gpu()
    T, E, H, I, k, G = 96, 8, 256, 160, 4, 64
    args, z = _gpu_args(_block(T, E, H, I, k, G, True, seed=19))
    x2 = args[0].flip(0).contiguous()
    ws = binding.alloc_workspace(T, H, E, k, I)
    ys = [torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [binding.moe_forward_int4(x, *args[1:], k=k, path=path, **z) for x in (args[0], x2)]
    torch.cuda.synchronize()
    graphs = []
    for x, y in zip((args[0], x2), ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.moe_forward_int4(x, *args[1:], k=k, y=y, workspace=ws, path=path, **z)
        graphs.append(g)
    for i in range(3):
        for y in ys:
            y.fill_(-1.0)
        ws.fill_(0xAB if i % 2 else 0x11)
        eager = binding.moe_forward_int4(x2, *args[1:], k=k, path=path, **z)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, want[1])
        assert all(torch.equal(y, w) for y, w in zip(ys, want)), i


def test_other_stream_with_its_own_workspace():
    _need_gpu()
    T, E, H, I, k, G = 96, 8, 256, 160, 4, 64
    args, z = _gpu_args(_block(T, E, H, I, k, G, False, seed=20))
    want = binding.moe_forward_int4(*args, k=k, **z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [binding.moe_forward_int4(*args, k=k, stream=s, **z) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(want, y) for y in got)


def test_no_tokens():
    _need_gpu()
    args, z = _gpu_args(_block(4, 4, 64, 32, 2, 32, False, seed=21))
    assert binding.moe_forward_int4(args[0][:0], *args[1:], k=2, **z).shape == (0, 64)


@pytest.mark.parametrize("raw", [False, True])
def test_stages_on_another_stream(raw):
    """A torch stream or a raw handle; outputs given and left to the call."""
    _need_gpu()
    T, E, H, I, k, G = 9, 8, 96, 64, 2, 32
    args, z = _gpu_args(_block(T, E, H, I, k, G, True, seed=47))
    cnt, off, rows, pos = binding.moe_permute(torch.from_numpy(_routing(T, E, k, 48)).cuda(), E)
    want = binding.moe_gate_up_int4(args[0], *args[3:6], cnt, off, rows, k, Wgu_z=z["Wgu_z"])
    o = binding.moe_down_int4(want, *args[6:9], cnt, off, T, k, Wd_z=z["Wd_z"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    buf = torch.full((T * k + 3, I), 7.0, dtype=torch.bfloat16, device="cuda")   # longer than the rows: left as it was
    torch.cuda.synchronize()
    for h in (None, buf):
        got = binding.moe_gate_up_int4(args[0], *args[3:6], cnt, off, rows, k, Wgu_z=z["Wgu_z"], h=h, stream=stream)
        got_o = binding.moe_down_int4(got, *args[6:9], cnt, off, T, k, Wd_z=z["Wd_z"], stream=stream)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(got_o, o)
    assert (buf[T * k:] == 7).all()
