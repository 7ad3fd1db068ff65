"""The block's gradients against the float64 oracle (needs an MI355X).  Every
call goes through the C ABI.

Bounds, derived element by element from the oracle's values:
 - a product of K bf16 pairs (exact in float32) is within (K / 16 + 9) 2^-23 of
   the sum of its terms' magnitudes (each matrix instruction adds 16 terms and
   is within an ulp of their sum); so are d, gate and up (with the bias);
 - dgate = w d (u + 1) f'(g), f(g) = g sigmoid(1.702 g), |f'| <= 1.1, |f''| <= 0.9,
   u + 1 <= 8; dup = w d f(g): the errors of d, gate and up go through these
   slopes, the hardware exponential and reciprocal add 2^-18 of each factor's
   bound; where gate or up is nearer to a clamp than its error, either side is
   allowed; rounding to bf16 adds 2^-8;
 - w h likewise; dw's sum over i in float32 (I / 16 + 20 additions), dl from it;
 - the outputs: the operands' errors times the other operand's magnitudes, the
   product's own error, and 2^-8 for the rounding to bf16.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import bf16_bits, dev, host_f64  # noqa: E402

pytestmark = pytest.mark.gpu
ULP, HALF = 2.0 ** -23, 2.0 ** -8
NAMES = ("dx", "dWr", "dbr", "dWgu", "dbgu", "dWd", "dbd")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(T, E, H, I, seed, gate_std=4.0):
    x = d.normal_bf16((T, H), 50.0 * gate_std / np.sqrt(H), seed, 1, T, H)
    Wr = d.normal_bf16((E, H), 0.02, seed, 2, E, H)
    Wgu, bgu = d.normal_bf16((E, H, 2 * I), 0.02, seed, 4, E, H), d.normal_bf16((E, 2 * I), 0.3, seed, 5, E, I)
    Wd, bd = d.normal_bf16((E, I, H), 0.02, seed, 6, E, I), d.normal_bf16((E, H), 0.3, seed, 7, E, H)
    return d.normal_bf16((T, H), 0.05, seed, 8, T, H), x, Wr, Wgu, bgu, Wd, bd


def _routing(T, E, k, seed, live=None):
    """Different ids in a row, among the first `live` experts, and softmax weights (float32)."""
    rng = np.random.default_rng([seed, T, E])
    ids = np.stack([rng.permutation(live or E)[:k] for _ in range(T)]).astype(np.int32)
    p = np.exp(rng.standard_normal((T, k)))
    return ids, (p / p.sum(axis=1, keepdims=True)).astype(np.float32)


def _bounds(dy, x, Wr, Wgu, bgu, Wd, bd, ids, w, g):
    """How far each gradient may be from the oracle's g."""
    dyv, xv, w = np.abs(orc.widen(dy)), orc.widen(x), w.astype(np.float64)
    (T, H), (E, I) = xv.shape, Wd.shape[:2]
    b = {n: np.zeros_like(v) for n, v in g.items()}
    e_dw, m_dw = np.zeros_like(w), np.zeros_like(w)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        Wg, Wo, wt = orc.widen(Wgu[e]), orc.widen(Wd[e]), w[t, j][:, None]
        u = xv[t] @ Wg + orc.widen(bgu[e])
        e_u = (H / 16 + 9) * ULP * (np.abs(xv[t]) @ np.abs(Wg) + np.abs(orc.widen(bgu[e])))
        dv = np.abs(orc.widen(dy)[t] @ Wo.T)
        e_d = (H / 16 + 9) * ULP * (dyv[t] @ np.abs(Wo).T)
        eg, eu = e_u[:, 0::2], e_u[:, 1::2]
        gate, up = np.minimum(u[:, 0::2], 7.0), np.clip(u[:, 1::2], -7.0, 7.0)
        with np.errstate(over="ignore"):
            z = 1.0 / (1.0 + np.exp(-1.702 * gate))
        f, fp, hw = np.abs(gate * z), np.abs(z + 1.702 * gate * z * (1 - z)), 2.0 ** -18
        up1 = np.abs(up + 1.0)
        h, e_h = up1 * f, 8.8 * eg + eu * (f + 1.1 * eg) + hw * 8 * f
        e_dg = wt * (e_d * 8.8 + dv * (eu * 1.1 + up1 * (0.9 * eg + 1.1 * hw)))
        e_du = wt * (e_d * (f + 1.1 * eg) + dv * (1.1 * eg + hw * f))
        e_dg += np.where(np.abs(u[:, 0::2] - 7.0) <= eg, wt * (dv + e_d) * up1 * 1.1, 0)
        e_du += np.where(np.abs(np.abs(u[:, 1::2]) - 7.0) <= eu, wt * (dv + e_d) * f, 0)
        m = np.empty_like(u)
        m[:, 0::2], m[:, 1::2] = wt * dv * up1 * fp, wt * dv * f
        e_m = np.empty_like(u)
        e_m[:, 0::2], e_m[:, 1::2] = e_dg, e_du
        e_m += HALF * (m + e_m)                                                # rounded to bf16
        e_wh = wt * e_h + HALF * wt * (h + e_h)
        n = t.size
        np.add.at(b["dx"], t, e_m @ np.abs(Wg).T + (2 * I / 16 + 9) * ULP * ((m + e_m) @ np.abs(Wg).T))
        b["dWgu"][e] = np.abs(xv[t]).T @ (e_m + (n / 16 + 9) * ULP * (m + e_m))
        b["dbgu"][e] = (e_m + (n + 9) * ULP * (m + e_m)).sum(axis=0)
        b["dWd"][e] = (e_wh + (n / 16 + 9) * ULP * wt * h).T @ dyv[t]
        b["dbd"][e] = (n + 9) * ULP * (wt * dyv[t]).sum(axis=0)
        bd_dy = dyv[t] @ np.abs(orc.widen(bd[e]))
        m_dw[t, j] = (h * dv).sum(axis=1) + bd_dy
        e_dw[t, j] = (e_h * dv + h * e_d + e_h * e_d).sum(axis=1) + ((I + H) / 16 + 40) * ULP * m_dw[t, j]
    e_dl = w * (e_dw + (w * e_dw).sum(axis=1, keepdims=True)) + 12 * ULP * w * (m_dw + (w * m_dw).sum(axis=1, keepdims=True))
    m_dl = w * (m_dw + (w * m_dw).sum(axis=1, keepdims=True))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        el, ml, n = e_dl[t, j], m_dl[t, j], t.size
        np.add.at(b["dx"], t, (el + 9 * ULP * ml)[:, None] * np.abs(orc.widen(Wr[e]))[None])
        b["dWr"][e], b["dbr"][e] = (el + (n + 9) * ULP * ml) @ np.abs(xv[t]), (el + (n + 9) * ULP * ml).sum()
    return {n: v + HALF * (np.abs(g[n]) + v) + 1e-37 for n, v in b.items()}


def _run(inputs, ids, w, **kw):
    return binding.moe_backward(*[dev(a) for a in inputs], torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), **kw)


def _check(inputs, ids, w, got, names=NAMES):
    ref = orc.moe_backward(*inputs, ids, w)
    tol = _bounds(*inputs, ids, w, ref)
    assert tuple(got) == tuple(names)
    for n in names:
        v = host_f64(got[n])
        bad = np.argwhere(~(np.abs(v - ref[n]) <= tol[n]))
        assert bad.size == 0, (f"{n}: {len(bad)} of {v.size} off, first {bad[0].tolist()}: {v[tuple(bad[0])]} for "
                               f"{ref[n][tuple(bad[0])]} +- {tol[n][tuple(bad[0])]}")
        # the bound covers the worst case; what is usual is bf16's own rounding
        norm = np.linalg.norm(ref[n])
        assert np.linalg.norm(v - ref[n]) <= 6e-3 * norm + 1e-30, (n, np.linalg.norm(v - ref[n]) / norm)


# T, E, k, H, I, live experts
SIZES = [
    (1, 1, 1, 8, 8, None),          # the smallest
    (1, 4, 2, 64, 40, None),        # one token: two experts with a row, two without
    (3, 2, 2, 72, 24, None),        # H and I end inside a 16-byte chunk's run
    (17, 3, 1, 264, 136, 2),        # one column past a tile of 256; an expert without rows
    (70, 2, 2, 520, 360, None),     # 70 rows: K of the weights' gradients ends inside the second stage
    (300, 1, 1, 256, 128, None),    # past one tile of rows; exactly a tile of columns
    (129, 4, 3, 96, 264, None),
    (64, 40, 8, 128, 64, 30),       # many experts, k = 8
    (520, 2, 1, 40, 512, None),     # one K stage that is not full; two tiles of rows
    (33, 2, 2, 2880, 104, None),    # the full hidden size
    (20, 2, 1, 104, 2880, None),    # the full intermediate size
    (400, 1, 1, 328, 200, None),    # 400 rows of one expert: wide tiles of the gradients, ragged both ways
    (777, 3, 2, 712, 392, None),    # several of them in both directions
    (50, 2, 1, 192, 96, None),      # exactly a tile of 192 columns
    (130, 2, 2, 200, 192, None),    # two rows past a tile of 128; eight columns past a tile
    (65, 1, 1, 448, 288, None),     # one row past half a tile; whole K stages
]


@pytest.mark.parametrize("T,E,k,H,I,live", SIZES)
def test_gradients(T, E, k, H, I, live):
    _need_gpu()
    inputs, (ids, w) = _inputs(T, E, H, I, 21), _routing(T, E, k, 22, live)
    _check(inputs, ids, w, _run(inputs, ids, w))


def test_clamped_values():
    """Pre-activations exactly on the clamps, and beyond: one-hot rows against weights of 7 and their neighbours."""
    _need_gpu()
    T, E, H, I = 16, 1, 16, 32
    dy, x, Wr, Wgu, bgu, Wd, bd = _inputs(T, E, H, I, 23)
    x[:] = 0
    x[np.arange(T), np.arange(H)] = 0x3F80
    vals = np.array([7.0, 7.03125, 6.96875, -7.0, -7.03125, -6.96875, 0.0, 30.0, -30.0, 100.0, -100.0, 1.0], np.float32)
    Wgu[:] = d.f32_to_bf16_bits(np.random.default_rng(1).choice(vals, Wgu.size).astype(np.float32)).reshape(Wgu.shape)
    bgu[:] = 0
    ids, w = _routing(T, E, 1, 24)
    _check((dy, x, Wr, Wgu, bgu, Wd, bd), ids, w, _run((dy, x, Wr, Wgu, bgu, Wd, bd), ids, w))


def test_skipped_slots_and_unused_experts():
    """Slots of no expert add nothing, a token without any gets 0, and what the buffers held before is gone."""
    _need_gpu()
    T, E, k, H, I = 40, 5, 2, 136, 72
    inputs, (ids, w) = _inputs(T, E, H, I, 25), _routing(T, E, k, 26, 4)
    ids[7], w[7] = -1, 0
    ids[30:], w[30:] = -1, 0
    g = {n: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for n, s in
         (("dx", (T, H)), ("dWr", (E, H)), ("dbr", (E,)), ("dWgu", (E, H, 2 * I)), ("dbgu", (E, 2 * I)), ("dWd", (E, I, H)),
          ("dbd", (E, H)))}
    ws = binding.alloc_workspace_backward(T, H, E, k, I).fill_(0xFF)
    got = _run(inputs, ids, w, workspace=ws, **g)
    assert all(got[n] is g[n] for n in NAMES)
    _check(inputs, ids, w, got)
    assert (got["dx"][7] == 0).all() and (got["dx"][30:] == 0).all()
    assert all((got[n][4] == 0).all() for n in NAMES[1:])
    # all of them
    ids[:], w[:] = -1, 0
    assert all((v == 0).all() for v in _run(inputs, ids, w).values())


def test_frozen_weights():
    _need_gpu()
    T, E, k, H, I = 50, 3, 2, 264, 40
    inputs, (ids, w) = _inputs(T, E, H, I, 27), _routing(T, E, k, 28)
    whole = _run(inputs, ids, w)
    for router in (False, True):
        for experts in (False, True):
            got = _run(inputs, ids, w, router=router, experts=experts)
            want = NAMES[:1] + (NAMES[1:3] if router else ()) + (NAMES[3:] if experts else ())
            assert tuple(got) == want and all((bf16_bits(got[n]) == bf16_bits(whole[n])).all() for n in want)
    assert {n: tuple(v.shape) for n, v in binding.moe_backward(
        *[dev(a[:0] if i < 2 else a) for i, a in enumerate(inputs)], torch.empty((0, k), dtype=torch.int32, device="cuda"),
        torch.empty((0, k), device="cuda")).items() if (v != 0).any()} == {}


def test_behind_the_forward_and_against_differences():
    """Forward, padded forward and backward as a training step uses them; the gradients against central differences of
    the float64 forward along random directions, router included."""
    _need_gpu()
    T, E, k, H, I = 48, 4, 2, 136, 104
    dy, x, Wr, Wgu, bgu, Wd, bd = _inputs(T, E, H, I, 29, gate_std=2.0)
    br = d.normal_bf16((E,), 0.1, 30, 1, E, 1)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    binding.moe_forward(dev(x), dev(Wr), dev(br), dev(Wgu), dev(bgu), dev(Wd), dev(bd), k=k, topk_ids=ids, topk_w=w)
    got = binding.moe_backward(*[dev(a) for a in (dy, x, Wr, Wgu, bgu, Wd, bd)], ids, w)
    _check((dy, x, Wr, Wgu, bgu, Wd, bd), ids.cpu().numpy(), w.cpu().numpy(), got)
    p = [torch.from_numpy(orc.widen(v)) for v in (x, Wr, br, Wgu, bgu, Wd, bd)]
    dyt, idt = torch.from_numpy(orc.widen(dy)), ids.cpu().long()

    def loss(x, Wr, br, Wgu, bgu, Wd, bd):
        wt = torch.softmax(torch.gather(x @ Wr.t() + br, 1, idt), dim=1)
        u = torch.matmul(x[None], Wgu) + bgu[:, None]
        gate, up = u[..., 0::2].clamp(max=7.0), u[..., 1::2].clamp(-7.0, 7.0)
        o = torch.matmul((up + 1) * gate * torch.sigmoid(1.702 * gate), Wd) + bd[:, None]
        return float(((o[idt, torch.arange(T)[:, None]] * wt[:, :, None]).sum(dim=1) * dyt).sum())
    rng = np.random.default_rng(2)
    for i, n in enumerate(NAMES):
        # along the gradient itself, disturbed: nothing cancels, so the rounding's 2^-8 is a share of the result
        v = got[n].cpu().double() * torch.from_numpy(rng.uniform(0.5, 1.5, p[i].shape))
        h = 1e-5 / max(1e-30, float(v.abs().max()))
        diff = (loss(*(q + h * v if j == i else q for j, q in enumerate(p))) -
                loss(*(q - h * v if j == i else q for j, q in enumerate(p)))) / (2 * h)
        want = float((got[n].cpu().double() * v).sum())
        assert abs(diff - want) <= 8e-3 * want, (n, diff, want)
    # a static batch whose tail is padding
    n_valid = torch.tensor([31], dtype=torch.int32, device="cuda")
    binding.moe_forward_padded(dev(x), dev(Wr), dev(br), dev(Wgu), dev(bgu), dev(Wd), dev(bd), k=k, n_valid=n_valid,
                               topk_ids=ids, topk_w=w)
    got = binding.moe_backward(*[dev(a) for a in (dy, x, Wr, Wgu, bgu, Wd, bd)], ids, w)
    part = binding.moe_backward(*[dev(a[:31] if j < 2 else a) for j, a in enumerate((dy, x, Wr, Wgu, bgu, Wd, bd))],
                                ids[:31].contiguous(), w[:31].contiguous())
    assert (got["dx"][31:] == 0).all() and (bf16_bits(got["dx"])[:31] == bf16_bits(part["dx"])).all()
    assert all((bf16_bits(got[n]) == bf16_bits(part[n])).all() for n in NAMES[1:])


def test_nan_reaches_its_own_rows_only():
    _need_gpu()
    T, E, k, H, I = 24, 4, 1, 72, 40
    dy, *rest = _inputs(T, E, H, I, 31)
    ids, w = _routing(T, E, k, 32)
    clean = _run((dy, *rest), ids, w)
    dy = dy.copy()
    dy[5, 3] = 0x7FC0
    got = _run((dy, *rest), ids, w)
    e = int(ids[5, 0])
    assert torch.isnan(got["dx"][5]).all() and torch.isnan(got["dWd"][e][:, 3]).all()
    keep = [t for t in range(T) if t != 5]
    assert (bf16_bits(got["dx"])[keep] == bf16_bits(clean["dx"])[keep]).all()
    for n in NAMES[1:]:
        others = [i for i in range(E) if i != e]
        assert (bf16_bits(got[n])[others] == bf16_bits(clean[n])[others]).all(), n


def test_repeats_graph_and_other_stream():
    """The same bits again, over other bytes in the workspace, from a captured graph's replays and on another stream."""
    _need_gpu()
    T, E, k, H, I = 300, 6, 4, 264, 200
    inputs, (ids, w) = _inputs(T, E, H, I, 33), _routing(T, E, k, 34)
    a = [dev(v) for v in inputs] + [torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()]
    ws = binding.alloc_workspace_backward(T, H, E, k, I)
    g = binding.moe_backward(*a, workspace=ws)
    want = {n: bf16_bits(v).copy() for n, v in g.items()}

    def same(got):
        assert all((bf16_bits(got[n]) == want[n]).all() for n in NAMES)
    ws.fill_(0x7F)
    same(binding.moe_backward(*a, workspace=ws))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = binding.moe_backward(*a, stream=s)
    s.synchronize()
    same(other)
    with torch.cuda.stream(s):
        binding.moe_backward(*a, workspace=ws, **g)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_backward(*a, workspace=ws, **g)
    for i in range(4):
        for v in g.values():
            v.view(torch.int16).fill_(-1)
        ws.fill_(0xAB if i % 2 else 0x11)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(g)


def test_same_expert_twice_in_a_row():
    """A token that names an expert twice has two slots there."""
    _need_gpu()
    T, E, k, H, I = 60, 3, 3, 136, 104
    inputs, (ids, w) = _inputs(T, E, H, I, 35), _routing(T, E, k, 36)
    ids[::2, 2] = ids[::2, 0]
    _check(inputs, ids, w, _run(inputs, ids, w))


def test_two_calls_at_once():
    """Two streams, each with its own workspace, in turn without a wait between them."""
    _need_gpu()
    E, k, H, I = 4, 2, 264, 136
    calls = []
    for T in (90, 333):
        inputs, (ids, w) = _inputs(T, E, H, I, 37), _routing(T, E, k, 38)
        calls.append([dev(v) for v in inputs] + [torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()])
    want = [{n: bf16_bits(v) for n, v in binding.moe_backward(*c).items()} for c in calls]
    spaces = [binding.alloc_workspace_backward(c[0].shape[0], H, E, k, I) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[binding.moe_backward(*c, workspace=ws, stream=s) for c, ws, s in zip(calls, spaces, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    for pair in got:
        for g, bits in zip(pair, want):
            assert all((bf16_bits(g[n]) == bits[n]).all() for n in NAMES)


def test_rows_past_four_gib():
    """Slots whose rows of d and of its gradients lie beyond 2^32 bytes: the last tokens' dx, alone and at the end of a
    batch, are the same bits (every row is summed in the same order)."""
    _need_gpu()
    T, n, E, k, H, I = 200000, 100, 2, 2, 64, 2880
    small, (ids, w) = _inputs(n, E, H, I, 39), _routing(n, E, k, 40)
    part = [dev(v) for v in small] + [torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()]
    alone = bf16_bits(binding.moe_backward(*part, router=False, experts=False)["dx"])
    dy, x = (torch.randn((T, H), device="cuda").bfloat16() for _ in range(2))
    ids_all = torch.tensor([0, 1], dtype=torch.int32, device="cuda").repeat(T, 1)
    w_all = torch.full((T, k), 0.5, device="cuda")
    for whole, piece in ((dy, part[0]), (x, part[1]), (ids_all, part[7]), (w_all, part[8])):
        whole[T - n:] = piece
    got = binding.moe_backward(dy, x, *part[2:7], ids_all, w_all, router=False, experts=False)["dx"]
    assert (bf16_bits(got[T - n:]) == alone).all()
