"""Whole int4 and norm + FP8 blocks on both sides of 768 tokens, where the
router behind them changes from the exact one to the MFMA one, against the
float64 oracle (needs an MI355X): ids, weights and rows of whole batches,
padded batches and expert-parallel ranks."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_layer_route_amd import binding, datagen as d  # noqa: E402
import oracle.moe_oracle as orc  # noqa: E402
from checks import assert_routing, assert_y_close, bf16_bits, dev, host_f64  # noqa: E402

pytestmark = pytest.mark.gpu
H, I, G = 256, 96, 64
SIZES = [(768, 8, 2), (769, 8, 2), (769, 128, 4), (1100, 8, 4), (1100, 128, 4)]   # T, E, k


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _up(a):
    return dev(a) if a.dtype == np.uint16 else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _matrix(E, K, N, seed):
    """Plain int4 codes, scales and zero points."""
    rng = np.random.default_rng([seed, E, K, N])
    q = rng.integers(0, 16, (E, K, N), dtype=np.uint8)
    s = d.f32_to_bf16_bits((0.02 / 4.6 * 2.0 ** rng.uniform(-1, 1, (E, -(-K // G), N))).astype(np.float32))
    return q, s, rng.integers(6, 11, s.shape, dtype=np.uint8)


def _int4(T, E, k):
    cfg = d.small_config(T=T, E=E, H=H, I=I, k=k, x_scale=d.scale_for_hidden(H))
    x = d.make_activations(cfg, T)
    Wr, br = d.make_router(cfg, T)
    gu, down = _matrix(E, H, 2 * I, T), _matrix(E, I, H, T + 1)
    bgu, bd = d.normal_bf16((E, 2 * I), 0.01, T, 5, E, I), d.normal_bf16((E, H), 0.01, T, 7, E, H)
    return x, Wr, br, gu, bgu, down, bd


def _on_gpu(b):
    x, Wr, br, gu, bgu, down, bd = b
    up = [dev(x), dev(Wr), dev(br)]
    for (q, s, z), bias in ((gu, bgu), (down, bd)):
        up += [torch.from_numpy(orc.int4_pack(q)).cuda(), dev(s), dev(bias)]
    return up, {"Wgu_z": _up(gu[2]), "Wd_z": _up(down[2])}


def _picks(T, k):
    return (torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.full((T, k), -7.0, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("T,E,k", SIZES)
def test_int4(T, E, k):
    _need_gpu()
    b = _int4(T, E, k)
    args, z = _on_gpu(b)
    ids, w = _picks(T, k)
    y = binding.moe_forward_int4(*args, k=k, topk_ids=ids, topk_w=w, **z)
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"], f"T{T} E{E}")


@pytest.mark.parametrize("n", [0, 700, 1023])
@pytest.mark.parametrize("T,E,k", [(769, 128, 4), (1100, 8, 4)])
def test_int4_padded(T, E, k, n):
    """Fewer real tokens than rows (more, for the shorter batch: none is padding then)."""
    _need_gpu()
    b = _int4(T, E, k)
    args, z = _on_gpu(b)
    ids, w = _picks(T, k)
    counts = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    y = binding.moe_forward_padded_int4(*args, k=k, n_valid=torch.tensor([n], dtype=torch.int32, device="cuda"),
                                        expert_counts=counts, topk_ids=ids, topk_w=w, **z)
    m = min(n, T)
    assert (host_f64(y)[m:] == 0).all() and (ids[m:] == -1).all() and (w[m:] == 0).all()
    ref = orc.moe_forward_int4(*b, k=k, G=G)
    assert (counts.cpu().numpy() == np.bincount(ref["ids"][:m].ravel(), minlength=E)).all()
    if m:
        assert_routing(ids[:m].cpu().numpy(), w[:m].cpu().numpy(), ref["ids"][:m], ref["w"][:m], ref["logits"][:m], k)
        assert_y_close(host_f64(y)[:m], ref["y"][:m])


@pytest.mark.parametrize("T,E,k,lo,n", [(769, 128, 4, 16, 16), (1100, 8, 4, 3, 5), (1100, 128, 4, 127, 1)])
def test_int4_rank(T, E, k, lo, n):
    _need_gpu()
    b = _int4(T, E, k)
    args, z = _on_gpu(b)
    ids, w = _picks(T, k)
    c = slice(lo, lo + n)
    part = binding.moe_forward_ep_int4(*args[:3], *[a[c] for a in args[3:]], e_begin=lo, k=k, Wgu_z_local=z["Wgu_z"][c],
                                       Wd_z_local=z["Wd_z"][c], topk_ids=ids, topk_w=w)
    ref = orc.moe_forward_int4(*b, k=k, G=G, experts=(lo, lo + n))
    assert_routing(ids.cpu().numpy(), w.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(part), ref["y"], f"experts {lo}..{lo + n - 1}")


@pytest.mark.parametrize("T,E,k", SIZES)
def test_norm_fp8(T, E, k):
    _need_gpu()
    cfg = d.small_config(T=T, E=E, H=H, I=I, k=k)
    x, res = d.normal_bf16((T, H), 3.0, T, 91, T, H), d.normal_bf16((T, H), 3.0, T, 92, T, H)
    gamma = d.f32_to_bf16_bits((1.0 + 0.3 * np.random.default_rng(T).standard_normal(H)).astype(np.float32))
    w = (*d.make_router(cfg, T), *d.make_experts_fp8(cfg, T, threads=4))
    ids, tw = _picks(T, k)
    y, r = binding.moe_forward_norm_fp8(dev(x), dev(gamma), *[_up(a) for a in w], k=k, residual=dev(res), topk_ids=ids,
                                        topk_w=tw)
    ref = orc.moe_forward_norm_fp8(x, res, gamma, 1e-5, *w, k=k)
    assert (bf16_bits(r) == (ref["residual"].astype(np.float32).view(np.uint32) >> 16)).all()
    assert_routing(ids.cpu().numpy(), tw.cpu().numpy(), ref["ids"], ref["w"], ref["logits"], k)
    assert_y_close(host_f64(y), ref["y"], f"T{T} E{E}")


# ---------------------------------------------------------------------------
# few slots: run one by one, and in groups (a padded batch without padding)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (1, 32, 4), (2, 32, 4), (4, 64, 4), (8, 256, 8), (64, 256, 1)])
def test_few_slots_and_groups(T, E, k):
    """The two forms' weights are within one float32 step of each other (2^-23 of a value), so their float32 sums over a
    token's k picks differ by at most 2^-23 sum |w o| and the sums' own roundings, k 2^-24 of as much on each side (twice
    that is allowed, as the terms are the oracle's); the two bf16 roundings add half a step each, 2^-7 of the larger in all."""
    _need_gpu()
    b = _int4(T, E, k)
    args, z = _on_gpu(b)
    ys, ws = [], []
    for call in (binding.moe_forward_int4, binding.moe_forward_padded_int4):
        ids, w = _picks(T, k)
        ys.append(host_f64(call(*args, k=k, topk_ids=ids, topk_w=w, **z)))
        ws.append(w)
    assert (ws[0] - ws[1]).abs().le(2.0 ** -23 * ws[1]).all()
    ref = orc.moe_forward_int4(*b, k=k, G=G, keep=True)
    terms = (np.abs(ref["o"]).reshape(T, k, H) * ref["w"].reshape(T, k, 1)).sum(axis=1)
    tol = 2.0 ** -7 * np.maximum(np.abs(ys[0]), np.abs(ys[1])) + (1 + k) * 2.0 ** -22 * terms
    assert (np.abs(ys[0] - ys[1]) <= tol).all()
