"""Cases that time the block with 4 bits on both sides and the block's backward pass: MXFP4 quantisation of rows and
reading them back, the down product of MXFP4 rows and MXFP4 weights, the whole block on such products, and the gradients
of the bf16 block.

``own`` chooses between the plain form (elementary torch operations, float32 or float64) and the library's calls.

MXFP4: 32 values share a power of two, 2^(s - 127) with s one byte; a value is a 4-bit E2M1 number (bit 3 the sign, then
the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) times it.  Weights as ``moe_quantize_mxfp4`` writes them: codes uint8
[E][N][K/2], the even k in the low half of a byte, and scales uint8 [E][K/32][N].  Rows as ``moe_quantize_rows_mxfp4``
writes them: codes uint8 [R][K/2] and scales uint8 [ceil(K/128)][R][4], four blocks of a row side by side.
"""
import math

import torch

own = False

H0 = 2880            # hidden and intermediate size of the repository's own workloads
X_NORM = 190.85      # |x| of a row where the GLU's clamps are reached at about 5%, as the repository's generator draws them


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's row: latency
        {"name": "rows_t1", "op": "rows", "R": 1, "K": H0},
        # the largest prefill batch of the repository's workloads
        {"name": "rows_t16384", "op": "rows", "R": 16384, "K": H0},
        # the down product of a decode batch: about eight rows an expert, bound by the weights' bytes
        {"name": "down_t64", "op": "down", "T": 64, "E": 32, "k": 4, "H": H0, "I": H0},
        # of a prefill chunk of odd length: about 128 rows an expert, none a multiple of a tile
        {"name": "down_t1021", "op": "down", "T": 1021, "E": 32, "k": 4, "H": H0, "I": H0},
        # the whole block for one token: latency, four live experts
        {"name": "forward_t1", "op": "forward", "T": 1, "E": 32, "k": 4, "H": H0, "I": H0},
        # a decode batch
        {"name": "forward_t64", "op": "forward", "T": 64, "E": 32, "k": 4, "H": H0, "I": H0},
        # a verify step over many experts
        {"name": "forward_t256_e128", "op": "forward", "T": 256, "E": 128, "k": 4, "H": H0, "I": H0},
        # a prefill batch: 512 rows an expert
        {"name": "forward_t4096", "op": "forward", "T": 4096, "E": 32, "k": 4, "H": H0, "I": H0},
        # the gradients of a small model's layer: few ragged rows an expert, sizes that no tile divides
        {"name": "backward_t77_small", "op": "backward", "T": 77, "E": 8, "k": 2, "H": 520, "I": 360},
        # of a short micro-batch: 64 rows an expert, as much weight and gradient traffic as products
        {"name": "backward_t512", "op": "backward", "T": 512, "E": 32, "k": 4, "H": H0, "I": H0},
        # of a micro-batch at many experts, ragged length
        {"name": "backward_t2047_e128", "op": "backward", "T": 2047, "E": 128, "k": 4, "H": H0, "I": H0},
        # of a training batch: 512 rows an expert
        {"name": "backward_t4096", "op": "backward", "T": 4096, "E": 32, "k": 4, "H": H0, "I": H0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rows", "down", "forward", "forward", "backward", "backward"))
    if op == "rows":
        K = 32 * _log(rng, 2, 256)
        return {"op": op, "R": _log(rng, 1, min(16384, 16384 * H0 // K)), "K": K}
    case = {"op": op, "E": rng.choice((4, 8, 16, 32, 60, 64, 128)), "k": rng.choice((1, 2, 4, 4))}
    if op == "backward":
        case |= {"H": 8 * _log(rng, 16, 360), "I": 8 * _log(rng, 16, 360), "T": _log(rng, 1, 16384 // case["k"])}
        case["E"] = min(case["E"], 64)
    else:
        case |= {"H": 32 * _log(rng, 4, 90), "I": 32 * _log(rng, 4, 90), "T": _log(rng, 1, 16384 // case["k"])}
    return case


def work(case):
    if case["op"] == "rows":
        n = case["R"] * case["K"]
        return {"bytes": 2 * (2 * n + n // 2 + n // 32), "flops": 6 * n}
    T, E, k, H, I = (case[v] for v in ("T", "E", "k", "H", "I"))
    S = T * k
    live = E * (1.0 - (1.0 - k / E) ** T)   # experts that some token picks, routing spread evenly

    def fp4(K, N):
        return live * (K * N * 17 / 32 + 2 * N)

    if case["op"] == "down":
        return {"bytes": fp4(I, H) + S * I * 17 / 32 + 4 * S * H, "flops": 2 * S * H * I}
    if case["op"] == "forward":
        return {"bytes": fp4(H, 2 * I) + fp4(I, H) + 2 * E * H + 2 * E + 4 * T * H, "flops": 6 * S * H * I + 2 * T * E * H}
    weights = 3 * H * I + 2 * I + H
    return {"bytes": 2 * weights * (live + E) + 4 * E * H + 6 * T * H + 8 * S,
            "flops": 16 * S * H * I + 4 * S * H}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def _fp4(g, E, K, N):
    """MXFP4 weights of deviation about 0.02 (uniform codes have one of 2.9 units)."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(119, 121, (E, K // 32, N), generator=g, device="cuda", dtype=torch.uint8)
    return q, s


def _ids(g, T, E, k):
    return torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.int()


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c)
    if c["op"] == "rows":
        R, K = c["R"], c["K"]
        # rows of a residual stream: a few channels far above the others
        loud = torch.exp2(3.0 * (torch.rand(K, generator=g, device="cuda") < 0.01))
        st["a"] = (torch.randn((R, K), generator=g, device="cuda") * loud * 3.5).bfloat16()
        st["codes"] = torch.empty((R, K // 2), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty((-(-K // 128), R, 4), dtype=torch.uint8, device="cuda")
        st["values"] = torch.empty_like(st["a"])
        return st
    T, E, k, H, I = (c[v] for v in ("T", "E", "k", "H", "I"))
    S = T * k
    st["bd"] = _normal(g, E, H, std=0.01)
    if c["op"] == "down":
        flat = _ids(g, T, E, k).flatten().long()
        st["cnt"] = torch.bincount(flat, minlength=E).int()
        st["off"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int32), st["cnt"].cumsum(0).int()])
        st["cap"] = int(st["cnt"].max())
        st["hq"] = torch.randint(0, 256, (S, I // 2), generator=g, device="cuda", dtype=torch.uint8)
        st["hs"] = torch.randint(125, 129, (-(-I // 128), S, 4), generator=g, device="cuda", dtype=torch.uint8)
        st["q"], st["s"] = _fp4(g, E, I, H)
        st["out"] = torch.empty((S, H), dtype=torch.float32, device="cuda")
        return st
    st["Wr"], st["br"] = _normal(g, E, H, std=0.02), _normal(g, E, std=0.1)
    st["bgu"] = _normal(g, E, 2 * I, std=0.01)
    if c["op"] == "forward":
        st["x"] = _normal(g, T, H, std=X_NORM / math.sqrt(H))
        st["gu_q"], st["gu_s"] = _fp4(g, E, H, 2 * I)
        st["d_q"], st["d_s"] = _fp4(g, E, I, H)
        st["y"] = torch.empty_like(st["x"])
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        st["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        # the rows that a plain program sets aside for the fullest expert
        st["cap"] = int(torch.bincount(_route(st)[0].flatten(), minlength=E).max())
        # the scratch buffer a serving loop keeps (a little more than the library asks for)
        st["ws"] = torch.empty(S * (I + 4 * H + 64) + T * (H + 64) + (1 << 16), dtype=torch.uint8, device="cuda")
        return st
    # a training step: gates of deviation 2, of which a few reach the clamps; the routing as the forward pass left it
    st["x"] = _normal(g, T, H, std=0.53 * X_NORM / math.sqrt(H))
    st["dy"] = _normal(g, T, H, std=0.05)
    st["Wgu"], st["Wd"] = _normal(g, E, H, 2 * I, std=0.02), _normal(g, E, I, H, std=0.02)
    ids, w = _route(st)
    st["ids"], st["w"] = ids.int().contiguous(), w.contiguous()
    st["cap"] = int(torch.bincount(ids.flatten(), minlength=E).max())
    st["grads"] = {"dx": torch.empty_like(st["x"]), "dWr": torch.empty_like(st["Wr"]), "dbr": torch.empty_like(st["br"]),
                   "dWgu": torch.empty_like(st["Wgu"]), "dbgu": torch.empty_like(st["bgu"]),
                   "dWd": torch.empty_like(st["Wd"]), "dbd": torch.empty_like(st["bd"])}
    # the scratch buffer a training loop keeps
    st["ws"] = torch.empty(S * (12 * I + 4 * H + 512) + 512 * E * (I + H) + (1 << 24), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------ the plain forms
_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(v):
    """Values of the nearest MXFP4 row blocks of float32 [..][K] (finite)."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(dim=-1, keepdim=True)
    e = torch.where(amax == 0, torch.full_like(amax, -127.0), (torch.frexp(amax).exponent - 3).float()).clamp(-127.0, 127.0)
    unit = torch.exp2(e)
    m = b.abs() / unit
    code = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    table = torch.tensor(_MAGNITUDES, device=v.device)
    return (table.take(code.long()) * b.sign() * unit).flatten(-2)


def _values(codes, t):
    """E2M1 values [..][K] of packed codes [..][K/2]."""
    table = torch.tensor([*_MAGNITUDES, *(-m for m in _MAGNITUDES)], device=codes.device, dtype=t)
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], dim=1)      # byte -> its two values
    return pairs.index_select(0, codes.flatten().int()).view(*codes.shape[:-1], 2 * codes.shape[-1])


def _weights(q, s, t):
    """Weights [E][N][K]."""
    return (_values(q, t).unflatten(-1, (-1, 32)) * torch.exp2(s.to(t) - 127.0).transpose(1, 2).unsqueeze(-1)).flatten(-2)


def _row_units(s, K):
    """Row scales [ceil(K/128)][R][4] -> bytes [R][K/32]."""
    return s.permute(1, 0, 2).flatten(1)[:, :K // 32]


def _glu(gu):
    gate, up = gu[..., 0::2].clamp(max=7.0), gu[..., 1::2].clamp(-7.0, 7.0)
    return (up + 1.0) * (gate / (1.0 + torch.exp(-1.702 * gate)))


def _route(st):
    """The k largest router logits (float64, decided after rounding to float32; ties to the lower index), softmax weights."""
    logits = (st["x"].double() @ st["Wr"].double().t() + st["br"].double()).float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :st["k"]], ids[:, :st["k"]]
    p = torch.exp(top - top[:, :1])
    return ids, p / p.sum(dim=1, keepdim=True)


def _dispatch(ids, E, cap):
    """Row of [E * cap] for each (token, slot), slots in token order within an expert."""
    flat = ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    start = torch.bincount(flat, minlength=E).cumsum(0) - torch.bincount(flat, minlength=E)
    at = torch.empty_like(flat)
    at[order] = torch.arange(flat.numel(), device=flat.device) - start[flat[order]]
    return flat * cap + at


def _spread(v, at, E, cap):
    """Rows of v put at `at` of zeros [E][cap][..]."""
    out = torch.zeros((E * cap, v.shape[1]), dtype=v.dtype, device=v.device)
    out[at] = v
    return out.view(E, cap, v.shape[1])


def _plain(st):
    op = st["op"]
    if op == "rows":
        return {"values": _quantize(st["a"].float()).bfloat16()}
    E, k, cap = st["E"], st["k"], st["cap"]
    if op == "down":
        unit = torch.exp2(_row_units(st["hs"], st["I"]).float() - 127.0)
        h = (_values(st["hq"], torch.float32).unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)
        e = torch.repeat_interleave(torch.arange(E, device=h.device), st["cnt"].long(), output_size=h.shape[0])
        at = e * cap + torch.arange(h.shape[0], device=h.device) - st["off"].long()[e]
        o = torch.bmm(_spread(h, at, E, cap), _weights(st["q"], st["s"], torch.float32).transpose(1, 2))
        return (o + st["bd"].float().unsqueeze(1)).flatten(0, 1)[at]
    if op == "forward":
        ids, w = _route(st)
        at = _dispatch(ids, E, cap)
        xs = _spread(_quantize(st["x"].float()).repeat_interleave(k, dim=0), at, E, cap)
        gu = torch.bmm(xs, _weights(st["gu_q"], st["gu_s"], torch.float32).transpose(1, 2))
        h = _quantize(_glu(gu + st["bgu"].float().unsqueeze(1)).bfloat16().float())
        o = torch.bmm(h, _weights(st["d_q"], st["d_s"], torch.float32).transpose(1, 2)) + st["bd"].float().unsqueeze(1)
        y = (o.flatten(0, 1)[at].view(-1, k, st["H"]) * w.unsqueeze(2)).sum(dim=1)
        return {"y": y.bfloat16(), "ids": ids.int(), "w": w}
    ids, w, x, dy = st["ids"].long(), st["w"], st["x"].float(), st["dy"].float()
    Wgu, Wd = st["Wgu"].float(), st["Wd"].float()
    at = _dispatch(ids, E, cap)
    xs, ds = (_spread(v.repeat_interleave(k, dim=0), at, E, cap) for v in (x, dy))
    ws = _spread(w.flatten().unsqueeze(1), at, E, cap)
    gu = torch.bmm(xs, Wgu) + st["bgu"].float().unsqueeze(1)
    d = torch.bmm(ds, Wd.transpose(1, 2))
    gate, up = gu[..., 0::2], gu[..., 1::2]
    g, u = gate.clamp(max=7.0), up.clamp(-7.0, 7.0)
    s = 1.0 / (1.0 + torch.exp(-1.702 * g))
    h = (u + 1.0) * g * s
    dw = ((h * d).sum(dim=2) + (ds * st["bd"].float().unsqueeze(1)).sum(dim=2)).flatten()[at].view_as(w)
    dl = w * (dw - (w * dw).sum(dim=1, keepdim=True))
    dh = ws * d
    dgu = torch.stack([dh * (u + 1.0) * s * (1.0 + 1.702 * g * (1.0 - s)) * (gate <= 7.0), dh * g * s * (up.abs() <= 7.0)],
                      dim=3).flatten(2)
    dx = torch.bmm(dgu, Wgu.transpose(1, 2)).flatten(0, 1)[at].view(-1, k, st["H"]).sum(dim=1)
    dx += (dl.unsqueeze(2) * st["Wr"].float()[ids]).sum(dim=1)
    dls = torch.zeros((x.shape[0], E), device=x.device).scatter_(1, ids, dl)
    grads = {"dx": dx, "dWr": dls.t() @ x, "dbr": dls.sum(dim=0), "dWgu": torch.bmm(xs.transpose(1, 2), dgu),
             "dbgu": dgu.sum(dim=1), "dWd": torch.bmm((ws * h).transpose(1, 2), ds), "dbd": (ws * ds).sum(dim=1)}
    return {n: v.bfloat16() for n, v in grads.items()}


def _own(st):
    from moe_layer_route_amd import binding as moe
    op = st["op"]
    if op == "rows":
        codes, scales = moe.moe_quantize_rows_mxfp4(st["a"], codes=st["codes"], scales=st["scales"])
        return {"values": moe.moe_dequantize_rows_mxfp4(codes, scales, out=st["values"])}
    if op == "down":
        return moe.moe_down_w4a4(st["hq"], st["hs"], st["q"], st["s"], st["bd"], st["cnt"], st["off"], T=st["T"], k=st["k"],
                                 o=st["out"])
    if op == "forward":
        y = moe.moe_forward_w4a4(st["x"], st["Wr"], st["br"], st["gu_q"], st["gu_s"], st["bgu"], st["d_q"], st["d_s"],
                                 st["bd"], k=st["k"], y=st["y"], workspace=st["ws"], topk_ids=st["ids"], topk_w=st["w"])
        return {"y": y, "ids": st["ids"], "w": st["w"]}
    return moe.moe_backward(st["dy"], st["x"], st["Wr"], st["Wgu"], st["bgu"], st["Wd"], st["bd"], st["ids"], st["w"],
                            workspace=st["ws"], **st["grads"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ in 64 bits
def _quantize64(v):
    """Nearest MXFP4 blocks of float64 values: the step of a magnitude is half its power of two, at least half the unit."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(dim=-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(amax.clamp(min=2.0 ** -125))) - 2.0)
    m = b / unit
    step = torch.exp2(torch.floor(torch.log2(m.abs().clamp(min=1.0))) - 1.0)
    return ((torch.round(m / step) * step).clamp(-6.0, 6.0) * unit).flatten(-2)


def _value64(codes):
    """E2M1 numbers from their bits."""
    v = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    sign = torch.where(v >= 8, -1.0, 1.0)
    m = v % 8
    exponent, half = torch.floor(m / 2), m % 2
    return sign * torch.where(exponent == 0, half / 2, (1 + half / 2) * torch.exp2(exponent - 1))


def _weight64(q, s, e):
    """Expert e's weights [N][K]."""
    return _value64(q[e]) * torch.exp2(s[e].double() - 127).t().repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "rows":
        return {"values": _quantize64(st["a"].double())}
    E, k = st["E"], st["k"]
    if op == "down":
        unit = st["hs"].permute(1, 0, 2).reshape(st["hs"].shape[1], -1)[:, :st["I"] // 32].double()
        h = _value64(st["hq"]) * torch.exp2(unit - 127).repeat_interleave(32, dim=1)
        out, off = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda"), st["off"].tolist()
        for e in range(E):
            out[off[e]:off[e + 1]] = h[off[e]:off[e + 1]] @ _weight64(st["q"], st["s"], e).t() + st["bd"][e].double()
        return out
    x = st["x"].double()
    if op == "forward":
        logits = x @ st["Wr"].double().t() + st["br"].double()
        order = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
        p = torch.softmax(torch.gather(logits, 1, order), dim=1)
        v, y = _quantize64(x), torch.zeros_like(x)
        for e in range(E):
            t, j = torch.nonzero(order == e, as_tuple=True)
            if t.numel():
                h = _glu(v[t] @ _weight64(st["gu_q"], st["gu_s"], e).t() + st["bgu"][e].double())
                h = _quantize64(h.bfloat16().double())                      # h is bf16, then MXFP4, by definition
                o = h @ _weight64(st["d_q"], st["d_s"], e).t() + st["bd"][e].double()
                y.index_add_(0, t, o * p[t, j].unsqueeze(1))
        return {"y": y, "ids": order.int(), "w": p}
    # gradients by the chain rule, expert by expert, the router's last
    ids, w, dy = st["ids"], st["w"].double(), st["dy"].double()
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    out = {n: torch.zeros(v.shape, dtype=torch.float64, device="cuda") for n, v in st["grads"].items()}
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        Wgu, Wd, a, b = st["Wgu"][e].double(), st["Wd"][e].double(), x[t], dy[t]
        gu = (a @ Wgu + st["bgu"][e].double()).requires_grad_()
        with torch.enable_grad():
            gate = torch.where(gu[:, 0::2] > 7, torch.full_like(gu[:, 0::2], 7.0), gu[:, 0::2])
            h = (gu[:, 1::2].clamp(-7, 7) + 1) * gate * torch.sigmoid(1.702 * gate)
        dw[t, j] = ((h.detach() @ Wd + st["bd"][e].double()) * b).sum(dim=1)
        do = b * w[t, j].unsqueeze(1)
        dgu, = torch.autograd.grad(h, gu, do @ Wd.t())
        dx.index_add_(0, t, dgu @ Wgu.t())
        out["dWgu"][e], out["dbgu"][e] = a.t() @ dgu, dgu.sum(dim=0)
        out["dWd"][e], out["dbd"][e] = h.detach().t() @ do, do.sum(dim=0)
    dlogits = torch.zeros((x.shape[0], E), dtype=torch.float64, device="cuda")
    dlogits.scatter_(1, ids.long(), w * dw - w * (w * dw).sum(dim=1, keepdim=True))
    out["dx"] = dx + dlogits @ st["Wr"].double()
    out["dWr"], out["dbr"] = dlogits.t() @ x, dlogits.sum(dim=0)
    return out
