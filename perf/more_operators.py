"""Measured cases of the operators around the expert layer: the norms before and
after a block with its gate and residual scales, their gradients, expert weights
in 4 bits with group scales, and the experts' products with them.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs, ``run()``
one pass (the plain torch form, or with ``own`` set the library's calls),
``work()`` the bytes and operations a pass cannot do without and ``exact()``
the result from the definitions in 64 bits.

Norms: ``x`` is the residual stream and ``y`` a block's output (what combine
returns); ``gate`` multiplies the output per token or per channel; ``offset`` is
added to the norms' weights (1 where they are kept as a difference from one).

Products: rows belong to groups (experts).  ``layout`` says where: "dense"
(groups one behind the other), "aligned" (each group's block rounded up to 128
rows of which the rest is zero padding) or "static" (group g owns ``cap`` rows
from g*cap, of which the first counts[g] are used).  ``spread``: "even" (every
row picks a group uniformly), "zipf" (popularity (rank+1)^-1.2, so most rows sit
in few groups and some groups are empty), "apart" (every row in another group:
the experts of one token).
"""
import numpy as np
import torch

own = False

_BLOCK = 128   # channels of one scale of an 8-bit row
_GROUP = 32    # weights of one scale of 4-bit weights
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token between two layers, its norm in 8 bits for dispatch: latency alone
        {"name": "norm, one token", "op": "norm", "T": 1, "H": 7168, "x": "bfloat16", "w": "bfloat16", "y": True,
         "y_norm": False, "y_weight": False, "gate": "none", "norm": True, "offset": 0.0, "quantize": True},
        # a decode batch of a model with norms on both sides of its blocks
        {"name": "norm, decode", "op": "norm", "T": 128, "H": 4096, "x": "bfloat16", "w": "float32", "y": True,
         "y_norm": True, "y_weight": True, "gate": "token", "norm": True, "offset": 1.0, "quantize": True},
        # prefill or a training step's forward pass
        {"name": "norm, prefill", "op": "norm", "T": 16384, "H": 7168, "x": "bfloat16", "w": "bfloat16", "y": True,
         "y_norm": True, "y_weight": True, "gate": "token", "norm": True, "offset": 0.0, "quantize": True},
        # a residual stream kept in 32 bits, a learned scale of every channel, ragged sizes
        {"name": "norm, 32-bit stream", "op": "norm", "T": 8191, "H": 2056, "x": "float32", "w": "float32", "y": True,
         "y_norm": False, "y_weight": False, "gate": "channel", "norm": True, "offset": 0.0, "quantize": False},
        # gradients of a small model's step
        {"name": "norm backward, small", "op": "norm_back", "T": 509, "H": 1000, "x": "float32", "w": "float32",
         "y": True, "y_norm": True, "y_weight": True, "gate": "channel", "norm": True, "offset": 1.0},
        # gradients of a training step on 16384 tokens
        {"name": "norm backward, training", "op": "norm_back", "T": 16384, "H": 7168, "x": "bfloat16",
         "w": "bfloat16", "y": True, "y_norm": True, "y_weight": True, "gate": "token", "norm": True, "offset": 0.0},
        # a small expert set's weights to 4 bits and back, as a step that trains for them has it
        {"name": "weights, small", "op": "weights", "G": 8, "N": 512, "K": 1024, "w": "float32"},
        # one rank's expert weights
        {"name": "weights", "op": "weights", "G": 32, "N": 4096, "K": 7168, "w": "bfloat16"},
        # one token's eight experts among 32
        {"name": "product, one token", "op": "product", "R": 8, "G": 32, "N": 4096, "K": 7168,
         "layout": "dense", "spread": "apart", "cap": 0},
        # decode on one of 8 ranks: 128 tokens of each of 2 ranks, 32 local experts, static layout
        {"name": "product, decode", "op": "product", "R": 256, "G": 32, "N": 4096, "K": 7168,
         "layout": "static", "spread": "even", "cap": 128},
        # skewed routing over 64 experts of a middle-sized model, ragged blocks
        {"name": "product, skewed", "op": "product", "R": 4096, "G": 64, "N": 2816, "K": 2048,
         "layout": "dense", "spread": "zipf", "cap": 0},
        # prefill on one of 8 ranks: 2048 tokens of each rank, top-8, 32 local experts
        {"name": "product, prefill", "op": "product", "R": 16384, "G": 32, "N": 4096, "K": 7168,
         "layout": "aligned", "spread": "even", "cap": 0},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _multiple(rng, lo, hi, m):
    return max(1, _log(rng, lo, hi) // m) * m


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "norm_back", "weights", "product", "product", "product"])
    if op in ("norm", "norm_back"):
        y = rng.random() < 0.85
        c = {"op": op, "T": _log(rng, 1, 16384), "x": rng.choice(["bfloat16", "bfloat16", "float32"]),
             "w": rng.choice(["bfloat16", "float32"]), "y": y, "y_norm": y and rng.random() < 0.5,
             "y_weight": y and rng.random() < 0.5, "gate": rng.choice(["none", "token", "channel"]) if y else "none",
             "norm": not y or rng.random() < 0.85, "offset": rng.choice([0.0, 1.0])}
        quantize = op == "norm" and c["norm"] and rng.random() < 0.5
        c["H"] = _multiple(rng, 128, 7168, 128 if quantize else 8)
        if c["x"] == "float32":
            c["T"] = max(1, c["T"] // 2)
        if op == "norm":
            c["quantize"] = quantize
        return c
    if op == "weights":
        return {"op": op, "G": _log(rng, 1, 32), "N": _multiple(rng, 128, 4096, 128),
                "K": _multiple(rng, 128, 7168, 128), "w": rng.choice(["bfloat16", "float32"])}
    G = _log(rng, 1, 64)
    N, K = _multiple(rng, 128, 4096, 128), _multiple(rng, 128, 7168, 128)
    spread = rng.choice(["even", "even", "zipf", "apart"])
    if spread == "apart":
        return {"op": op, "R": rng.randint(1, G), "G": G, "N": N, "K": K, "layout": "dense", "spread": spread, "cap": 0}
    R = _log(rng, 1, 8192 if spread == "even" else 2048)
    layout = rng.choice(["dense", "dense", "aligned", "static"])
    cap = 0
    if layout == "static":
        cap = rng.choice([16, 64, 128, 250])
        R = min(R, max(1, G * cap // 3))
    return {"op": op, "R": R, "G": G, "N": N, "K": K, "layout": layout, "spread": spread, "cap": cap}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _counts(case, seed):
    """Rows of each group: R picks of a group, at most cap in each of a static layout."""
    r = np.random.default_rng([int(seed), 23])
    G, R = case["G"], case["R"]
    if case["spread"] == "apart":
        n = np.zeros(G, dtype=np.int64)
        n[r.permutation(G)[:R]] = 1
        return n
    p = np.ones(G) if case["spread"] == "even" else (r.permutation(G) + 1.0) ** -1.2
    n = r.multinomial(R, p / p.sum())
    return np.minimum(n, case["cap"]) if case["layout"] == "static" else n


def _groups(case, seed):
    """(used rows of each group, offsets [G+1] that the calls take, first row of each group, rows in all)"""
    n = _counts(case, seed)
    if case["layout"] == "static":
        return n, np.concatenate([[0], np.cumsum(n)]), np.arange(case["G"]) * case["cap"], case["G"] * case["cap"]
    size = (n + 127) // 128 * 128 if case["layout"] == "aligned" else n
    off = np.concatenate([[0], np.cumsum(size)])
    # an aligned layout's rows: the room a dispatch without readback makes
    return n, off, off[:-1], case["R"] + case["G"] * 127 if case["layout"] == "aligned" else int(off[-1])


def _rows_fp8(gen, rows, width, used):
    """8-bit rows as dispatch leaves them: rows of different sizes, zero where no token is."""
    x = torch.where(used[:, None], _normal(gen, rows, width) * torch.exp2(_normal(gen, rows, 1)), 0.0)
    b = x.view(rows, width // _BLOCK, _BLOCK)
    a = b.abs().amax(dim=-1, keepdim=True).clamp(min=2.0 ** -64)
    q = (b * (448.0 / a)).view(rows, width).to(torch.float8_e4m3fn)
    return q, torch.where(used[:, None], (a / 448.0)[:, :, 0], 0.0)


def _to_fp4(w):
    """4-bit codes (two in a byte, the even k in its low half) and the exponents' bytes of [N, K] fp32 weights."""
    b = w.view(w.shape[0], -1, _GROUP)
    m, e = torch.frexp(b.abs().amax(dim=-1))
    byte = (e + (m >= 0.875) + 124).clamp(0, 254)
    v = torch.ldexp(b, 127 - byte[:, :, None]).view(w.shape)
    a = v.abs()
    code = torch.zeros(w.shape, dtype=torch.uint8, device=w.device)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if up else (a > border)
    code |= torch.signbit(v).to(torch.uint8) << 3
    return code[:, 0::2] | code[:, 1::2] << 4, byte.to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 13)
    op = case["op"]
    st = dict(case)
    if op in ("norm", "norm_back"):
        T, H = case["T"], case["H"]
        xt, wt = getattr(torch, case["x"]), getattr(torch, case["w"])
        # a residual stream has channels that are far larger than the others
        large = torch.where(torch.rand(1, H, generator=gen, device=dev) < 0.005, 20.0, 1.0)
        st["x"] = (_normal(gen, T, H) * large * torch.exp2(_normal(gen, T, 1))).to(xt)
        st["y"] = (_normal(gen, T, H) * 0.3 * torch.exp2(_normal(gen, T, 1))).to(torch.bfloat16) if case["y"] else None
        weight = lambda: (1.0 - case["offset"] + 0.2 * _normal(gen, H)).to(wt)  # noqa: E731
        st["weight"] = weight() if case["norm"] else None
        st["y_weight"] = weight() if case["y_weight"] else None
        st["gate"] = None
        if case["gate"] == "token":
            st["gate"] = torch.rand(T, 1, generator=gen, device=dev)
        elif case["gate"] == "channel":
            st["gate"] = (0.1 + 0.05 * _normal(gen, 1, H)).to(wt)
        st["residual_scale"], st["y_scale"], st["eps"] = (0.75, 1.25, 1e-6) if case["y"] else (1.0, 1.0, 1e-6)
        if op == "norm_back":
            st["grad_x"] = (_normal(gen, T, H) * 1e-2).to(xt)
            st["grad_h"] = (_normal(gen, T, H) * 1e-2).to(torch.bfloat16) if case["norm"] else None
        return st
    if op == "weights":
        w = _normal(gen, case["G"], case["N"], case["K"]) * 0.02
        st["w"] = w.to(getattr(torch, case["w"]))
        return st
    n, off, first, rows = _groups(case, seed)
    st["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
    st["first"] = torch.tensor(first, dtype=torch.int64, device=dev)
    # what the host knows of the groups: the average, and the largest (the plain form pads to it)
    st["expected"] = max(1, -(-case["R"] // case["G"]))
    size = np.diff(off)
    st["most"] = max(1, int(size.max()))
    real = np.zeros(rows, dtype=bool)   # rows that hold a token
    held = np.zeros(rows, dtype=bool)   # rows of a group, padding included
    for f, c, z in zip(first, n, size):
        real[f:f + c] = True
        held[f:f + z] = True
    st["held"] = torch.from_numpy(held).to(dev)
    G, N, K = case["G"], case["N"], case["K"]
    st["xq"], st["xs"] = _rows_fp8(gen, rows, K, torch.from_numpy(real).to(dev))
    st["wq"] = torch.empty(G, N, K // 2, dtype=torch.uint8, device=dev)
    st["ws"] = torch.empty(G, N, K // _GROUP, dtype=torch.uint8, device=dev)
    for g in range(G):
        st["wq"][g], st["ws"][g] = _to_fp4(_normal(gen, N, K) * 0.02)
    st["ws"] = st["ws"].view(torch.float8_e8m0fnu)
    st["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _norm_parts(st):
    """(y's normalised rows, their factors, the weighted ones, the gate, the new stream, its factors)"""
    x = st["x"].float()
    if st["y"] is None:
        z = rz = n = gate = None
        out = x
    else:
        z = st["y"].float()
        rz = 1.0 / torch.sqrt((z * z).mean(dim=1, keepdim=True) + st["eps"]) if st["y_norm"] else None
        z = z * rz if st["y_norm"] else z
        n = z * (st["offset"] + st["y_weight"].float()) if st["y_weight"] is not None else z
        gate = st["gate"].float() if st["gate"] is not None else 1.0
        out = st["residual_scale"] * x + st["y_scale"] * gate * n
    r = 1.0 / torch.sqrt((out * out).mean(dim=1, keepdim=True) + st["eps"])
    return z, rz, n, gate, out, r


def _plain_norm(st):
    _, _, _, _, x, r = _norm_parts(st)
    out = {}
    if st["y"] is not None:
        out["x"] = x.to(st["x"].dtype)
    if st["norm"]:
        h = x * r * (st["offset"] + st["weight"].float())
        out["h"] = h.to(torch.bfloat16)
        if st["quantize"]:
            b = h.view(h.shape[0], -1, _BLOCK)
            a = b.abs().amax(dim=-1, keepdim=True).clamp(min=2.0 ** -64)
            out["codes"] = (b * (448.0 / a)).view(h.shape).to(torch.float8_e4m3fn)
            out["scales"] = (a / 448.0)[:, :, 0]
    return out


def _plain_norm_back(st):
    z, rz, n, gate, x, r = _norm_parts(st)
    out = {}
    g = st["grad_x"].float()
    if st["norm"]:
        gh, xh = st["grad_h"].float(), x * r
        d = gh * (st["offset"] + st["weight"].float())
        g = g + r * (d - xh * (d * xh).mean(dim=1, keepdim=True))
        out["weight"] = (gh * xh).sum(dim=0).to(st["weight"].dtype)
    out["x"] = (st["residual_scale"] * g).to(st["x"].dtype)
    if z is None:
        return out
    e = st["y_scale"] * g
    if st["gate"] is not None:
        out["gate"] = (e * n).sum(dim=1 if st["gate"].shape[1] == 1 else 0, keepdim=True).to(st["gate"].dtype)
    d = e * gate
    if st["y_weight"] is not None:
        out["y_weight"] = (d * z).sum(dim=0).to(st["y_weight"].dtype)
        d = d * (st["offset"] + st["y_weight"].float())
    if st["y_norm"]:
        d = rz * (d - z * (d * z).mean(dim=1, keepdim=True))
    out["y"] = d.to(torch.bfloat16)
    return out


def _plain_weights(st):
    w = st["w"].float()
    b = w.view(*w.shape[:-1], -1, _GROUP)
    m, e = torch.frexp(b.abs().amax(dim=-1))
    k = (e + (m >= 0.875) - 3).clamp(-127, 127)   # the smallest power of two that leaves |values| below 7
    v = torch.ldexp(b, -k[..., None])
    a = v.abs()
    # the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6; ties to the even code
    half = torch.round(a * 2.0) * 0.5
    near = torch.where(a < 2.0, half, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0).clamp(max=6.0))
    scale = torch.ldexp(torch.ones_like(m), k)
    return {"values": (torch.copysign(near, v) * scale[..., None]).view(w.shape).to(torch.bfloat16),
            "scales": scale.to(torch.float8_e8m0fnu)}


def _deq_weights(wq, ws):
    """4-bit weights as fp32 [G, N, K]."""
    G, N, K2 = wq.shape
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=wq.device)
    v = torch.stack([table[(wq & 15).int()], table[(wq >> 4).int()]], dim=-1)
    return (v.view(G, N, -1, _GROUP) * ws.float()[..., None]).view(G, N, 2 * K2)


def _plain_product(st):
    rows, K = st["xq"].shape
    x = (st["xq"].float().view(rows, -1, _BLOCK) * st["xs"][:, :, None]).view(rows, K)
    w = _deq_weights(st["wq"], st["ws"])
    size = (st["offsets"][1:] - st["offsets"][:-1]).long()
    i = torch.arange(st["most"], device=x.device)
    at = torch.where(i[None, :] < size[:, None], st["first"][:, None] + i[None, :], 0)
    y = torch.bmm(x[at], w.transpose(1, 2))
    # group and place in it of each row; of groups that begin at the same row, all but the last are empty
    r = torch.arange(rows, device=x.device)
    g = (torch.searchsorted(st["first"], r, right=True) - 1).clamp(min=0)
    place = (r - st["first"][g]).clamp(max=st["most"] - 1)
    return st["out"].copy_(torch.where(st["held"][:, None], y[g, place], 0.0).to(torch.bfloat16))


def _plain(st):
    op = st["op"]
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_back":
        return _plain_norm_back(st)
    if op == "weights":
        return _plain_weights(st)
    return _plain_product(st)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(st):
    import combine_get_dispatch_scan_amd as ep
    op = st["op"]
    if op in ("norm", "norm_back"):
        how = dict(norm=st["norm"], weight=st["weight"], y_norm=st["y_norm"], y_weight=st["y_weight"], gate=st["gate"],
                   residual_scale=st["residual_scale"], y_scale=st["y_scale"], eps=st["eps"], weight_offset=st["offset"])
        if op == "norm":
            o = ep.block_norm(st["x"], st["y"], quantize=st["quantize"], **how)
            out = {"x": o.x} if st["y"] is not None else {}
            if st["norm"]:
                out["h"] = o.h
            if st["quantize"]:
                out["codes"], out["scales"] = o.codes, o.scales
            return out
        o = ep.block_norm_backward(st["x"], st["y"], grad_x=st["grad_x"], grad_h=st["grad_h"], **how)
        out = {"x": o.x, "y": o.y, "weight": o.weight, "y_weight": o.y_weight, "gate": o.gate}
        return {k: v for k, v in out.items() if v is not None}
    if op == "weights":
        q = ep.quantize_weights_fp4(st["w"])
        return {"values": ep.dequantize_weights_fp4(q), "scales": q.scales}
    return ep.grouped_gemm_fp4(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], group_stride=st["cap"],
                               expected_rows=st["expected"], out=st["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        n, H = case["T"] * case["H"], case["H"]
        b, wb = (4 if case[k] == "float32" else 2 for k in ("x", "w"))
        params = (case["norm"] + case["y_weight"] + (case["gate"] == "channel")) * H * wb
        params += 4 * case["T"] * (case["gate"] == "token")
        if op == "norm":
            per = b + (2 + b if case["y"] else 0) + (2 if case["norm"] else 0) + (1 + 1 / 32 if case["quantize"] else 0)
            return {"bytes": n * per + params, "flops": 10 * n}
        per = 3 * b + (4 if case["y"] else 0) + (2 if case["norm"] else 0)
        return {"bytes": n * per + 2 * params, "flops": 30 * n}
    if op == "weights":
        n = case["G"] * case["N"] * case["K"]
        return {"bytes": n * ((4 if case["w"] == "float32" else 2) + 2) + n // 32, "flops": 4 * n}
    R, G, N, K = case["R"], case["G"], case["N"], case["K"]
    busy = min(R, G)  # at least: groups that no row picked are not read
    return {"bytes": R * K + R * K // 32 + busy * N * K // 2 + busy * N * K // 32 + 2 * R * N, "flops": 2 * R * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e2m1(v):
    """The value of a 4-bit float nearest to v (ties to even), 2 exponent bits and 1 mantissa bit, at most 6."""
    m, e = torch.frexp(v.abs().clamp(min=2.0 ** -60))
    step = torch.ldexp(torch.ones_like(m), (e - 1).clamp(min=0) - 1)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _exact_norm(st, x, y, weight, y_weight, gate):
    s = x
    if y is not None:
        b = y
        if st["y_norm"]:
            b = b * (b.square().mean(1, True) + st["eps"]).rsqrt()
        if y_weight is not None:
            b = b * (y_weight + st["offset"])
        if gate is not None:
            b = b * gate
        s = x * st["residual_scale"] + b * st["y_scale"]
    h = s * (s.square().mean(1, True) + st["eps"]).rsqrt() * (weight + st["offset"]) if weight is not None else None
    return s, h


def exact(case, seed):
    op = case["op"]
    if op == "product" and 2.0 * case["R"] * case["N"] * case["K"] > 1.1e15:
        return None
    st = prepare(case, seed)
    if op in ("norm", "norm_back"):
        names = ["x", "y", "weight", "y_weight", "gate"]
        v = {k: st[k].double() if st[k] is not None else None for k in names}
        if op == "norm":
            s, h = _exact_norm(st, **v)
            out = {"x": s} if case["y"] else {}
            if case["norm"]:
                out["h"] = h
            if case["quantize"]:
                top = h.unflatten(1, (-1, _BLOCK)).abs().amax(2).clamp(min=2.0 ** -64)
                out["codes"] = h * (448.0 / top).repeat_interleave(_BLOCK, 1)   # as h: not rounded
                out["scales"] = top / 448.0
            return out
        leaves = [k for k in names if v[k] is not None]
        for k in leaves:
            v[k].requires_grad_()
        s, h = _exact_norm(st, **v)
        into = [(o, g.double()) for o, g in ((s, st["grad_x"]), (h, st["grad_h"])) if g is not None]
        grads = torch.autograd.grad([o for o, _ in into], [v[k] for k in leaves], [g for _, g in into])
        return dict(zip(leaves, grads))
    if op == "weights":
        values = torch.empty(st["w"].shape, dtype=torch.float64, device="cuda")
        scales = []
        for g in range(case["G"]):
            w = st["w"][g].double()
            top = w.unflatten(1, (-1, _GROUP)).abs().amax(2)
            s = torch.exp2(torch.floor(torch.log2(top)) - 2.0)
            s = torch.where(top >= 7.0 * s, 2.0 * s, s).clamp(min=2.0 ** -127)
            full = s.repeat_interleave(_GROUP, 1)
            values[g] = _e2m1(w / full) * full
            scales.append(s)
        return {"values": values, "scales": torch.stack(scales)}
    n, off, first, rows = _groups(case, seed)
    y = torch.zeros(rows, case["N"], dtype=torch.float64, device="cuda")
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    for g, (f, z) in enumerate(zip(first, np.diff(off))):
        if z > 0:
            a, b = int(f), int(f + z)
            x = st["xq"][a:b].double() * st["xs"][a:b].double().repeat_interleave(_BLOCK, 1)
            q = torch.empty(case["N"], case["K"], dtype=torch.int64, device="cuda")
            q[:, 0::2], q[:, 1::2] = st["wq"][g].long() % 16, st["wq"][g].long() // 16
            w = torch.where(q >= 8, -grid[q % 8], grid[q % 8]) * st["ws"][g].double().repeat_interleave(_GROUP, 1)
            y[a:b] = x @ w.T
    return y
