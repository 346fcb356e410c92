"""Measured cases of the expert-layer operators: gate, quantisers, grouped FP8
product, grouped weight gradient, SwiGLU with an 8-bit checkpoint.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs, ``run()``
one pass (the plain torch form, or with ``own`` set the library's calls),
``work()`` the bytes and operations a pass cannot do without and ``exact()``
the result from the definitions in 64 bits.

Rows belong to groups (experts).  ``layout`` says where: "dense" (groups one
behind the other), "aligned" (each group's block rounded up to 128 rows of
which the rest is zero padding) or "static" (group g owns ``cap`` rows from
g*cap, of which the first counts[g] are used).  ``spread`` says how the rows
fall on the groups: "even" (every row picks a group uniformly), "zipf"
(popularity (rank+1)^-1.2, so most rows sit in few groups and some groups are
empty).
"""
import numpy as np
import torch

own = False

_BLOCK = 128


def listed():
    return [
        # the router of a decode batch: 128 tokens, 256 experts; latency alone
        {"name": "gate decode", "op": "gate", "T": 128, "E": 256, "K": 8, "dtype": "float32",
         "score": "sigmoid", "normalize": True, "pad": 0.0},
        # the router of a training step on 16384 tokens with padding, forward and backward
        {"name": "gate training", "op": "gate_train", "T": 16384, "E": 256, "K": 8, "dtype": "bfloat16",
         "score": "softmax", "normalize": True, "pad": 0.05},
        # gradients of the experts' outputs on their way into the backward product
        {"name": "quantise rows", "op": "quant_rows", "R": 32768, "H": 7168, "layout": "dense",
         "G": 32, "spread": "even"},
        # one rank's expert weights after an optimizer step, both orientations
        {"name": "quantise weights", "op": "quant_weights", "G": 32, "N": 4096, "K": 7168,
         "dtype": "bfloat16"},
        # the smallest product: a small model's experts on a handful of tokens
        {"name": "product small", "op": "product", "R": 256, "G": 16, "N": 512, "K": 256,
         "layout": "dense", "spread": "even", "cap": 0},
        # decode on one of 8 ranks: 128 tokens of each of 2 ranks, 32 local experts, static layout
        {"name": "product decode", "op": "product", "R": 256, "G": 32, "N": 4096, "K": 7168,
         "layout": "static", "spread": "even", "cap": 128},
        # skewed routing over 64 experts of a middle-sized model, ragged blocks
        {"name": "product skewed", "op": "product", "R": 24576, "G": 64, "N": 2816, "K": 4096,
         "layout": "dense", "spread": "zipf", "cap": 0},
        # prefill or training on one of 8 ranks: 8192 tokens of each rank, top-8, 32 local experts
        {"name": "product prefill", "op": "product", "R": 65536, "G": 32, "N": 4096, "K": 7168,
         "layout": "aligned", "spread": "even", "cap": 0},
        # weight gradients of a small expert set with few rows each
        {"name": "weight gradient skewed", "op": "wgrad", "R": 4096, "G": 16, "N": 1408, "K": 2048,
         "layout": "dense", "spread": "zipf", "dtype": "bfloat16"},
        # weight gradients of the up projection on one of 8 ranks
        {"name": "weight gradient", "op": "wgrad", "R": 32768, "G": 32, "N": 4096, "K": 7168,
         "layout": "dense", "spread": "even", "dtype": "bfloat16"},
        # the activation between the two products, with the checkpoint for the backward pass
        {"name": "swiglu", "op": "swiglu", "R": 32768, "I": 2048, "G": 32, "layout": "dense",
         "spread": "even", "cap": 0, "checkpoint": True},
        # its backward pass from the 8-bit checkpoint
        {"name": "swiglu backward", "op": "swiglu_back", "R": 32768, "I": 2048, "G": 32,
         "layout": "dense", "spread": "even", "cap": 0},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _m128(rng, lo, hi):
    return max(1, _log(rng, lo, hi) // 128) * 128


def draw(rng):
    op = rng.choice(["gate", "gate_train", "quant_rows", "quant_weights", "product", "product",
                     "product", "wgrad", "wgrad", "swiglu", "swiglu_back"])
    if op in ("gate", "gate_train"):
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "K": rng.randint(1, min(16, E)),
                "dtype": rng.choice(["float32", "bfloat16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "normalize": rng.random() < 0.7,
                "pad": rng.choice([0.0, 0.05, 0.4])}
    if op == "quant_rows":
        return {"op": op, "R": _log(rng, 1, 32768), "H": _m128(rng, 256, 7168),
                "layout": "dense", "G": _log(rng, 1, 256), "spread": rng.choice(["even", "zipf"])}
    if op == "quant_weights":
        return {"op": op, "G": _log(rng, 1, 32), "N": _m128(rng, 128, 4096),
                "K": _m128(rng, 128, 7168), "dtype": rng.choice(["bfloat16", "float32"])}
    spread = rng.choice(["even", "zipf"])
    if op in ("swiglu", "swiglu_back"):
        c = {"op": op, "R": _log(rng, 1, 32768), "I": _m128(rng, 128, 2048), "G": _log(rng, 1, 256),
             "layout": "dense", "spread": spread, "cap": 0}
        if op == "swiglu":
            c["checkpoint"] = rng.random() < 0.5
        return c
    R = _log(rng, 1, 32768 if spread == "even" else 8192)
    G = _log(rng, 1, 64)
    N, K = _m128(rng, 128, 4096), _m128(rng, 128, 7168)
    if op == "wgrad":
        return {"op": op, "R": R, "G": G, "N": N, "K": K, "layout": "dense", "spread": spread,
                "dtype": "bfloat16"}
    layout = rng.choice(["dense", "dense", "aligned", "static"])
    cap = 0
    if layout == "static":
        cap = rng.choice([16, 64, 128, 250])
        R = min(R, max(1, G * cap // 3))
    return {"op": op, "R": R, "G": G, "N": N, "K": K, "layout": layout, "spread": spread, "cap": cap}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _counts(case, seed):
    """Rows of each group: R picks of a group, at most cap in each of a static layout."""
    r = np.random.default_rng([int(seed), 17])
    G, R = case["G"], case["R"]
    p = np.ones(G) if case["spread"] == "even" else (r.permutation(G) + 1.0) ** -1.2
    n = r.multinomial(R, p / p.sum())
    return np.minimum(n, case["cap"]) if case["layout"] == "static" else n


def _groups(case, seed):
    """(used rows of each group, offsets [G+1] that the calls take, first row of each group, rows in all)"""
    n = _counts(case, seed)
    if case["layout"] == "static":
        first, rows = np.arange(case["G"]) * case["cap"], case["G"] * case["cap"]
        off = np.concatenate([[0], np.cumsum(n)])
    else:
        size = (n + 127) // 128 * 128 if case["layout"] == "aligned" else n
        off = np.concatenate([[0], np.cumsum(size)])
        first, rows = off[:-1], int(off[-1])
        if case["layout"] == "aligned":  # the room a dispatch without readback makes
            rows = case["R"] + case["G"] * 127
    return n, off, first, rows


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _to_fp8(x, block_rows):
    """Codes and scales of an input that arrives in 8 bits: blocks of block_rows x 128."""
    s = x.shape
    b = x.reshape(*s[:-2], s[-2] // block_rows, block_rows, s[-1] // _BLOCK, _BLOCK)
    a = b.abs().amax(dim=(-3, -1), keepdim=True).clamp(min=2.0 ** -64)
    q = (b * (448.0 / a)).reshape(s).to(torch.float8_e4m3fn)
    return q, (a / 448.0).squeeze(-1).squeeze(-2).contiguous()


def _rows_fp8(gen, rows, width, used):
    """8-bit rows as dispatch leaves them: rows of different sizes, zero where no token is."""
    x = _normal(gen, rows, width) * torch.exp2(_normal(gen, rows, 1))
    x = torch.where(used[:, None], x, torch.zeros((), device=x.device))
    q, s = _to_fp8(x, 1)
    return q, torch.where(used[:, None], s, torch.zeros((), device=x.device))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 11)
    op = case["op"]
    st = dict(case)
    if op in ("gate", "gate_train"):
        T, E, K = case["T"], case["E"], case["K"]
        dt = getattr(torch, case["dtype"])
        st["logits"] = (_normal(gen, T, E) + 0.5 * _normal(gen, 1, E)).to(dt)
        st["mask"] = None
        if case["pad"]:
            st["mask"] = (torch.rand(T, generator=gen, device=dev) >= case["pad"]).to(torch.uint8)
        st["scale"], st["coef"] = (2.5, 1e-3) if case["score"] == "sigmoid" else (1.0, 1e-2)
        if op == "gate_train":
            st["grad_w"] = _normal(gen, T, K)
            st["grad_loss"] = torch.rand(1, generator=gen, device=dev) + 0.5
        return st
    if op == "quant_weights":
        w = _normal(gen, case["G"], case["N"], case["K"]) * 0.02
        st["w"] = w.to(getattr(torch, case["dtype"]))
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
    used = torch.from_numpy(real).to(dev)
    if op == "quant_rows":
        H = case["H"]
        st["x"] = (_normal(gen, rows, H) * torch.exp2(2 * _normal(gen, rows, 1)) * 1e-3).to(torch.bfloat16)
        return st
    if op == "product":
        N, K = case["N"], case["K"]
        st["x"], st["xs"] = _rows_fp8(gen, rows, K, used)
        st["w"], st["ws"] = _to_fp8(_normal(gen, case["G"], N, K) * 0.02, 128)
        st["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
        return st
    if op == "wgrad":
        N, K = case["N"], case["K"]
        st["x"], st["xs"] = _rows_fp8(gen, rows, K, used)
        st["dy"] = (_normal(gen, rows, N) * 1e-2).to(torch.bfloat16)
        return st
    inner = case["I"]
    if op == "swiglu":
        st["h"] = (_normal(gen, rows, 2 * inner) * torch.exp2(0.5 * _normal(gen, rows, 1))).to(torch.bfloat16)
        return st
    st["ckpt"], st["ckpt_s"] = _rows_fp8(gen, rows, 2 * inner, used)
    st["da"] = (_normal(gen, rows, inner) * 1e-2).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _deq_rows(q, s):
    R, H = q.shape
    return (q.float().view(R, H // _BLOCK, _BLOCK) * s[:, :, None]).view(R, H)


def _deq_weights(q, s):
    G, N, K = q.shape
    return (q.float().view(G, N // _BLOCK, _BLOCK, K // _BLOCK, _BLOCK) * s[:, :, None, :, None]).view(G, N, K)


def _quant_rows(x):
    R, H = x.shape
    b = x.view(R, H // _BLOCK, _BLOCK)
    a = b.abs().amax(dim=-1, keepdim=True).clamp(min=2.0 ** -64)
    return (b * (448.0 / a)).view(R, H).to(torch.float8_e4m3fn), (a / 448.0)[:, :, 0]


def _padded(st):
    """[G, most] row of each group's i-th row, and whether it has one."""
    size = (st["offsets"][1:] - st["offsets"][:-1]).long()
    i = torch.arange(st["most"], device=size.device)
    has = i[None, :] < size[:, None]
    return torch.where(has, st["first"][:, None] + i[None, :], 0), has


def _place(st, rows):
    """Group and place in it of each row (rows of no group: a place that is not used)."""
    r = torch.arange(rows, device=st["offsets"].device)
    g = (torch.searchsorted(st["first"], r, right=True) - 1).clamp(min=0)
    # of groups that begin at the same row, all but the last are empty
    return g, (r - st["first"][g]).clamp(max=st["most"] - 1)


def _scores(st):
    x = st["logits"].float()
    if st["score"] == "softmax":
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        return p, p
    s = 1.0 / (1.0 + torch.exp(-x))
    return s / s.sum(dim=1, keepdim=True), s


def _gate(st):
    E, K = st["E"], st["K"]
    p, r = _scores(st)
    idx = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)[1][:, :K]
    w = torch.gather(r, 1, idx)
    if st["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * st["scale"]
    ok = torch.ones(st["T"], dtype=torch.bool, device=p.device) if st["mask"] is None else st["mask"] != 0
    idx = torch.where(ok[:, None], idx, -1)
    w = torch.where(ok[:, None], w, 0.0)
    p = torch.where(ok[:, None], p, 0.0)
    counts = (idx.reshape(-1, 1) == torch.arange(E, device=p.device)[None, :]).sum(dim=0)
    V = ok.sum().float().clamp(min=1.0)
    f = counts.float() * E / (K * V)
    loss = st["coef"] * (f * (p.sum(dim=0) / V)).sum()
    return idx, w, counts.to(torch.int32), loss.reshape(1), p, r, ok, f / V


def _gate_grad(st, idx, w, p, r, ok, f):
    d = st["coef"] * st["grad_loss"] * f                       # d loss / d p, the same for every token
    g = torch.where(ok[:, None], st["grad_w"] * st["scale"], 0.0)
    at = idx.clamp(min=0)
    sel = torch.gather(r, 1, at)
    if st["normalize"]:
        n = sel.sum(dim=1, keepdim=True)
        g = (g - (g * sel / n).sum(dim=1, keepdim=True)) / n   # d / d score of a chosen expert
    if st["score"] == "softmax":
        full = d[None, :] + torch.zeros_like(p).scatter(1, at, g)
        out = p * (full - (p * full).sum(dim=1, keepdim=True))
    else:
        total = r.sum(dim=1, keepdim=True)
        full = (d[None, :] - (p * d[None, :]).sum(dim=1, keepdim=True)) / total
        full = full + torch.zeros_like(p).scatter(1, at, g)
        out = r * (1.0 - r) * full
    return torch.where(ok[:, None], out, 0.0).to(st["logits"].dtype)


def _plain(st):
    op = st["op"]
    if op in ("gate", "gate_train"):
        idx, w, counts, loss, p, r, ok, f = _gate(st)
        out = {"idx": idx, "weights": w, "counts": counts, "loss": loss}
        if op == "gate_train":
            out["grad"] = _gate_grad(st, idx, w, p, r, ok, f)
        return out
    if op == "quant_rows":
        q, s = _quant_rows(st["x"].float())
        return {"codes": q, "scales": s}
    if op == "quant_weights":
        w = st["w"].float()
        G, N, K = w.shape
        b = w.view(G, N // _BLOCK, _BLOCK, K // _BLOCK, _BLOCK)
        a = b.abs().amax(dim=(2, 4), keepdim=True).clamp(min=2.0 ** -64)
        q = (b * (448.0 / a)).view(G, N, K).to(torch.float8_e4m3fn)
        s = (a / 448.0)[:, :, 0, :, 0]
        return {"codes": q, "scales": s, "codes_t": q.view(torch.uint8).transpose(1, 2).contiguous().view(q.dtype),
                "scales_t": s.transpose(1, 2).contiguous()}
    if op == "product":
        x, w = _deq_rows(st["x"], st["xs"]), _deq_weights(st["w"], st["ws"])
        at, _ = _padded(st)
        y = torch.bmm(x[at], w.transpose(1, 2))
        g, i = _place(st, x.shape[0])
        out = torch.where(st["held"][:, None], y[g, i], 0.0).to(torch.bfloat16)
        return st["out"].copy_(out)
    if op == "wgrad":
        at, has = _padded(st)
        if st["x"].shape[0] == 0:
            return torch.zeros(st["G"], st["N"], st["K"], dtype=torch.bfloat16, device=at.device)
        x = _deq_rows(st["x"], st["xs"])[at] * has[:, :, None]
        dy = st["dy"].float()[at] * has[:, :, None]
        return torch.bmm(dy.transpose(1, 2), x).to(torch.bfloat16)
    if op == "swiglu":
        h = st["h"].float()
        g, u = h[:, :st["I"]], h[:, st["I"]:]
        q, s = _quant_rows(g / (1.0 + torch.exp(-g)) * u)
        out = {"codes": q, "scales": s}
        if st["checkpoint"]:
            out["ckpt"], out["ckpt_scales"] = _quant_rows(h)
        return out
    h = _deq_rows(st["ckpt"], st["ckpt_s"])
    g, u, da = h[:, :st["I"]], h[:, st["I"]:], st["da"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    dh = torch.cat([da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg], dim=1)
    q, s = _quant_rows(dh)
    return {"grad": dh.to(torch.bfloat16), "codes": q, "scales": s}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(st):
    import combine_get_dispatch_scan_amd as ep
    op = st["op"]
    if op in ("gate", "gate_train"):
        g = ep.gate(st["logits"], st["K"], score=st["score"], normalize=st["normalize"], scale=st["scale"],
                    balance_coef=st["coef"], token_mask=st["mask"])
        out = {"idx": g.topk_idx, "weights": g.topk_weights, "counts": g.num_tokens_per_expert, "loss": g.loss}
        if op == "gate_train":
            out["grad"] = ep.gate_backward(st["logits"], g, grad_weights=st["grad_w"], grad_loss=st["grad_loss"])
        return out
    if op == "quant_rows":
        q, s = ep.quantize_rows(st["x"], st["offsets"])
        return {"codes": q, "scales": s}
    if op == "quant_weights":
        w = ep.quantize_weights(st["w"], transposed=True)
        return {"codes": w.codes, "scales": w.scales, "codes_t": w.codes_t, "scales_t": w.scales_t}
    if op == "product":
        return ep.grouped_gemm_fp8(st["x"], st["xs"], st["w"], st["ws"], st["offsets"], group_stride=st["cap"],
                                   expected_rows=st["expected"], out=st["out"])
    if op == "wgrad":
        return ep.grouped_wgrad_fp8(st["dy"], st["x"], st["xs"], st["offsets"])
    if op == "swiglu":
        q, s, ck, cs = ep.swiglu_fp8(st["h"], st["offsets"], checkpoint=st["checkpoint"])
        out = {"codes": q, "scales": s}
        if st["checkpoint"]:
            out["ckpt"], out["ckpt_scales"] = ck, cs
        return out
    dh, q, s = ep.swiglu_fp8_backward(st["da"], st["ckpt"], st["ckpt_s"], st["offsets"])
    return {"grad": dh, "codes": q, "scales": s}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("gate", "gate_train"):
        T, E, K = case["T"], case["E"], case["K"]
        b = 4 if case["dtype"] == "float32" else 2
        if op == "gate":
            return {"bytes": T * E * b + T * K * 12 + E * 4 + 4, "flops": 4 * T * E}
        return {"bytes": 2 * T * E * b + T * K * 16 + E * 4 + 8, "flops": 10 * T * E}
    if op == "quant_weights":
        n = case["G"] * case["N"] * case["K"]
        return {"bytes": n * ((4 if case["dtype"] == "float32" else 2) + 2) + n // 2048, "flops": 2 * n}
    R, G = case["R"], case["G"]
    if op == "quant_rows":
        return {"bytes": R * case["H"] * 3 + R * case["H"] // 32, "flops": 2 * R * case["H"]}
    if op == "product":
        N, K = case["N"], case["K"]
        busy = min(R, G)  # at least: groups that no row picked are not read
        return {"bytes": R * K + R * K // 32 + busy * N * K + busy * N * K // 4096 + 2 * R * N, "flops": 2 * R * N * K}
    if op == "wgrad":
        N, K = case["N"], case["K"]
        return {"bytes": 2 * R * N + R * K + R * K // 32 + 2 * G * N * K, "flops": 2 * R * N * K}
    n = R * case["I"]
    if op == "swiglu":
        return {"bytes": 4 * n + n + n // 32 + (2 * n + n // 16 if case["checkpoint"] else 0), "flops": 8 * n}
    return {"bytes": 2 * n + 2 * n + n // 16 + 4 * n + 2 * n + n // 16, "flops": 14 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(v):
    """The value of an 8-bit float nearest to v (ties to even), 4 exponent and 3 mantissa bits, at most 448."""
    a = v.abs().clamp(min=2.0 ** -30)
    m, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _block_max(v):
    return v.abs().unflatten(-1, (-1, _BLOCK)).amax(-1).clamp(min=2.0 ** -64)


def _exact_rows(v):
    a = _block_max(v)
    return _e4m3(v * (448.0 / a).repeat_interleave(_BLOCK, dim=-1)), a / 448.0


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("gate", "gate_train"):
        x = st["logits"].double()
        T, E, K = case["T"], case["E"], case["K"]
        live = torch.ones(T, dtype=torch.float64, device=x.device) if st["mask"] is None else st["mask"].double()
        soft = case["score"] == "softmax"
        s = torch.softmax(x, 1) if soft else torch.sigmoid(x)
        total = s.sum(1)
        # order by value, then by id
        order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -x.cpu().numpy()), axis=1)[:, :K]
        top = torch.from_numpy(np.ascontiguousarray(order)).to(x.device)
        picked = torch.zeros_like(x).scatter_(1, top, 1.0) * live[:, None]
        chosen_sum = (s * picked).sum(1) + (1.0 - live)
        wn = s * picked / chosen_sum[:, None] if case["normalize"] else s * picked
        weights = st["scale"] * wn.gather(1, top)
        V = max(1.0, float(live.sum()))
        counts = picked.sum(0)
        share = E * counts / (K * V)
        prob = s / total[:, None]
        loss = st["coef"] * (share @ ((prob * live[:, None]).sum(0) / V))
        out = {"idx": torch.where(live[:, None] > 0, top, -1), "weights": weights,
               "counts": counts.long(), "loss": loss.reshape(1)}
        if op == "gate_train":
            gw = torch.zeros_like(x).scatter_(1, top, st["grad_w"].double() * st["scale"]) * picked
            if case["normalize"]:
                ds = picked * (gw - (gw * wn).sum(1, keepdim=True)) / chosen_sum[:, None]
            else:
                ds = gw
            dp = (st["coef"] * float(st["grad_loss"]) / V) * share[None, :] * live[:, None]
            ds = ds + (dp - (dp * prob).sum(1, keepdim=True)) / total[:, None]
            if soft:
                grad = s * (ds - (ds * s).sum(1, keepdim=True))
            else:
                grad = ds * s * (1.0 - s)
            out["grad"] = grad
        return out
    if op == "quant_rows":
        q, s = _exact_rows(st["x"].double())
        return {"codes": q, "scales": s}
    if op == "quant_weights":
        q, s = torch.empty(st["w"].shape, dtype=torch.float64, device="cuda"), []
        for g in range(case["G"]):
            v = st["w"][g].double()
            a = _block_max(v).unflatten(0, (-1, _BLOCK)).amax(1)
            full = a.repeat_interleave(_BLOCK, 0).repeat_interleave(_BLOCK, 1)
            q[g] = _e4m3(v * (448.0 / full))
            s.append(a / 448.0)
        s = torch.stack(s)
        return {"codes": q, "scales": s, "codes_t": q.transpose(1, 2), "scales_t": s.transpose(1, 2)}
    n, off, first, rows = _groups(case, seed)
    spans = [(int(f), int(f + z)) for f, z in zip(first, np.diff(off))]
    if op == "product":
        y = torch.zeros(rows, case["N"], dtype=torch.float64, device="cuda")
        sx = st["xs"].double()
        for g, (a, b) in enumerate(spans):
            if b > a:
                x = st["x"][a:b].double() * sx[a:b].repeat_interleave(_BLOCK, 1)
                w = st["w"][g].double() * st["ws"][g].double().repeat_interleave(_BLOCK, 0).repeat_interleave(_BLOCK, 1)
                y[a:b] = x @ w.T
        return y
    if op == "wgrad":
        d = torch.zeros(case["G"], case["N"], case["K"], dtype=torch.float64, device="cuda")
        for g, (a, b) in enumerate(spans):
            if b > a:
                x = st["x"][a:b].double() * st["xs"][a:b].double().repeat_interleave(_BLOCK, 1)
                d[g] = st["dy"][a:b].double().T @ x
        return d
    inner = case["I"]
    if op == "swiglu":
        h = st["h"].double()
        q, s = _exact_rows(torch.sigmoid(h[:, :inner]) * h[:, :inner] * h[:, inner:])
        out = {"codes": q, "scales": s}
        if case["checkpoint"]:
            out["ckpt"], out["ckpt_scales"] = _exact_rows(h)
        return out
    h = st["ckpt"].double() * st["ckpt_s"].double().repeat_interleave(_BLOCK, 1)
    gate, up, da = h[:, :inner], h[:, inner:], st["da"].double()
    sig = torch.sigmoid(gate)
    dh = torch.cat([da * up * (sig + gate * sig * (1.0 - sig)), da * gate * sig], 1)
    q, s = _exact_rows(dh)
    return {"grad": dh, "codes": q, "scales": s}
