"""GPU checks of the norms around a block and of 4-bit expert weights against their
formulas in 64 bits.

Tolerances count roundings.  u = 2^-24 is fp32's half step; bf16 rounds by at most
2^-8, E4M3 by 2^-4 of a value.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
BF = torch.bfloat16


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _randn(g, *s):
    return torch.randn(s, generator=g, device=g.device)


# ----------------------------------------------------------------------------
# norms
# ----------------------------------------------------------------------------

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
# Relative error of a row's factor 1 / sqrt(mean + eps): a sum of squares over at most 32 values of a lane, 6 levels of
# a wave and 16 waves (54 roundings, every term positive), times 1 / width, plus eps, half of that for the root, whose
# own error is one step (2 u).  A product of it with up to six factors adds 2 u for each.
C = 48 * U


def _norm_case(seed, T, H, xt=BF, wt=BF, y=True, y_norm=True, y_weight=True, weight=True, gate="token", gt=torch.float32,
               offset=0.0, a=0.75, b=1.25, pad=0):
    """Inputs and options of a block norm; pad: extra elements between rows."""
    g = _gen(seed)
    row = lambda dt, s: (_randn(g, T, H + pad) * s * torch.exp2(2 * _randn(g, T, 1))).to(dt)[:, :H]  # noqa: E731
    o = dict(x=row(xt, 1.0), y=row(BF, 0.5) if y else None)
    if y and T > 2:
        o["y"][T // 2] = 0                       # a token none of whose pairs were dispatched
    w = lambda: (1 - offset + 0.3 * _randn(g, H)).to(wt)  # noqa: E731
    o["weight"] = w() if weight else None
    o["y_weight"] = w() if y and y_weight else None
    o["y_norm"] = bool(y and y_norm)
    o["gate"] = None
    if y and gate == "token":
        o["gate"] = _randn(g, T, 1).to(gt)
    elif y and gate == "channel":
        o["gate"] = _randn(g, 1, H).to(gt)
    o["residual_scale"], o["y_scale"] = (a, b) if y else (1.0, b)
    o["eps"], o["weight_offset"] = 1e-5, offset
    return o


def _norm64(o, norm=True):
    """Every quantity of the forward pass in 64 bits, with the magnitude X of x' (its terms' absolute values added)."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, eps, off = d(o["x"]), o["eps"], o["weight_offset"]
    H = x.shape[1]
    f = {}
    # options arrive as fp32
    a, b, eps, off = (float(np.float32(v)) for v in (o["residual_scale"], o["y_scale"], eps, off))
    f["a"], f["b"], f["off"] = a, b, off
    if o["y"] is None:
        f["v"], f["X"] = x, x.abs()
        f["t2"] = torch.zeros_like(x)
    else:
        y = d(o["y"])
        f["rz"] = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if o["y_norm"] else torch.ones_like(y[:, :1])
        f["z"] = y * f["rz"]
        f["wy"] = off + d(o["y_weight"]) if o["y_weight"] is not None else torch.ones(H, dtype=torch.float64, device=x.device)
        f["gate"] = d(o["gate"]) if o["gate"] is not None else torch.ones(1, 1, dtype=torch.float64, device=x.device)
        f["t2"] = b * f["gate"] * f["z"] * f["wy"]
        # o + w may cancel: its rounding is one of the larger of the two
        f["v"], f["X"] = a * x + f["t2"], (a * x).abs() + f["t2"].abs()
    f["r"] = 1 / torch.sqrt((f["v"] ** 2).mean(1, keepdim=True) + eps)
    f["w"] = off + d(o["weight"]) if o["weight"] is not None else torch.ones(H, dtype=torch.float64, device=x.device)
    # by how much an error of X's size in x' moves r
    f["kap"] = 1 + (f["X"] ** 2).mean(1, keepdim=True) * f["r"] ** 2
    return f


def _check_norm(ep, o, norm=True, quantize=False):
    f = _norm64(o, norm)
    n = ep.block_norm(norm=norm, quantize=quantize, **o)
    xt = o["x"].dtype
    if o["y"] is None:
        assert n.x is o["x"]
    else:
        assert n.x.dtype == xt and ((n.x.double() - f["v"]).abs() <= C * f["X"] + (HALF[xt] + U) * f["v"].abs()).all()
    if not norm:
        assert n.h is None and n.codes is None
        return n
    h = f["v"] * f["r"] * f["w"]
    tol = C * (f["X"] * f["r"] * f["w"].abs() + 2 * f["kap"] * h.abs())
    assert n.h.dtype == BF and ((n.h.double() - h).abs() <= tol + 2.0 ** -8 * (h.abs() + tol) + 2.0 ** -134).all()
    if quantize:
        T, H = h.shape
        top, ttop = (t.view(T, H // 128, 128).amax(2) for t in (h.abs(), tol))
        top = top.clamp(min=2.0 ** -64)                    # the scale's rounding is one of this quotient
        s = n.scales.double()
        assert ((s - top / 448).abs() <= (ttop + 4 * U * top) / 448).all()
        full = s.repeat_interleave(128, 1)
        got = n.codes.double() * full
        # half a step of E4M3, or of its subnormals (2^-10 of the scale), and the scale's own error
        assert ((got - h).abs() <= tol + (2.0 ** -4 + 8 * U) * (h.abs() + tol) + 2.0 ** -10 * full).all()
    return n


def _check_norm_backward(ep, o, seed=0, norm=True, with_gx=True, with_gh=True):
    f = _norm64(o, norm)
    T, H = o["x"].shape
    g = _gen(seed + 500)
    gx = (_randn(g, T, H) * 0.1).to(o["x"].dtype) if with_gx else None
    gh = (_randn(g, T, H)).to(BF) if norm and with_gh else None
    q = ep.block_norm_backward(grad_x=gx, grad_h=gh, norm=norm, **o)
    zero = torch.zeros(T, H, dtype=torch.float64, device=o["x"].device)
    G, M = (gx.double(), gx.double().abs()) if gx is not None else (zero, zero)
    E = zero                                               # error of g
    r, kap = f["r"], f["kap"]
    # a sum over tokens: the rows of a workgroup (256 of them or more share the rows; four waves meet when narrow), up to
    # eight workgroups of a share, four shares of a wave, sixteen waves
    depth = T / 256 + 1 + 4 + 8 + 4 + 16
    if gh is not None:
        ghd = gh.double()
        d, xh, Xh = ghd * f["w"], f["v"] * r, f["X"] * r
        # w's own rounding (o + w) is one more u of each term
        D = ghd.abs() * (f["w"].abs() + U * abs(f["off"]))
        G = G + r * (d - xh * (d * xh).mean(1, keepdim=True))
        M = M + r * (D + Xh * (D * Xh).mean(1, keepdim=True))
        E = C * (1 + 4 * kap) * M
        if o["weight"] is not None:
            want, mag = (ghd * xh).sum(0), (ghd.abs() * Xh)
            tol = (C * (1 + kap) * mag).sum(0) + depth * U * mag.sum(0)
            assert q.weight.dtype == o["weight"].dtype
            assert ((q.weight.double() - want).abs() <= tol + HALF[q.weight.dtype] * (want.abs() + tol)).all()
    a, b = f["a"], f["b"]
    assert q.x.dtype == o["x"].dtype
    assert ((q.x.double() - a * G).abs() <= a * E + 2 * U * a * M + HALF[q.x.dtype] * (abs(a) * (G.abs() + E)) + 1e-40).all()
    if o["y"] is None:
        assert q.y is None and q.gate is None and q.y_weight is None
        return q
    fy = b * f["wy"] * (f["gate"] if o["gate"] is not None and o["gate"].shape[0] == 1 and o["gate"].shape[1] == H else 1.0)
    FY = abs(b) * (f["wy"].abs() + U * abs(f["off"])) * (fy / (b * f["wy"])).abs() if torch.is_tensor(fy) else abs(fy)
    fy = fy.expand(T, H) if fy.dim() == 2 else fy
    token = o["gate"] is not None and o["gate"].shape == (T, 1)
    gt = f["gate"] if token else torch.ones(1, 1, dtype=torch.float64, device=zero.device)
    z, rz = f["z"], f["rz"]
    s = (G * fy * z).sum(1, keepdim=True)
    es = ((E + C * M) * fy.abs() * z.abs()).sum(1, keepdim=True)
    if token:
        want, tol = s, es
    elif o["gate"] is not None:
        mag = b * M * z.abs() * f["wy"].abs()
        want = (b * G * z * f["wy"]).sum(0, keepdim=True)
        tol = (b * (E + C * M) * (z * f["wy"]).abs() + depth * U * mag).sum(0, keepdim=True)
    if o["gate"] is not None:
        assert q.gate.shape == o["gate"].shape and q.gate.dtype == o["gate"].dtype
        assert ((q.gate.double() - want).abs() <= tol + HALF[q.gate.dtype] * (want.abs() + tol) + 1e-40).all()
    if o["y_weight"] is not None:
        e2 = b * G * f["gate"]
        mag = b * M * f["gate"].abs() * z.abs()
        want = (e2 * z).sum(0)
        tol = (b * (E + C * M) * f["gate"].abs() * z.abs() + depth * U * mag).sum(0)
        assert q.y_weight.dtype == o["y_weight"].dtype
        assert ((q.y_weight.double() - want).abs() <= tol + HALF[q.y_weight.dtype] * (want.abs() + tol) + 1e-40).all()
    want = G * fy * gt
    tol = (E + C * M) * fy.abs() * gt.abs()
    if o["y_norm"]:
        want = rz * (want - z * gt * s / H)
        S = (M * fy.abs() * z.abs()).sum(1, keepdim=True)
        tol = rz * (tol + (z * gt).abs() * (es + C * S) / H + C * ((M * fy * gt).abs() + (z * gt).abs() * S / H))
    assert q.y.dtype == BF and ((q.y.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38).all()
    return q


# the widths of every team: a wave with one and two vectors, workgroups with one, two (to 512 and to 1024 threads), four
WIDTHS = [8, 136, 512, 520, 1000, 1024, 1032, 2048, 2056, 5120, 7168, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("xt", [BF, torch.float32])
def test_block_norm_widths(ep, H, xt):
    for T in (1, 37):
        o = _norm_case(H + T, T, H, xt, torch.float32 if H % 3 else BF, gate="token" if H % 5 else "channel")
        _check_norm(ep, o, quantize=H % 128 == 0)
        _check_norm_backward(ep, o, H)


@pytest.mark.parametrize("T,H", [(5, 264), (700, 1024), (1500, 640)])
@pytest.mark.parametrize("y,y_norm,y_weight,gate,norm", [
    (False, False, False, "none", True), (True, False, False, "none", True), (True, False, False, "none", False),
    (True, True, False, "token", True), (True, True, True, "channel", True), (True, False, True, "channel", False),
    (True, False, True, "token", False), (True, True, True, "none", False),
])
@pytest.mark.parametrize("offset,wt", [(0.0, torch.float32), (1.0, BF)])
def test_block_norm_forms(ep, T, H, y, y_norm, y_weight, gate, norm, offset, wt):
    o = _norm_case(T, T, H, BF, wt, y, y_norm, y_weight, norm, gate, torch.float32 if offset else BF, offset)
    _check_norm(ep, o, norm, quantize=norm and H % 128 == 0)
    _check_norm_backward(ep, o, T, norm)


def test_block_norm_without_weights_and_gradients_in_part(ep):
    o = _norm_case(1, 40, 384, weight=False, y_weight=False, gate="token", gt=BF)
    _check_norm(ep, o, quantize=True)
    _check_norm_backward(ep, o)
    o = _norm_case(2, 40, 384, torch.float32, torch.float32, gate="channel", gt=torch.float32)
    _check_norm_backward(ep, o, 1, with_gx=False)
    _check_norm_backward(ep, o, 2, with_gh=False)      # the norm's weight gets a zero gradient
    q = ep.block_norm_backward(grad_x=o["x"], **o)
    assert not q.weight.any()
    full = ep.block_norm_backward(grad_x=o["x"], grad_h=o["y"], **o)
    for name in ("x", "y", "weight", "y_weight", "gate"):
        q = ep.block_norm_backward(grad_x=o["x"], grad_h=o["y"], need=(name,), **o)
        for other in ("x", "y", "weight", "y_weight", "gate"):
            assert (getattr(q, other) is None) == (other != name)
        assert torch.equal(getattr(q, name), getattr(full, name))


def test_block_norm_strided_rows_in_place_and_outputs_in_part(ep):
    o = _norm_case(3, 50, 640, pad=136)
    assert o["x"].stride(0) == 776
    n = _check_norm(ep, o, quantize=True)
    _check_norm_backward(ep, o)
    dense = dict(o, x=o["x"].contiguous(), y=o["y"].contiguous())
    m = ep.block_norm(quantize=True, **dense)
    for k in ("x", "h", "codes", "scales"):
        assert torch.equal(getattr(n, k).view(torch.uint8), getattr(m, k).view(torch.uint8))
    m = ep.block_norm(quantize=True, write_h=False, **dense)
    assert m.h is None and torch.equal(m.codes.view(torch.uint8), n.codes.view(torch.uint8))
    x = dense["x"].clone()
    m = ep.block_norm(**dict(dense, x=x), x_out=x)
    assert m.x is x and torch.equal(x, n.x) and torch.equal(m.h, n.h)
    gx = dense["x"].clone()
    q = ep.block_norm_backward(grad_x=gx, grad_h=dense["y"], **dense)
    want = ep.block_norm_backward(grad_x=dense["x"], grad_h=dense["y"], **o)
    assert torch.equal(q.x, want.x) and torch.equal(q.weight, want.weight)


def test_block_norm_rows_of_zeros_and_odd_rows(ep):
    """Zeros stay finite; a row with NaN or infinities touches no other row's outputs."""
    o = _norm_case(4, 33, 256, gate="token")
    o["x"][3] = 0
    o["y"][3] = 0
    n = _check_norm(ep, o, quantize=True)
    assert not n.x[3].any() and not n.h[3].any() and (n.scales[3] == float(np.float32(2.0 ** -64) / np.float32(448))).all()
    gx, gh = o["x"].clone(), o["y"].clone()
    q = ep.block_norm_backward(grad_x=gx, grad_h=gh, **o)
    bad = dict(o, x=o["x"].clone(), y=o["y"].clone())
    bad["x"][7, 3], bad["x"][9, 5], bad["y"][11, 200] = math.nan, math.inf, -math.inf
    m = ep.block_norm(quantize=True, **bad)
    p = ep.block_norm_backward(grad_x=gx, grad_h=gh, **bad)
    keep = [t for t in range(33) if t not in (7, 9, 11)]
    for k in ("x", "h", "codes", "scales"):
        assert torch.equal(getattr(m, k).view(torch.uint8)[keep], getattr(n, k).view(torch.uint8)[keep])
    assert torch.equal(p.x[keep], q.x[keep]) and torch.equal(p.y[keep], q.y[keep]) and torch.equal(p.gate[keep], q.gate[keep])
    assert torch.isnan(m.x[7, 3]) and torch.isnan(m.h[7]).all() and torch.isnan(p.weight).any()


def test_block_norm_without_rows(ep):
    dev = _dev()
    e = torch.empty(0, 256, dtype=BF, device=dev)
    w = torch.ones(256, dtype=torch.float32, device=dev)
    n = ep.block_norm(e, e.clone(), weight=w, y_weight=w, gate=torch.empty(0, 1, device=dev), quantize=True)
    assert n.x.shape == n.h.shape == n.codes.shape == (0, 256) and n.scales.shape == (0, 2)
    q = ep.block_norm_backward(e, e.clone(), grad_x=e, grad_h=e, weight=w, y_weight=w, gate=torch.ones(1, 256, device=dev))
    assert q.x.shape == (0, 256) and not q.weight.any() and not q.y_weight.any() and not q.gate.any()


def test_block_norm_repeats_and_reused_workspace(ep):
    o = _norm_case(6, 3000, 512, gate="channel", gt=torch.float32, wt=torch.float32)
    gx, gh = o["x"] * 0.1, o["y"] * 0.1
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(3000, 512), dtype=torch.uint8, device=_dev())
    a = ep.block_norm_backward(grad_x=gx, grad_h=gh, **o)
    ws.fill_(255)
    for _ in range(3):
        b = ep.block_norm_backward(grad_x=gx, grad_h=gh, ws=ws, **o)
        for k in ("x", "y", "weight", "y_weight", "gate"):
            assert torch.equal(getattr(a, k), getattr(b, k))


@pytest.mark.parametrize("gate,y_norm", [("token", True), ("channel", True), ("channel", False)])
def test_block_norm_gradient_against_differences(ep, gate, y_norm):
    """Directional derivatives of the forward pass in 32 bits against the backward pass.

    The loss is linear in x', whose fp32 values are off by C X; with a step of 2^-6 in each input the difference
    quotient's own error is of second order in the step (checked to 2^-5 of the gradients' size)."""
    o = _norm_case(8, 24, 64, torch.float32, torch.float32, gate=gate, y_norm=y_norm)
    g = _gen(9)
    gx = _randn(g, 24, 64)
    q = ep.block_norm_backward(grad_x=gx, norm=False, **dict(o, weight=None))
    for name in ("x", "y_weight", "gate"):
        d = _randn(g, *o[name].shape)
        h = 2.0 ** -6
        loss = []
        for sign in (1, -1):
            p = dict(o, weight=None)
            p[name] = (o[name].double() + sign * h * d.double()).to(o[name].dtype)
            loss.append(float((ep.block_norm(norm=False, **p).x.double() * gx.double()).sum()))
        # x' is linear in each of these three: only roundings (of x', and of the moved inputs) are left
        want = (loss[0] - loss[1]) / (2 * h)
        got = float((getattr(q, name).double() * d.double()).sum())
        f = _norm64(o, False)
        tol = 2 * float((gx.double().abs() * (C + 4 * U) * (f["X"] + 8)).sum()) / (2 * h) + 1e-4 * abs(got)
        assert abs(got - want) <= tol, (name, got, want, tol)


def test_block_norm_gradient_of_the_norms_against_differences(ep):
    """Of h towards x and of x' towards y, where the function is not linear: the plain formula in 64 bits is differenced
    (its error is h^2) and the backward pass compared with it."""
    o = _norm_case(10, 6, 40, torch.float32, torch.float32, gate="token")
    g = _gen(11)
    gx, gh = _randn(g, 6, 40), _randn(g, 6, 40).to(BF)
    q = ep.block_norm_backward(grad_x=gx, grad_h=gh, **o)

    def loss(p):
        f = _norm64(p)
        return float((f["v"] * gx.double()).sum() + (f["v"] * f["r"] * f["w"] * gh.double()).sum())

    for name in ("x", "y", "weight", "y_weight", "gate"):
        base = o[name].double()
        d = _randn(g, *base.shape).double()
        if name == "y":
            d[3] = 0                             # the row of zeros: its factor is steep there
        h = 1e-5
        want = (loss(dict(o, **{name: base + h * d})) - loss(dict(o, **{name: base - h * d}))) / (2 * h)
        got = float((getattr(q, name).double() * d).sum())
        size = float((getattr(q, name).double() * d).abs().sum())
        step = 2.0 ** -8 if name == "y" else 64 * C
        assert abs(got - want) <= step * size + 1e-6 * abs(want), (name, got, want)


@pytest.mark.parametrize("T,H", [(3000, 4096), (9500, 7168)])
def test_block_norm_of_many_rows_is_that_of_few(ep, T, H):
    """Outputs of 49 and 272 MB are stored in other ways than those of up to 16 MB; a row's bits do not depend on it."""
    o = _norm_case(12, T, H)
    n = ep.block_norm(quantize=True, **o)
    for a in (0, 1000, T - 500):
        part = slice(a, a + 500)
        m = ep.block_norm(quantize=True, **dict(o, **{k: o[k][part] for k in ("x", "y", "gate")}))
        for k in ("x", "h", "codes", "scales"):
            assert torch.equal(getattr(n, k)[part].view(torch.uint8), getattr(m, k).view(torch.uint8)), (a, k)


def test_block_norm_binding_refusals(ep):
    dev = _dev()
    x = torch.zeros(4, 256, dtype=BF, device=dev)
    w = torch.zeros(256, dtype=BF, device=dev)
    cases = [
        (dict(x=x.half()), TypeError, "x must"), (dict(x=x[0]), ValueError, "matrix"), (dict(x=x.t()), ValueError, "contiguous"),
        (dict(x=x[:1].expand(4, 256)), ValueError, "stride"), (dict(x=x[:, :250]), ep.EpError, "width"),
        (dict(x=torch.zeros(4, 260, dtype=BF, device=dev)[:, :256]), ValueError, "stride"),
        (dict(y=x.float()), TypeError, "y must"), (dict(y=x[:3]), ValueError, "y must"), (dict(y=x.cpu()), ValueError, "device"),
        (dict(weight=w[:255]), ValueError, "weight must"), (dict(weight=w.half()), TypeError, "weight must"),
        (dict(y=x, weight=w, y_weight=w.float()), TypeError, "one type"), (dict(y=x, y_weight=w[None]), ValueError, "y_weight"),
        (dict(y=x, gate=w), ValueError, "gate must"), (dict(y=x, gate=x[:2, :1]), ValueError, "gate must"),
        (dict(y=x, gate=x[:, :1].half()), TypeError, "gate"), (dict(y=x, gate=x[:, :1]), ValueError, "contiguous"),
        (dict(y_norm=True), ValueError, "need y"), (dict(gate=x[:, :1]), ValueError, "need y"),
        (dict(residual_scale=0.5), ValueError, "need y"), (dict(norm=False), ValueError, "without y"),
        (dict(y=x, norm=False, weight=w), ValueError, "weight needs"), (dict(y=x, norm=False, quantize=True), ValueError, "quantize"),
        (dict(x_out=x), ValueError, "x_out needs"), (dict(y=x, x_out=x.float()), TypeError, "x_out"),
        (dict(y=x, x_out=x[:3]), ValueError, "x_out"),
    ]
    for kw, err, msg in cases:
        with pytest.raises(err, match=msg):
            ep.block_norm(**{"x": x, **kw})
    with pytest.raises(ep.EpError, match="eps"):
        ep.block_norm(x, eps=0.0)
    with pytest.raises(ep.EpError, match="multiple of 128"):
        ep.block_norm(x[:, :200].contiguous(), quantize=True)
    for kw, err, msg in [(dict(grad_x=x.float()), TypeError, "grad_x"), (dict(grad_h=x.float()), TypeError, "grad_h"),
                         (dict(grad_h=x[:2]), ValueError, "grad_h"), (dict(grad_x=x[:, ::2]), ValueError, "grad_x"),
                         (dict(need=("z",)), ValueError, "need"), (dict(y=x, norm=False, grad_h=x), ValueError, "grad_h needs"),
                         (dict(grad_h=x, weight=w, ws=torch.empty(8, dtype=torch.uint8, device=dev)), ep.EpError, "too small")]:
        with pytest.raises(err, match=msg):
            ep.block_norm_backward(**{"x": x, **kw})


# ----------------------------------------------------------------------------
# 4-bit weights
# ----------------------------------------------------------------------------

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _fp4_64(w):
    """Codes and exponents' bytes of [.., K] weights, in 64 bits on the CPU."""
    v = w.double().cpu().numpy()
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2
    e = np.where(top >= 7 * np.exp2(e), e + 1, e)
    e = np.where(top > 0, np.maximum(e, -127), -127)
    a = np.abs(b) / np.exp2(e)[..., None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    low = np.searchsorted(mid, a, side="left")             # a tie stays below
    tie = (low < 7) & (a == mid[np.minimum(low, 6)])
    code = np.where(tie & (low % 2 == 1), low + 1, low)    # ... and goes to the even code
    return (code | (np.signbit(b) * 8)).reshape(v.shape), (e + 127).astype(np.int64)


def _unpack(codes):
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)


def _values(codes, byte):
    c = np.asarray(codes)
    v = np.where(c >= 8, -GRID[c & 7], GRID[c & 7])
    return (v.reshape(*c.shape[:-1], -1, 32) * np.exp2(byte - 127.0)[..., None]).reshape(c.shape)


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (3, 256, 384), (2, 640, 1024)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantize_fp4(ep, G, N, K, dtype):
    """Bit for bit: the division by a power of two and the ties are exact."""
    g = _gen(G + K)
    w = _randn(g, G, N, K) * torch.exp2(6 * _randn(g, G, N, K // 32, 1)).expand(G, N, K // 32, 32).reshape(G, N, K)
    flat = w.view(-1, 32)
    flat[0] = 0
    flat[1] = 2.0 ** -130                                 # below the smallest scale's codes
    flat[2] = 3e38
    flat[3] = 2.0 ** -140
    flat[4, 1:] = 0.0
    flat[5] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device=w.device)   # every tie
    flat[6] = -flat[5]
    flat[7] = flat[5] * 6.99 / 6.0
    flat[8] = torch.tensor([7.0] + [0.25, -0.75, 1.25] * 10 + [-0.0], device=w.device)          # the next scale
    flat[9] = torch.tensor([6.984375] + [0.25, -0.75, 1.25] * 10 + [-0.0], device=w.device)
    w = w.to(dtype)
    q = ep.quantize_weights_fp4(w)
    code, byte = _fp4_64(w)
    assert q.codes.shape == (G, N, K // 2) and q.scales.dtype == torch.float8_e8m0fnu and q.scales.shape == (G, N, K // 32)
    assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), byte)
    assert np.array_equal(_unpack(q.codes), code)
    want = _values(code, byte)
    for dt in (BF, torch.float32):
        got = ep.dequantize_weights_fp4(q, dt)
        assert got.dtype == dt
        fine = np.abs(want) < 2.0 ** 128
        assert np.array_equal(got.double().cpu().numpy()[fine], want[fine])
        assert np.isinf(got.double().cpu().numpy()[~fine]).all()
    # no weight is off by more than half a step of its own code
    err = np.abs(want - w.double().cpu().numpy()).reshape(-1, 32)
    s = np.exp2(byte.reshape(-1) - 127.0)
    assert (err <= s[:, None]).all()


def test_quantize_fp4_nan_and_infinity(ep):
    w = _randn(_gen(3), 1, 128, 256)
    w[0, 5, 40], w[0, 7, 0], w[0, 7, 200] = math.nan, math.inf, -math.inf
    for dt in (BF, torch.float32):
        q = ep.quantize_weights_fp4(w.to(dt))
        clean = torch.isfinite(w).view(1, 128, 8, 32).all(-1)
        assert ((q.scales.view(torch.uint8) == 255) == ~clean).all()
        for out in (BF, torch.float32):
            v = ep.dequantize_weights_fp4(q, out).view(1, 128, 8, 32)
            assert torch.isnan(v[~clean]).all() and torch.isfinite(v[clean]).all()
    # products with such a column are NaN, the others are not touched
    x, xs = (_randn(_gen(4), 5, 256) * 50).to(F8), torch.ones(5, 2, device=_dev())
    off = torch.tensor([0, 5], dtype=torch.int32, device=_dev())
    y = ep.grouped_gemm_fp4(x, xs, q.codes, q.scales, off)
    cols = torch.isnan(y).any(0)
    assert cols[[5, 7]].all() and int(cols.sum()) == 2 and torch.isnan(y[:, [5, 7]]).all()


@pytest.mark.parametrize("G,N,K,dtype", [(4, 8192, 4224, BF), (8, 4096, 2304, torch.float32)])
def test_quantize_fp4_of_many_weights_is_that_of_few(ep, G, N, K, dtype):
    """Weights or results of more than 256 MB are read and stored in another way."""
    w = torch.randn((G, N, K), generator=_gen(5), device=_dev(), dtype=dtype)
    q = ep.quantize_weights_fp4(w)
    for i in range(G):
        p = ep.quantize_weights_fp4(w[i:i + 1])
        assert torch.equal(q.codes[i], p.codes[0]) and torch.equal(q.scales[i].view(torch.uint8), p.scales[0].view(torch.uint8))
    v = ep.dequantize_weights_fp4(q, dtype)
    for i in range(G):
        assert torch.equal(v[i], ep.dequantize_weights_fp4(ep.Fp4Weights(q.codes[i:i + 1], q.scales[i:i + 1]), dtype)[0])


def _fp8_rows(g, rows, K, column_major=False):
    x = (_randn(g, rows, K) * 60).clamp(-448, 448).to(F8)
    s = torch.rand(rows, K // 128, generator=g, device=g.device) * torch.exp2(3 * _randn(g, rows, 1)) + 1e-3
    if not column_major:
        return x, s, s
    ld = (rows + 3) // 4 * 4 + 4
    t = torch.full((K // 128, ld), math.nan, device=g.device)
    t[:, :rows] = s.T
    return x, s, t


def _deq(q, s):
    return q.double() * s.double().repeat_interleave(128, 1)


def _largest8(t):
    return t.abs().view(*t.shape[:-1], -1, 8).amax(-1)


def _check_product(ep, counts, N, K, expected, column_major=False, stride=0, seed=0):
    dev = _dev()
    g = _gen(N + K + expected + seed)
    G = len(counts)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
    rows = G * stride if stride else int(sum(counts)) + 3
    first = np.arange(G) * stride if stride else np.concatenate([[0], np.cumsum(counts)])[:-1]
    x, xs, given = _fp8_rows(g, rows, K, column_major)
    used = np.zeros(rows, bool)
    for f, c in zip(first, counts):
        used[f:f + c] = True
    free = torch.from_numpy(~used).to(dev)
    x.view(torch.uint8)[free] = 0x7F                       # rows of no group hold NaN: they are not read
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(118, 128, (G, N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    out = torch.full((rows, N), 7.0, dtype=BF, device=dev)
    got = ep.grouped_gemm_fp4(x, given, codes, byte.view(torch.float8_e8m0fnu), off, group_stride=stride,
                              expected_rows=expected, column_major_scales=column_major, out=out)
    assert got is out
    w = torch.from_numpy(_values(_unpack(codes), byte.cpu().numpy().astype(np.int64))).to(dev)
    for i, (f, c) in enumerate(zip(first, counts)):
        if c == 0:
            continue
        xd = _deq(x[f:f + c], xs[f:f + c])
        y, mag = xd @ w[i].T, xd.abs() @ w[i].abs().T
        # The matrix instruction adds eight neighbouring k at a time, as multiples of 2^-13 of a power of two that is at
        # most the largest of the eight products (below, cut off: test_product_fp4_matrix_instruction): seven of them
        # lose up to 2^-13 of it each, and it is at most the largest |x| times the largest |w| of the eight.  Then 16
        # sums of eight, the scale (1 rounding) and the block sums (2 u each where they may be cut).
        cut = _largest8(xd) @ _largest8(w[i]).T
        tol = 7 * 2.0 ** -13 * cut + (16 + K // 128 + 8) * 2 * U * mag + 2.0 ** -8 * y.abs()
        assert ((out[f:f + c].double() - y).abs() <= tol * (1 + 2.0 ** -7)).all(), i
    assert (out[free] == 7.0).all()


COUNTS = {"one": [1], "few": [3, 0, 1, 17, 0], "mixed": [40, 0, 130, 5, 257, 16], "empty": [0, 0], "apart": [0, 1, 0, 0, 1, 1, 0]}


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (256, 640), (512, 2048), (128, 5248)])
@pytest.mark.parametrize("expected", [1, 12, 40, 100000])
def test_product_fp4(ep, name, N, K, expected):
    """Every form (chosen by the typical rows; the large tiles are so few that they are split) on every distribution."""
    _check_product(ep, COUNTS[name], N, K, expected)


@pytest.mark.parametrize("expected", [1, 12, 40, 100000])
@pytest.mark.parametrize("N,K", [(256, 512), (384, 640), (128, 7168)])
def test_product_fp4_column_major_scales_and_static_layout(ep, N, K, expected):
    _check_product(ep, [5, 0, 300, 17], N, K, expected, column_major=True)
    _check_product(ep, [5, 0, 33, 17], N, K, expected, stride=33)


@pytest.mark.parametrize("N,K", [(2176, 128), (2048, 256), (2048, 640), (2176, 1024), (2048, 5248)])
@pytest.mark.parametrize("column_major,stride", [(False, 0), (True, 0), (False, 1100)])
def test_product_fp4_whole_large_tiles(ep, N, K, column_major, stride):
    """More than 64 tiles of 256 x 256, fewer than 256: none of them is split."""
    _check_product(ep, [700, 0, 130, 1025, 300, 16, 257], N, K, 100000, column_major=column_major, stride=stride)


@pytest.mark.parametrize("K", [128, 384, 512])
@pytest.mark.parametrize("column_major,stride", [(False, 0), (True, 0), (True, 701)])
def test_product_fp4_whole_and_split_large_tiles(ep, K, column_major, stride):
    """264 tiles: a round of 256, and the eight left over in quarters, with some that hold no row or no column."""
    _check_product(ep, [700, 0, 130, 257, 16, 1], 8320, K, 100000, column_major=column_major, stride=stride)


def _products_of(ep, x, w):
    """Sums over 128 products of x and of E2M1 values w, through the call."""
    dev = _dev()
    codes = torch.tensor([int(np.flatnonzero(GRID == abs(v))[0]) + 8 * (v < 0) for v in w], dtype=torch.uint8, device=dev)
    codes = (codes[0::2] | codes[1::2] << 4).expand(1, 128, 64).contiguous()
    s = torch.full((1, 128, 4), 127, dtype=torch.uint8, device=dev)
    x = torch.tensor([x], dtype=torch.float32, device=dev).to(F8)
    off = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    return float(ep.grouped_gemm_fp4(x, torch.ones(1, 1, device=dev), codes, s, off)[0, 0])


def test_product_fp4_matrix_instruction(ep):
    """What the tolerance of the products counts on: beside a product of 2^E, those of the same eight k are cut to
    multiples of 2^(E - 13); others are not."""
    for r in range(8, 18):
        for at, kept in ((2, r <= 13), (7, r <= 13), (8, True), (31, True), (127, True)):
            x, w = [0.0] * 128, [0.0] * 128
            x[0] = x[1] = 256.0
            w[0], w[1], w[at] = 1.0, -1.0, 1.0
            x[at] = 2.0 ** (8 - r)
            assert _products_of(ep, x, w) == (x[at] if kept else 0.0), (r, at)
    x, w = [0.0] * 128, [0.0] * 128
    x[0] = x[1] = 448.0                       # 448 * 6: exponents 8 and 2, and a product above 2^11
    w[0], w[1], w[2] = 6.0, -6.0, 1.0
    x[2] = 1.875 * 2.0 ** -3
    assert _products_of(ep, x, w) == 2.0 ** -3


@pytest.mark.parametrize("counts,N,K,column_major,stride", [
    ([1, 0, 3, 17], 128, 128, False, 0), ([40, 0, 130, 5, 257, 16], 384, 640, True, 0), ([5, 0, 33, 17], 256, 2048, False, 33),
    ([700, 0, 130, 1025, 300, 16, 257], 2176, 384, False, 0), ([700, 0, 130, 257, 16, 1], 8320, 512, True, 0), ([3, 260], 128, 5248, False, 0),
])
@pytest.mark.parametrize("expected", [1, 12, 40, 100000])
def test_product_fp4_exactly(ep, counts, N, K, column_major, stride, expected):
    """Where every sum is exact: products are multiples of 1/4 and at most 18 (nothing is cut), the powers of two leave
    multiples of 1/8 and sums below 2^18, so fp32 holds all of them and the output is their one rounding."""
    dev = _dev()
    g = _gen(N + K)
    G = len(counts)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
    rows = G * stride if stride else sum(counts)
    first = np.arange(G) * stride if stride else np.concatenate([[0], np.cumsum(counts)])[:-1]
    pick = lambda values, *s: torch.tensor(values, device=dev)[torch.randint(0, len(values), s, generator=g, device=dev)]  # noqa: E731
    x, xs = pick([1.0, 1.5, 2.0, 3.0, -1.0, -1.5, -2.0, -3.0], rows, K).to(F8), pick([1.0, 2.0], rows, K // 128)
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    byte = torch.randint(126, 128, (G, N, K // 32), generator=g, device=dev, dtype=torch.uint8)
    out = ep.grouped_gemm_fp4(x, xs.T.contiguous() if column_major and rows % 4 == 0 else xs, codes, byte, off,
                              group_stride=stride, expected_rows=expected,
                              column_major_scales=column_major and rows % 4 == 0)
    w = torch.from_numpy(_values(_unpack(codes), byte.cpu().numpy().astype(np.int64))).to(dev)
    for i, (f, c) in enumerate(zip(first, counts)):
        want = _deq(x[f:f + c], xs[f:f + c]) @ w[i].T
        assert torch.equal(out[f:f + c], want.to(torch.float32).to(BF)), i


def test_product_fp4_many_groups_and_long_rows(ep):
    _check_product(ep, ([3, 0, 1, 2] * 250), 128, 256, 0)
    _check_product(ep, [260, 3], 256, 7168, 100000)
    _check_product(ep, [2, 3], 128, 32768, 2)


@pytest.mark.parametrize("off,stride", [([-5, 3, 40, 12, 9], 0), ([0, 1 << 30, -(1 << 30), 20, 2 ** 31 - 1], 0),
                                        ([9, 7, 5, 3, 1], 0), ([0, 1 << 30, 5, 2, 2 ** 31 - 1], 8)])
@pytest.mark.parametrize("expected", [2, 40, 100000])
def test_fp4_offsets_outside_the_rows_are_clamped(ep, off, stride, expected):
    dev = _dev()
    g = _gen(3)
    rows, N, K, G = 32, 128, 256, 4
    x, xs, _ = _fp8_rows(g, rows, K)
    q = ep.quantize_weights_fp4(_randn(g, G, N, K))
    out = torch.zeros(rows, N, dtype=BF, device=dev)
    ep.grouped_gemm_fp4(x, xs, q.codes, q.scales, torch.tensor(off, dtype=torch.int32, device=dev), group_stride=stride,
                        expected_rows=expected, out=out)
    touched = torch.zeros(rows, dtype=torch.bool)
    for i in range(G):
        if stride:
            b = min(i * stride, rows)
            e = min(b + min(max(off[i + 1] - off[i], 0), stride), rows)
        else:
            b = min(max(off[i], 0), rows)
            e = min(max(off[i + 1], b), rows)
        touched[b:e] = True
    assert torch.equal(out.ne(0).any(1).cpu(), touched)


# ----------------------------------------------------------------------------
# offsets past 32 bits
# ----------------------------------------------------------------------------

def test_block_norm_past_2_to_the_31_elements(ep):
    """The last rows of 66000 x 32768 (and of a stride of 32776) equal a call on them alone."""
    dev = _dev()
    T, H = 66000, 32768
    x = torch.zeros(T, H + 8, dtype=BF, device=dev)[:, :H]
    y = torch.zeros(T, H, dtype=BF, device=dev)
    last = slice(T - 4, T)
    g = _gen(70)
    x[last], y[last] = _randn(g, 4, H).to(BF), _randn(g, 4, H).to(BF)
    w, gate = torch.randn(H, generator=g, device=dev), torch.ones(T, 1, device=dev)
    o = dict(weight=w, y_norm=True, y_weight=w)
    n = ep.block_norm(x, y, gate=gate, quantize=True, **o)
    m = ep.block_norm(x[last], y[last], gate=gate[last], quantize=True, **o)
    for k in ("x", "h", "codes", "scales"):
        assert torch.equal(getattr(n, k)[last].view(torch.uint8), getattr(m, k).view(torch.uint8)), k
        assert not getattr(n, k)[:8].float().isnan().any()
    del n
    q = ep.block_norm_backward(x, y, grad_x=y, grad_h=y, gate=gate, need=("x", "y", "gate"), **o)
    p = ep.block_norm_backward(x[last], y[last], grad_x=y[last], grad_h=y[last], gate=gate[last], need=("x", "y", "gate"), **o)
    for k in ("x", "y", "gate"):
        assert torch.equal(getattr(q, k)[last], getattr(p, k)), k


def test_fp4_past_2_to_the_31_elements(ep):
    """Weights, codes, rows and outputs whose offsets pass 32 bits: the last group against a call on it alone."""
    dev = _dev()
    G, N, K = 9, 32768, 16384
    w = torch.zeros(G, N, K, dtype=BF, device=dev)
    w[-1] = torch.randn((N, K), generator=_gen(71), device=dev, dtype=BF)
    q = ep.quantize_weights_fp4(w)
    r = ep.quantize_weights_fp4(w[-1:])
    del w
    assert torch.equal(q.codes[-1], r.codes[0]) and torch.equal(q.scales[-1].view(torch.uint8), r.scales[0].view(torch.uint8))
    assert torch.equal(ep.dequantize_weights_fp4(q)[-1], ep.dequantize_weights_fp4(r)[0])
    rows = 140000
    x = torch.zeros(rows, K, dtype=torch.uint8, device=dev).view(F8)
    xs = torch.ones(rows, K // 128, device=dev)
    x[-300:] = (_randn(_gen(72), 300, K) * 50).to(F8)
    few = torch.tensor([0, 300], dtype=torch.int32, device=dev)
    off = torch.full((G + 1,), rows - 300, dtype=torch.int32, device=dev)
    off[0], off[-1] = rows - 301, rows
    out = torch.empty(rows, N, dtype=BF, device=dev)
    for expected in (40, 100000):
        ep.grouped_gemm_fp4(x, xs, q.codes, q.scales, off, expected_rows=expected, out=out)
        assert torch.equal(out[-300:], ep.grouped_gemm_fp4(x[-300:], xs[-300:], r.codes, r.scales, few, expected_rows=expected))
        assert not out[-301].any()
