"""GPU checks of the expert layer against its formulas in 64 bits.

Tolerances count roundings.  u = 2^-24 is fp32's half step; bf16 rounds by at
most 2^-8, E4M3 by 2^-4 of a value.  A sum of n fp32 terms is off by at most
n * 2u * (sum of the terms' magnitudes) -- 2u, since the matrix cores may cut
instead of round -- whatever its order.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
F8 = torch.float8_e4m3fn


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
# gate
# ----------------------------------------------------------------------------

def _gate64(x, K, score, normalize, scale, coef, mask, gw=None, gl=None):
    """ids, weights, counts, V, loss, gradient -- from the definitions, numpy in 64 bits."""
    T, E = x.shape
    live = np.ones(T, bool) if mask is None else mask != 0
    x = np.where(live[:, None], x, -np.inf)
    live &= ~np.isneginf(x).all(1)
    s = np.zeros((T, E))
    top = np.where(live, x.max(1, initial=-np.inf), 0.0)
    with np.errstate(over="ignore"):
        s[live] = np.exp(x[live] - top[live, None]) if score == "softmax" else 1 / (1 + np.exp(-x[live]))
    S = s.sum(1, keepdims=True)
    p = np.divide(s, S, out=np.zeros_like(s), where=S > 0)
    r = p if score == "softmax" else s
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -x), axis=1)[:, :K]
    idx = np.where(np.isneginf(np.take_along_axis(x, order, 1)), -1, order)
    sel = np.zeros((T, E), bool)
    for t in range(T):
        sel[t, idx[t][idx[t] >= 0]] = True
    rs = np.where(sel, r, 0.0)
    tot = rs.sum(1, keepdims=True)
    wn = np.divide(rs, tot, out=np.zeros_like(rs), where=tot > 0) if normalize else rs
    w = np.where(idx >= 0, np.take_along_axis(wn, np.maximum(idx, 0), 1), 0.0) * scale
    n, V = sel.sum(0), int(live.sum())
    f = E * n / (K * V) if V else np.zeros(E)
    loss = coef * (f * p.sum(0)).sum() / V if V else 0.0
    if gw is None:
        return idx, w, n, V, loss, None, None
    g = np.zeros((T, E))
    for t in range(T):
        for k in range(K):
            if idx[t, k] >= 0:
                g[t, idx[t, k]] = gw[t, k] * scale
    if normalize:
        inv = np.divide(1.0, tot, out=np.zeros_like(tot), where=tot > 0)
        ds = np.where(sel, (g - (g * wn).sum(1, keepdims=True)) * inv, 0.0)
        mag = np.where(sel, (np.abs(g) + (np.abs(g) * wn).sum(1, keepdims=True)) * inv, 0.0)
    else:
        ds, mag = g, np.abs(g)
    d = (coef * gl * f / V if V else np.zeros(E))[None, :] * live[:, None]
    if score == "softmax":
        o, m = ds + d, mag + np.abs(d)
        return idx, w, n, V, loss, p * (o - (p * o).sum(1, keepdims=True)), p * (m + (p * m).sum(1, keepdims=True))
    invS = np.divide(1.0, S, out=np.zeros_like(S), where=S > 0)
    o = ds + (d - (d * p).sum(1, keepdims=True)) * invS
    m = mag + (np.abs(d) + (np.abs(d) * p).sum(1, keepdims=True)) * invS
    return idx, w, n, V, loss, s * (1 - s) * o, s * m


def _check_gate(ep, x, K, score, normalize, mask=None, scale=1.5, coef=0.02, seed=0):
    dev = x.device
    T, E = x.shape
    g = _gen(seed + 1000)
    gw, gl = _randn(g, T, K), torch.rand(1, generator=g, device=dev) + 0.5
    q = ep.gate(x, K, score=score, normalize=normalize, scale=scale, balance_coef=coef, token_mask=mask)
    grad = ep.gate_backward(x, q, gw, gl)
    x64 = x.double().cpu().numpy()
    idx, w, n, V, loss, want, mag = _gate64(x64, K, score, normalize, scale, coef,
                                            None if mask is None else mask.cpu().numpy(),
                                            gw.double().cpu().numpy(), float(gl))
    assert np.array_equal(q.topk_idx.cpu().numpy(), idx)
    assert np.array_equal(q.num_tokens_per_expert.cpu().numpy(), n)
    assert int(q.num_valid) == V
    # a score: the logit's difference (one rounding, times the exponent's size: |x| u), the exponential and
    # the quotient (2 u each), the sum of E positive terms (at most 16 + 6 in a chain)
    big = np.abs(np.where(np.isfinite(x64), x64, 0)).max(initial=0.0)
    rel = (2 * big + 40) * U
    assert (np.abs(q.topk_weights.double().cpu().numpy() - w) <= 2 * rel * np.abs(w) + 1e-37).all()
    # chains of the sum over tokens: a lane's tokens, 16 waves, 256 workgroups in stripes
    assert abs(float(q.loss) - loss) <= (rel + (T / 4 + 60) * U) * abs(loss) + 1e-37
    got = grad.double().cpu().numpy()
    assert grad.dtype == x.dtype and np.isfinite(got).all()
    out = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    assert (np.abs(got - want) <= 4 * rel * mag + out * np.abs(want) + 1e-37).all()
    return q


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,K,dtype", [
    (1, 1, 1, "float32"), (3, 7, 7, "float32"), (16, 256, 8, "bfloat16"), (17, 60, 4, "float32"),
    (65, 64, 16, "bfloat16"), (129, 128, 6, "float32"), (300, 256, 8, "float32"), (5000, 100, 3, "bfloat16"),
    (40, 384, 6, "bfloat16"), (21, 1024, 16, "float32"), (700, 1000, 2, "bfloat16"),
    # workgroups of 16 waves at each way of holding a token, and of four waves
    (2100, 1024, 8, "float32"), (4200, 512, 6, "bfloat16"), (1500, 64, 2, "float32"), (17000, 60, 4, "float32"),
])
def test_gate(ep, score, normalize, T, E, K, dtype):
    x = (2 * _randn(_gen(T + E), T, E)).to(getattr(torch, dtype))
    _check_gate(ep, x, K, score, normalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_masked_tokens_and_experts(ep, score):
    """Padding tokens whose logits hold NaN and infinities, masked experts, tokens
    with fewer experts left than K, with none, and logits at the type's lowest value."""
    g = _gen(5)
    T, E, K = 64, 64, 4
    x = _randn(g, T, E)
    x[:, 10:20] = -math.inf
    x[3] = -math.inf
    x[4, 1:] = -math.inf
    x[5, 3:] = -math.inf
    mask = torch.ones(T, dtype=torch.uint8, device=x.device)
    mask[30:40] = 0
    x[30] = math.nan
    x[31] = math.inf
    x[32] = -math.inf
    q = _check_gate(ep, x, K, score, True, mask)
    assert (q.topk_idx[30:40] == -1).all() and (q.topk_weights[30:40] == 0).all()
    assert (q.topk_idx[3] == -1).all() and q.topk_idx[4].tolist() == [0, -1, -1, -1]
    low = torch.full((4, 32), torch.finfo(torch.float32).min, device=x.device)
    q = ep.gate(low, 3, score=score)
    assert q.topk_idx.tolist() == [[0, 1, 2]] * 4 and torch.isfinite(q.topk_weights).all()
    assert torch.isfinite(ep.gate_backward(low, q, torch.ones(4, 3, device=x.device))).all()
    none = torch.zeros(6, dtype=torch.bool, device=x.device)
    q = ep.gate(_randn(g, 6, 8), 2, score=score, balance_coef=1.0, token_mask=none)
    assert float(q.loss) == 0 and int(q.num_valid) == 0 and not q.num_tokens_per_expert.any()


def test_gate_ties_strides_and_empty(ep):
    dev = _dev()
    x = torch.zeros(9, 300, device=dev)
    x[:, 100:104] = 1.0
    q = ep.gate(x, 6)
    assert q.topk_idx.tolist() == [[100, 101, 102, 103, 0, 1]] * 9
    wide = _randn(_gen(8), 50, 131)
    for off in (0, 1, 2):                      # odd strides and unaligned rows
        _check_gate(ep, wide[:, off:off + 64], 4, "softmax", True)
    for T in (0,):
        q = ep.gate(torch.empty(T, 16, device=dev), 2, balance_coef=1.0)
        assert q.topk_idx.shape == (0, 2) and float(q.loss) == 0 and not q.num_tokens_per_expert.any()
        assert ep.gate_backward(torch.empty(T, 16, device=dev), q).shape == (0, 16)


def test_gate_repeats_bit_for_bit_and_none_gradients(ep):
    x = _randn(_gen(9), 20000, 256)
    a = ep.gate(x, 8, balance_coef=1.0)
    for _ in range(3):
        b = ep.gate(x, 8, balance_coef=1.0)
        assert torch.equal(a.loss, b.loss) and torch.equal(a.topk_idx, b.topk_idx)
    assert not ep.gate_backward(x[:64], ep.gate(x[:64], 8)).any()


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gate_gradient_against_differences(ep, score, normalize):
    """Central differences of the formula in 64 bits, counts and choice held."""
    g = _gen(11)
    T, E, K, scale, coef = 6, 12, 3, 1.5, 2.0
    x = _randn(g, T, E) * 2
    gw, gl = _randn(g, T, K), torch.ones(1, device=x.device)
    q = ep.gate(x, K, score=score, normalize=normalize, scale=scale, balance_coef=coef)
    got = ep.gate_backward(x, q, gw, gl).double().cpu()
    idx, n = q.topk_idx.cpu(), q.num_tokens_per_expert.cpu().double()

    def value(v):
        s = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
        p = s / s.sum(1, keepdim=True)
        w = torch.gather(s, 1, idx)
        if normalize:
            w = w / w.sum(1, keepdim=True)
        return (gw.cpu().double() * scale * w).sum() + coef * (E * n / (K * T) * p.mean(0)).sum()

    v, h = x.double().cpu(), 1e-4
    for t in range(T):
        for e in range(E):
            a, b = v.clone(), v.clone()
            a[t, e] += h
            b[t, e] -= h
            d = (value(a) - value(b)) / (2 * h)
            # the differences: h^2 / 6 times a third derivative of at most ~30
            assert abs(d - got[t, e]) <= 1e-5 * (1 + abs(d))


# ----------------------------------------------------------------------------
# quantisers
# ----------------------------------------------------------------------------

def _np_quant(v, amax):
    a = np.maximum(amax.astype(np.float32), np.float32(2.0 ** -64))
    scaled = v.astype(np.float32) * (np.float32(448.0) / a)
    codes = torch.from_numpy(np.ascontiguousarray(scaled, np.float32)).to(F8).view(torch.uint8).numpy()
    return codes, a / np.float32(448.0)


def _odd_values(g, *s):
    """Normal values of very different rows, zero rows, bf16's smallest and largest."""
    x = _randn(g, *s) * torch.exp2(torch.randint(-30, 30, (*s[:-1], 1), generator=g, device=g.device).float())
    x.view(-1)[::97] = 0.0
    x[..., 0, :] = 0.0
    x[..., s[-2] // 2, :128] = 1e-39
    x[..., s[-2] - 1, 5] = 3.38e38
    return x


@pytest.mark.parametrize("rows,H", [(1, 128), (3, 384), (70, 1024), (33, 7168)])
@pytest.mark.parametrize("column_major", [False, True])
def test_quantize_rows(ep, rows, H, column_major):
    x = _odd_values(_gen(rows), rows, H).to(torch.bfloat16)
    q, s = ep.quantize_rows(x, column_major_scales=column_major)
    v = x.float().cpu().numpy().reshape(rows, H // 128, 128)
    codes, scales = _np_quant(v, np.abs(v).max(2, keepdims=True))
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), codes.reshape(rows, H))
    got = s[:, :rows].t() if column_major else s
    assert np.array_equal(got.cpu().numpy(), scales[:, :, 0])


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (3, 256, 384), (2, 640, 1024)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_quantize_weights(ep, G, N, K, dtype):
    w = _odd_values(_gen(N), G, N, K).to(getattr(torch, dtype))
    q = ep.quantize_weights(w, transposed=True)
    v = w.float().cpu().numpy().reshape(G, N // 128, 128, K // 128, 128)
    codes, scales = _np_quant(v, np.abs(v).max((2, 4), keepdims=True))
    codes, scales = codes.reshape(G, N, K), scales[:, :, 0, :, 0]
    assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes_t.view(torch.uint8).cpu().numpy(), codes.transpose(0, 2, 1))
    assert np.array_equal(q.scales_t.cpu().numpy(), scales.transpose(0, 2, 1))
    p = ep.quantize_weights(w)
    assert p.codes_t is None and torch.equal(p.codes.view(torch.uint8), q.codes.view(torch.uint8))


# ----------------------------------------------------------------------------
# products
# ----------------------------------------------------------------------------

def _fp8_rows(g, rows, K, column_major=False):
    q = (_randn(g, rows, K) * 60).clamp(-448, 448).to(F8)
    s = torch.exp2(2 * _randn(g, rows, K // 128)) * 0.01
    if not column_major:
        return q, s, s
    ld = (rows + 3) // 4 * 4 + 4
    cm = torch.full((K // 128, ld), math.nan, device=s.device)
    cm[:, :rows] = s.t()
    return q, s, cm


def _deq(q, s):
    return q.double() * s.double().repeat_interleave(128, -1)


def _offsets(counts, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)


COUNTS = {
    "one": [1], "ragged": [5, 0, 17, 64, 1, 130, 0], "empty": [0, 0, 0], "tiles": [256, 300, 0, 1, 255],
    "deep": [700, 37],
}


def _check_product(ep, counts, N, K, expected, column_major=False, stride=0, seed=0):
    dev = _dev()
    g = _gen(seed + N + K)
    G = len(counts)
    off = _offsets(counts, dev)
    rows = G * stride if stride else int(sum(counts)) + 3      # three rows of no group at the end
    first = np.arange(G) * stride if stride else np.concatenate([[0], np.cumsum(counts)])[:-1]
    x, xs, given = _fp8_rows(g, rows, K, column_major)
    w = (_randn(g, G, N, K) * 50).clamp(-448, 448).to(F8)
    ws = torch.exp2(_randn(g, G, N // 128, K // 128)) * 0.01
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=dev)
    got = ep.grouped_gemm_fp8(x, given, w, ws, off, group_stride=stride, expected_rows=expected,
                              column_major_scales=column_major, out=out)
    assert got is out
    used = np.zeros(rows, bool)
    xd = _deq(x, xs)
    for i, (f, c) in enumerate(zip(first, counts)):
        used[f:f + c] = True
        if c == 0:
            continue
        wd = _deq(w[i], ws[i].repeat_interleave(128, 0))
        y, mag = xd[f:f + c] @ wd.T, xd[f:f + c].abs() @ wd.abs().T
        # 128 products in a block, then scale (2 roundings) and block sums
        tol = (128 + K // 128 + 8) * 2 * U * mag + 2.0 ** -8 * y.abs()
        assert ((out[f:f + c].double() - y).abs() <= tol).all(), i
    assert (out[torch.from_numpy(~used).to(dev)] == 7.0).all()


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (256, 640), (512, 2048)])
@pytest.mark.parametrize("expected", [2, 12, 100, 100000])
def test_product(ep, name, N, K, expected):
    """Every tile form (chosen by the typical rows) on every distribution."""
    _check_product(ep, COUNTS[name], N, K, expected)


@pytest.mark.parametrize("expected", [2, 12, 100, 100000])
@pytest.mark.parametrize("N,K", [(256, 512), (384, 640)])
def test_product_column_major_scales_and_static_layout(ep, N, K, expected):
    _check_product(ep, [5, 0, 300, 17], N, K, expected, column_major=True)
    _check_product(ep, [5, 0, 33, 17], N, K, expected, stride=33)


def test_product_many_groups_and_long_rows(ep):
    _check_product(ep, ([3, 0, 1, 2] * 250), 128, 256, 0)
    _check_product(ep, [260, 3], 256, 7168, 100000)


@pytest.mark.parametrize("off,stride", [([-5, 3, 40, 12, 9], 0), ([0, 1 << 30, -(1 << 30), 20, 2 ** 31 - 1], 0),
                                        ([9, 7, 5, 3, 1], 0), ([0, 1 << 30, 5, 2, 2 ** 31 - 1], 8)])
@pytest.mark.parametrize("expected", [2, 100000])
def test_offsets_outside_the_rows_are_clamped(ep, off, stride, expected):
    """Offsets that are no layout reach no row outside the buffers: the groups they
    describe are cut to the rows there are."""
    dev = _dev()
    g = _gen(3)
    rows, N, K, G = 32, 128, 256, 4
    x, xs, _ = _fp8_rows(g, rows, K)
    w, ws = (_randn(g, G, N, K) * 50).to(F8), torch.full((G, 1, K // 128), 0.01, device=dev)
    t = torch.tensor(off, dtype=torch.int32, device=dev)
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
    ep.grouped_gemm_fp8(x, xs, w, ws, t, group_stride=stride, expected_rows=expected, out=out)
    dw = ep.grouped_wgrad_fp8(out, x, xs, t, group_stride=stride)
    a8, _, c8, _ = ep.swiglu_fp8(_randn(g, rows, 256).bfloat16(), t, group_stride=stride, checkpoint=True)
    torch.cuda.synchronize()
    touched = torch.zeros(rows, dtype=torch.bool)
    for i in range(G):
        if stride:
            b = min(i * stride, rows)
            e = min(b + min(max(off[i + 1] - off[i], 0), stride), rows)
        else:
            b = min(max(off[i], 0), rows)
            e = min(max(off[i + 1], b), rows)
        touched[b:e] = True
        assert bool(dw[i].any()) == (e > b)
    assert torch.equal(out.ne(0).any(1).cpu(), touched)


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (256, 640), (640, 384)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_weight_gradient(ep, name, N, K, dtype):
    _check_wgrad(ep, COUNTS[name], N, K, getattr(torch, dtype))


def _check_wgrad(ep, counts, N, K, dtype, column_major=False, stride=0):
    dev = _dev()
    g = _gen(N + K)
    G = len(counts)
    off = _offsets(counts, dev)
    rows = G * stride if stride else int(sum(counts)) + 3
    first = np.arange(G) * stride if stride else np.concatenate([[0], np.cumsum(counts)])[:-1]
    x, xs, given = _fp8_rows(g, rows, K, column_major)
    dy = _randn(g, rows, N).bfloat16()
    used = torch.zeros(rows, dtype=torch.bool)
    for f, c in zip(first, counts):
        used[f:f + c] = True
    dy[~used.to(dev)] = math.nan                   # rows of no group are not read
    out = torch.full((G, N, K), math.nan, dtype=dtype, device=dev)
    ep.grouped_wgrad_fp8(dy, x, given, off, group_stride=stride, column_major_scales=column_major, out=out)
    # the definition rounds x * scale (one fp32 product) to bf16
    xr = (x.float() * xs.repeat_interleave(128, 1)).bfloat16().double()
    step = 2.0 ** -8 if dtype == torch.bfloat16 else U
    for i, (f, c) in enumerate(zip(first, counts)):
        d = dy[f:f + c].double()
        want, mag = d.T @ xr[f:f + c], d.abs().T @ xr[f:f + c].abs()
        assert ((out[i].double() - want).abs() <= (c + 4) * 2 * U * mag + step * want.abs()).all(), i


def test_weight_gradient_layouts(ep):
    _check_wgrad(ep, [5, 0, 300, 17], 384, 256, torch.bfloat16, column_major=True)
    _check_wgrad(ep, [5, 0, 33, 17], 128, 256, torch.bfloat16, stride=33)
    _check_wgrad(ep, [150, 0, 200, 17], 256, 384, torch.float32, stride=200)
    _check_wgrad(ep, [2, 0, 1] * 200, 128, 128, torch.bfloat16)


@pytest.mark.parametrize("N,K", [(128, 128), (384, 640), (512, 256)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_weight_gradient_many_rows(ep, N, K, dtype):
    """The larger tile, which many rows a group choose."""
    dt = getattr(torch, dtype)
    _check_wgrad(ep, [1030, 0, 700], N, K, dt)
    _check_wgrad(ep, [1100, 3], N, K, dt, column_major=True)
    _check_wgrad(ep, [600, 5], N, K, dt, stride=600)


# ----------------------------------------------------------------------------
# SwiGLU
# ----------------------------------------------------------------------------

def _check_codes(q, s, want, rel):
    """Codes and scales against values: half a step of E4M3 (2^-4 of a value, 2^-10 of the
    scale under the normal range) beside what the fp32 value may be off by (rel)."""
    amax = want.abs().unflatten(-1, (-1, 128)).amax(-1)
    # bf16-free: the scale follows the block's largest value
    ok = amax > 1e-15
    assert ((s.double() * 448 - amax).abs() <= (rel + 4 * U) * amax)[ok].all()
    err = (_deq(q, s) - want).abs()
    half = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s.double().repeat_interleave(128, -1))
    assert (err <= half * (1 + 8 * U) + rel * want.abs() + 1e-30).all()


def _silu_rel(h):
    # e^-g: |g| * u; the sum, the reciprocal and two products: 6 u
    return (float(h.abs().max()) * 2 + 8) * U


@pytest.mark.parametrize("rows,inner", [(1, 128), (5, 384), (77, 1024), (40, 2048)])
@pytest.mark.parametrize("checkpoint,column_major", [(True, False), (False, False), (True, True)])
def test_swiglu(ep, rows, inner, checkpoint, column_major):
    g = _gen(rows + inner)
    h = (_randn(g, rows, 2 * inner) * torch.exp2(2 * _randn(g, rows, 1))).clamp(-60, 60).bfloat16()
    q, s, ck, cs = ep.swiglu_fp8(h, checkpoint=checkpoint, column_major_scales=column_major)
    if column_major:
        s = s[:, :rows].t()
    d = h.double()
    gate, up = d[:, :inner], d[:, inner:]
    _check_codes(q, s, gate * torch.sigmoid(gate) * up, _silu_rel(h))
    if checkpoint:
        want, ws = ep.quantize_rows(h)
        assert torch.equal(ck.view(torch.uint8), want.view(torch.uint8)) and torch.equal(cs, ws)
    else:
        assert ck is None and cs is None


@pytest.mark.parametrize("rows,inner", [(1, 128), (5, 384), (77, 1024)])
@pytest.mark.parametrize("quantize,column_major", [(True, False), (False, False), (True, True)])
def test_swiglu_backward(ep, rows, inner, quantize, column_major):
    """The formula, and differences of the forward formula, at the checkpoint's values."""
    g = _gen(rows * inner)
    ck, cs = ep.quantize_rows((_randn(g, rows, 2 * inner) * 3).bfloat16())
    da = _randn(g, rows, inner).bfloat16()
    dh, q, s = ep.swiglu_fp8_backward(da, ck, cs, quantize=quantize, column_major_scales=column_major)
    h = _deq(ck, cs)
    gate, up, d = h[:, :inner], h[:, inner:], da.double()
    sg = torch.sigmoid(gate)
    want = torch.cat([d * up * sg * (1 + gate * (1 - sg)), d * gate * sg], 1)
    # 1 + g (1 - s) may cancel: its terms' magnitudes count
    mag = torch.cat([(d * up * sg).abs() * (1 + (gate * (1 - sg)).abs()), (d * gate * sg).abs()], 1)
    tol = 2 * _silu_rel(h) * mag
    assert ((dh.double() - want).abs() <= tol + 2.0 ** -8 * want.abs() + 1e-30).all()
    f = lambda a, b: d * a * torch.sigmoid(a) * b  # noqa: E731
    e = 1e-5
    diff = torch.cat([(f(gate + e, up) - f(gate - e, up)) / (2 * e), (f(gate, up + e) - f(gate, up - e)) / (2 * e)], 1)
    # differences: e^2 / 6 times a third derivative (< |d u|), and 2^-53 |f| / e
    assert ((dh.double() - diff).abs() <= tol + 2.0 ** -8 * want.abs() + 1e-9 * (1 + d.abs().max() * h.abs().max())).all()
    if quantize:
        s = s[:, :rows].t() if column_major else s
        err = (_deq(q, s) - want).abs()
        half = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s.double().repeat_interleave(128, -1))
        assert (err <= half * (1 + 8 * U) + 2 * tol).all()
    else:
        assert q is None and s is None


def test_swiglu_extreme_gates(ep):
    h = torch.zeros(2, 256, device=_dev())
    h[0, :128] = torch.linspace(-3e4, 3e4, 128)
    h[0, 128:] = 1.0
    q, s, ck, cs = ep.swiglu_fp8(h.bfloat16(), checkpoint=True)
    assert torch.isfinite(_deq(q, s)).all() and (_deq(q, s)[0, :60].abs() < 1e-3).all()
    dh, _, _ = ep.swiglu_fp8_backward(torch.ones(2, 128, device=h.device, dtype=torch.bfloat16), ck, cs)
    assert torch.isfinite(dh).all()


@pytest.mark.parametrize("stride", [0, 40])
def test_rows_of_no_group_stay_as_they_were(ep, stride):
    """Through the C calls on canary-filled buffers."""
    dev = _dev()
    counts, inner = [7, 0, 33, 2], 256
    rows = len(counts) * stride if stride else sum(counts) + 5
    first = np.arange(4) * stride if stride else np.concatenate([[0], np.cumsum(counts)])[:-1]
    used = torch.zeros(rows, dtype=torch.bool)
    for f, c in zip(first, counts):
        used[f:f + c] = True
    free = (~used).to(dev)
    off = _offsets(counts, dev)
    h = _randn(_gen(1), rows, 2 * inner).bfloat16()
    can = lambda w: torch.full((rows, w), 0x5A, dtype=torch.uint8, device=dev)  # noqa: E731
    fl = lambda w: torch.full((rows, w), -3.0, device=dev)  # noqa: E731
    c, s, ck, cs = can(inner), fl(2), can(2 * inner), fl(4)
    p = lambda t: t.data_ptr()  # noqa: E731
    st = ep._stream()
    assert ep.ep_swiglu_fp8(p(h), inner, p(off), 4, stride, rows, 0, p(c), p(s), p(ck), p(cs), st) == 0
    q, qs = can(2 * inner), fl(4)
    assert ep.ep_quantize_rows(p(h), 2 * inner, p(off), 4, stride, rows, 0, p(q), p(qs), st) == 0
    dh = torch.full((rows, 2 * inner), 9.0, dtype=torch.bfloat16, device=dev)
    d8, ds = can(2 * inner), fl(4)
    da = _randn(_gen(2), rows, inner).bfloat16()
    assert ep.ep_swiglu_fp8_backward(p(da), p(ck), p(cs), inner, p(off), 4, stride, rows, 0, p(dh), p(d8), p(ds), st) == 0
    torch.cuda.synchronize()
    for t, v in ((c, 0x5A), (ck, 0x5A), (q, 0x5A), (d8, 0x5A), (s, -3.0), (cs, -3.0), (qs, -3.0), (ds, -3.0), (dh, 9.0)):
        assert (t[free] == v).all()
    assert torch.equal(q[~free], ck[~free]) and torch.equal(qs[~free], cs[~free])
    for t in (s, cs, ds):
        assert (t[~free] > 0).all()


# ----------------------------------------------------------------------------
# together, as they are used
# ----------------------------------------------------------------------------

def _layer(ep, x, logits, w1, w2, K, static_cap=0, aligned=1, column_major=False):
    E = w1.codes.shape[0]
    g = ep.gate(logits, K)
    if static_cap:
        x8, xs, lay = ep.low_latency_dispatch(x, g.topk_idx, g.topk_weights, E, 1, static_cap, True)
        h = lay.handle
    else:
        lay = ep.get_dispatch_layout(g.topk_idx, E, 1, expert_alignment=aligned)
        x8, xs, h = ep.dispatch(x, g.topk_weights, lay, True, column_major_scales=column_major)
    y1 = ep.grouped_gemm_fp8(x8, xs, w1.codes, w1.scales, h, column_major_scales=column_major)
    a8, a_s, _, _ = ep.swiglu_fp8(y1, h)
    return ep.combine(ep.grouped_gemm_fp8(a8, a_s, w2.codes, w2.scales, h), h), g


def _layer_case(seed, T=70, H=256, inner=128, E=8):
    g = _gen(seed)
    x = _randn(g, T, H).bfloat16()
    return x, _randn(g, T, E), _randn(g, E, 2 * inner, H) * 0.1, _randn(g, E, H, inner) * 0.1


def test_layer_forward_in_every_layout(ep):
    """The same bits through the dense, aligned, column-major and static layouts, and
    the 64-bit layer within what its roundings add up to."""
    x, logits, w1, w2 = _layer_case(1)
    K = 2
    q1, q2 = ep.quantize_weights(w1), ep.quantize_weights(w2)
    out, g = _layer(ep, x, logits, q1, q2, K)
    for kw in (dict(static_cap=70), dict(aligned=64), dict(column_major=True), dict(aligned=128, column_major=True)):
        other, _ = _layer(ep, x, logits, q1, q2, K, **kw)
        assert torch.equal(out, other), kw
    d1 = _deq(q1.codes, q1.scales.repeat_interleave(128, 1))
    d2 = _deq(q2.codes, q2.scales.repeat_interleave(128, 1))
    xd = x.double()
    want = torch.zeros_like(xd)
    for t in range(x.shape[0]):
        for k in range(K):
            e = int(g.topk_idx[t, k])
            y = d1[e] @ xd[t]
            a = torch.nn.functional.silu(y[:128]) * y[128:]
            want[t] += g.topk_weights[t, k].double() * (d2[e] @ a)
    # two E4M3 roundings (2^-4 at most, 2^-4 / sqrt(3) / ... on average) and bf16's: of the
    # norm, under the largest a single rounding can be, twice
    assert float((out.double() - want).norm() / want.norm()) < 2 * 2.0 ** -4


def test_layer_captured_and_replayed(ep):
    """Gate, static dispatch, products, SwiGLU, combine and the backward calls in one
    graph; replays on new inputs equal the eager calls, with eager work in between."""
    dev = _dev()
    x, logits, w1, w2 = _layer_case(2, T=40)
    q1, q2 = ep.quantize_weights(w1, True), ep.quantize_weights(w2, True)
    E, K, T, H = 8, 2, 40, 256
    out = (torch.empty(E * T, H, dtype=F8, device=dev), torch.empty(E * T, H // 128, device=dev), None)
    ws = torch.empty(ep.ep_workspace_bytes(T, K, E, 1), dtype=torch.uint8, device=dev)

    def step(x, logits, go):
        g = ep.gate(logits, K, balance_coef=1.0)
        x8, xs, lay = ep.low_latency_dispatch(x, g.topk_idx, g.topk_weights, E, 1, T, True, ws=ws)
        h = lay.handle
        a8, a_s, ck, cs = ep.swiglu_fp8(ep.grouped_gemm_fp8(x8, xs, q1.codes, q1.scales, h), h, checkpoint=True)
        y = ep.grouped_gemm_fp8(a8, a_s, q2.codes, q2.scales, h)
        gy, gw = ep.combine_backward(go, h, y=y)
        g8, gs = ep.quantize_rows(gy, h)
        gh, gh8, ghs = ep.swiglu_fp8_backward(ep.grouped_gemm_fp8(g8, gs, q2.codes_t, q2.scales_t, h), ck, cs, h)
        gx = ep.dispatch_backward(ep.grouped_gemm_fp8(gh8, ghs, q1.codes_t, q1.scales_t, h), h)
        return [ep.combine(y, h), g.loss, gx, gw, ep.grouped_wgrad_fp8(gy, a8, a_s, h), ep.grouped_wgrad_fp8(gh, x8, xs, h),
                ep.gate_backward(logits, g, gw, torch.ones(1, device=dev))]

    go = _randn(_gen(3), T, H).bfloat16()
    bx, bl, bg = x.clone(), logits.clone(), go.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(bx, bl, bg)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(bx, bl, bg)
    for i in range(4):
        nx, nl, _, _ = _layer_case(10 + i, T=40)
        ng = _randn(_gen(20 + i), T, H).bfloat16()
        want = [t.clone() for t in step(nx, nl, ng)]
        bx.copy_(nx), bl.copy_(nl), bg.copy_(ng)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_calls_on_two_streams(ep):
    x, logits, w1, w2 = _layer_case(4, T=300)
    q1, q2 = ep.quantize_weights(w1), ep.quantize_weights(w2)
    want, _ = _layer(ep, x, logits, q1, q2, 2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(_layer(ep, x, logits, q1, q2, 2)[0])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_autograd_layer_gradients(ep):
    """gate and experts under autograd: every gradient equals the chain of the plain
    calls bit for bit, and the 64-bit layer's gradient within the 8-bit roundings."""
    import combine_get_dispatch_scan_amd.autograd as A
    x, logits, w1, w2 = _layer_case(6)
    K, E, I = 2, 8, 128
    go = _randn(_gen(7), *x.shape).bfloat16()
    lx, ll = x.clone().requires_grad_(), logits.clone().requires_grad_()
    l1, l2 = w1.clone().requires_grad_(), w2.bfloat16().requires_grad_()
    g = A.gate(ll, K, balance_coef=0.1)
    out = A.experts(lx, g.topk_idx, g.topk_weights, l1, l2)
    ((out * go).sum().float() + g.loss.sum()).backward()

    q1, q2 = ep.quantize_weights(w1, True), ep.quantize_weights(w2.bfloat16(), True)
    p = ep.gate(logits, K, balance_coef=0.1)
    lay = ep.get_dispatch_layout(p.topk_idx, E, 1)
    x8, xs, h = ep.dispatch(x, p.topk_weights, lay, True)
    a8, a_s, ck, cs = ep.swiglu_fp8(ep.grouped_gemm_fp8(x8, xs, q1.codes, q1.scales, h), h, checkpoint=True)
    y = ep.grouped_gemm_fp8(a8, a_s, q2.codes, q2.scales, h)
    assert torch.equal(out, ep.combine(y, h))
    gy, gw = ep.combine_backward(go, h, y=y)
    g8, gs = ep.quantize_rows(gy, h)
    gh, gh8, ghs = ep.swiglu_fp8_backward(ep.grouped_gemm_fp8(g8, gs, q2.codes_t, q2.scales_t, h), ck, cs, h)
    gx = ep.dispatch_backward(ep.grouped_gemm_fp8(gh8, ghs, q1.codes_t, q1.scales_t, h), h)
    assert torch.equal(lx.grad, gx)
    assert l1.grad.dtype == torch.float32 and torch.equal(l1.grad, ep.grouped_wgrad_fp8(gh, x8, xs, h, out_dtype=torch.float32))
    assert l2.grad.dtype == torch.bfloat16 and torch.equal(l2.grad, ep.grouped_wgrad_fp8(gy, a8, a_s, h))
    assert torch.equal(ll.grad, ep.gate_backward(logits, p, gw, torch.ones(1, device=x.device)))

    # the layer in 64 bits, its choice held
    x6, l6, a6, b6 = (t.double().detach().requires_grad_() for t in (x, logits, w1, w2.bfloat16()))
    pr = torch.softmax(l6, 1)
    sel = torch.gather(pr, 1, p.topk_idx)
    wt = sel / sel.sum(1, keepdim=True)
    n = p.num_tokens_per_expert.double()
    rows = []
    for t in range(x.shape[0]):
        acc = 0
        for k in range(K):
            e = int(p.topk_idx[t, k])
            hh = a6[e] @ x6[t]
            acc = acc + wt[t, k] * (b6[e] @ (torch.nn.functional.silu(hh[:I]) * hh[I:]))
        rows.append(acc)
    total = (torch.stack(rows) * go.double()).sum() + 0.1 * (E * n / (K * x.shape[0]) * pr.mean(0)).sum()
    total.backward()
    # the chain holds at most six E4M3 roundings of 2^-4 (x, w1, h, a or its gradient, w2, grad rows)
    for got, want in ((lx.grad, x6.grad), (l1.grad, a6.grad), (l2.grad, b6.grad), (ll.grad, l6.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 6 * 2.0 ** -4


def test_autograd_masked_pairs_and_frozen_inputs(ep):
    """Padding tokens get zero gradients; inputs without a gradient skip their products."""
    import combine_get_dispatch_scan_amd.autograd as A
    x, logits, w1, w2 = _layer_case(8)
    mask = torch.ones(x.shape[0], dtype=torch.bool, device=x.device)
    mask[50:] = False
    lx, ll = x.clone().requires_grad_(), logits.clone().requires_grad_()
    g = A.gate(ll, 2, balance_coef=0.1, token_mask=mask)
    out = A.experts(lx, g.topk_idx, g.topk_weights, w1, w2)
    assert not out[50:].any()
    out.float().square().sum().backward()
    assert lx.grad[:50].any() and not lx.grad[50:].any()
    assert ll.grad[:50].any() and not ll.grad[50:].any()
    assert torch.isfinite(lx.grad.float()).all() and torch.isfinite(ll.grad).all()
    l2 = w2.clone().requires_grad_()
    A.experts(x, g.topk_idx, g.topk_weights.detach(), w1, l2).float().sum().backward()
    assert torch.isfinite(l2.grad).all() and l2.grad.any()
    with torch.no_grad():
        assert torch.equal(A.experts(x, g.topk_idx, g.topk_weights, w1, w2), out)
    with pytest.raises(ValueError, match="do not fit"):
        A.experts(x, g.topk_idx, g.topk_weights, w2, w1)


def test_binding_refusals_on_the_gpu(ep):
    dev = _dev()
    x, xs, _ = _fp8_rows(_gen(1), 4, 256)
    w, ws = torch.zeros(2, 128, 256, dtype=torch.uint8, device=dev).view(F8), torch.zeros(2, 1, 2, device=dev)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(TypeError, match="groups"):
        ep.grouped_gemm_fp8(x, xs, w, ws, off.long())
    with pytest.raises(ValueError, match="one device"):
        ep.grouped_gemm_fp8(x, xs, w, ws, off.cpu())
    with pytest.raises(ValueError, match="groups"):
        ep.grouped_gemm_fp8(x, xs, w, ws, torch.zeros(4, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError, match="out must"):
        ep.grouped_gemm_fp8(x, xs, w, ws, off, out=torch.empty(4, 256, dtype=torch.bfloat16, device=dev))
    with pytest.raises(TypeError, match="out"):
        ep.grouped_wgrad_fp8(torch.zeros(4, 128, dtype=torch.bfloat16, device=dev), x, xs, off, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        ep.quantize_rows(torch.zeros(4, 512, dtype=torch.bfloat16, device=dev)[:, :256])
    with pytest.raises(ep.EpError, match="invalid dims"):
        ep.gate(torch.zeros(4, 8, device=dev), 9)
    with pytest.raises(ep.EpError, match="workspace too small"):
        ep.gate(torch.zeros(4, 8, device=dev), 2, ws=torch.empty(8, dtype=torch.uint8, device=dev))
    # no rows: nothing is launched on them
    e = torch.empty(0, 256, dtype=torch.uint8, device=dev).view(F8)
    es = torch.empty(0, 2, device=dev)
    assert ep.grouped_gemm_fp8(e, es, w, ws, off).shape == (0, 128)
    assert not ep.grouped_wgrad_fp8(torch.empty(0, 128, dtype=torch.bfloat16, device=dev), e, es, off).any()
    assert ep.quantize_rows(torch.empty(0, 256, dtype=torch.bfloat16, device=dev))[0].shape == (0, 256)
    assert ep.swiglu_fp8(torch.empty(0, 256, dtype=torch.bfloat16, device=dev), checkpoint=True)[2].shape == (0, 256)


def test_late_first_group_and_byte_codes(ep):
    """Groups that begin behind the first row and end before the last; codes passed as uint8."""
    dev = _dev()
    g = _gen(31)
    x, xs, _ = _fp8_rows(g, 200, 384)
    w, ws = (_randn(g, 3, 256, 384) * 50).to(F8), torch.rand(3, 2, 3, generator=g, device=dev) + 0.1
    off = torch.tensor([20, 20, 150, 190], dtype=torch.int32, device=dev)
    for expected in (1, 10, 50, 1000000):
        out = torch.full((200, 256), 5.0, dtype=torch.bfloat16, device=dev)
        ep.grouped_gemm_fp8(x.view(torch.uint8), xs, w.view(torch.uint8), ws, off, expected_rows=expected, out=out)
        assert (out[:20] == 5).all() and (out[190:] == 5).all() and (out[20:190] != 5).any(1).all()
    dw = ep.grouped_wgrad_fp8(_randn(g, 200, 256).bfloat16(), x, xs, off)
    assert not dw[0].any() and dw[1].any() and dw[2].any()


def test_reused_gate_workspace(ep):
    x = _randn(_gen(32), 500, 64)
    ws = torch.empty(ep.ep_gate_workspace_bytes(500, 64), dtype=torch.uint8, device=x.device)
    a, b, c = (ep.gate(x, 4, balance_coef=1.0, ws=t) for t in (ws, ws, None))
    assert torch.equal(a.loss, b.loss) and torch.equal(a.loss, c.loss) and torch.equal(a.topk_weights, c.topk_weights)


def test_autograd_without_tokens_and_under_capture(ep):
    import combine_get_dispatch_scan_amd.autograd as A
    dev = _dev()
    x = torch.zeros(0, 256, device=dev, dtype=torch.bfloat16, requires_grad=True)
    logits = torch.zeros(0, 8, device=dev, requires_grad=True)
    w1, w2 = (torch.randn(8, 256, n, device=dev, requires_grad=True) for n in (256, 128))
    g = A.gate(logits, 2, balance_coef=1.0)
    (A.experts(x, g.topk_idx, g.topk_weights, w1, w2).float().sum() + g.loss.sum()).backward()
    assert not w1.grad.any() and not w2.grad.any() and x.grad.shape == (0, 256)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="cannot be captured"):
        with torch.cuda.graph(graph):
            A.gate(w1.detach()[0].requires_grad_(), 2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_nan_logit_is_not_chosen_and_shows_in_the_loss(ep, score):
    x = _randn(_gen(33), 40, 100)
    x[7, 5] = math.nan
    x[9] = math.nan
    q = ep.gate(x, 8, score=score, balance_coef=1.0)
    ids = q.topk_idx.cpu()
    assert ((ids >= -1) & (ids < 100)).all() and 5 not in ids[7] and (ids[9] == -1).all()
    assert math.isnan(float(q.loss))
    keep = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(q.topk_idx[keep], ep.gate(x[keep].contiguous(), 8, score=score).topk_idx)
