"""GPU checks of the expert layer where its formulas are hard to hold (sigmoid scores
far from zero, padding rows on the way back, arguments at the ends of their range),
and of the form of a kernel that a call takes.  Tolerances count roundings as in
test_gpu_experts.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_gpu_experts import U, _check_wgrad, _dev, _gen, _layer_case, _randn

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ----------------------------------------------------------------------------
# sigmoid scores far from zero
# ----------------------------------------------------------------------------

def _sigmoid_gate64(x, idx, normalize, scale, coef, gw, gl):
    """Weights, loss, gradient and its terms' magnitudes, for the choice idx, from
    log s = -log(1 + e^-x) in 64 bits: no score underflows or cancels.  With q = s / max s,
        w = q_k / sum of the chosen q  (or s_k),    p = q / sum q,
        dl = (1 - s) (p (d - <p, d>) + wn (g - <g, wn>))      (normalised; else s g)"""
    T, E = x.shape
    K = idx.shape[1]
    ls = -np.logaddexp(0.0, -x)
    s, rest = np.exp(ls), np.exp(-np.logaddexp(0.0, x))        # s and 1 - s
    q = np.exp(ls - ls.max(1, keepdims=True))
    p = q / q.sum(1, keepdims=True)
    sel = np.zeros((T, E), bool)
    np.put_along_axis(sel, idx, True, 1)
    part = np.where(sel, ls, -np.inf)
    wn = np.where(sel, np.exp(part - part.max(1, keepdims=True)), 0.0)
    wn = wn / wn.sum(1, keepdims=True) if normalize else np.where(sel, s, 0.0)
    n = sel.sum(0)
    f = E * n / (K * T)
    loss = coef * (f * p.sum(0)).sum() / T
    g = np.zeros((T, E))
    np.put_along_axis(g, idx, gw * scale, 1)
    d = (coef * gl * f / T)[None, :]
    back = (g * wn).sum(1, keepdims=True) if normalize else 0.0
    mag = (np.abs(g) * wn).sum(1, keepdims=True) if normalize else 0.0
    dl = rest * (p * (d - (p * d).sum(1, keepdims=True)) + wn * (g - back))
    mg = rest * (p * (np.abs(d) + (p * np.abs(d)).sum(1, keepdims=True)) + wn * (np.abs(g) + mag))
    return np.take_along_axis(wn, idx, 1) * scale, loss, dl, mg


def _far_logits(where, T, E, dtype):
    u = torch.rand(T, E, generator=_gen(T + E), device=_dev())
    x = {"low": -80 - 40 * u, "vanishing": -104 + 17 * u, "lowest": torch.full_like(u, torch.finfo(dtype).min),
         "saturated": 12 + 18 * u, "both": torch.where(u < 0.5, -100 + 60 * u, 20 + 30 * u)}[where]
    return x.to(dtype)


def _check_far(ep, where, E, K, dtype, normalize):
    T, scale, coef = 37, 1.5, 0.5
    x = _far_logits(where, T, E, dtype)
    g = _gen(3)
    gw, gl = _randn(g, T, K), torch.ones(1, device=x.device)
    q = ep.gate(x, K, score="sigmoid", normalize=normalize, scale=scale, balance_coef=coef)
    got = ep.gate_backward(x, q, gw, gl)
    x64 = x.double().cpu().numpy()
    w, loss, dl, mag = _sigmoid_gate64(x64, q.topk_idx.cpu().numpy(), normalize, scale, coef,
                                       gw.double().cpu().numpy(), 1.0)
    # a score: the logit's distance from the largest (one rounding, times the exponent's size), the
    # exponential and the quotient (2 u each), the sum of E positive terms (at most 16 + 6 in a chain)
    rel = (2 * (x64.max(1) - x64.min(1)).max() + 40) * U
    # fp32's normal numbers end at 1.2e-38: factors of at most 100 beside them
    tiny = 1e-36
    assert (np.abs(q.topk_weights.double().cpu().numpy() - w) <= 2 * rel * w + tiny).all()
    if normalize:
        assert (np.abs(q.topk_weights.double().sum(1).cpu().numpy() - scale) <= 2 * (rel + K * U) * scale).all()
    assert abs(float(q.loss) - loss) <= (rel + 100 * U) * loss + tiny
    out = 2.0 ** -8 if dtype == torch.bfloat16 else U
    assert (np.abs(got.double().cpu().numpy() - dl) <= 4 * rel * mag + out * np.abs(dl) + tiny).all()


FAR = [(e, k, d) for e, k in ((8, 3), (64, 4), (300, 8), (1000, 4)) for d in (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("where", ["low", "vanishing", "lowest"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E,K,dtype", FAR)
def test_sigmoid_gate_at_low_logits(ep, where, normalize, E, K, dtype):
    """Scores under fp32's smallest number still have ratios: weights sum to the scale, the
    probabilities of the balance loss to one, and gradients are finite."""
    _check_far(ep, where, E, K, dtype, normalize)


@pytest.mark.parametrize("where", ["saturated", "both"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E,K,dtype", FAR)
def test_sigmoid_gate_at_saturated_logits(ep, where, normalize, E, K, dtype):
    """Scores near one: 1 - s is e^-x, not what a subtraction leaves of it."""
    _check_far(ep, where, E, K, dtype, normalize)


# ----------------------------------------------------------------------------
# padding rows of an aligned layout on the way back
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("alignment", [64, 128])
def test_weight_gradients_of_an_aligned_layout(ep, alignment):
    """The rows combine's backward pass writes go into the weight gradient with the padding
    rows of their blocks: whatever the memory held before, those add nothing."""
    x, logits, w1, w2 = _layer_case(21)
    q1, q2 = ep.quantize_weights(w1, True), ep.quantize_weights(w2, True)
    go = _randn(_gen(22), *x.shape).bfloat16()

    def grads(align):
        g = ep.gate(logits, 2)
        lay = ep.get_dispatch_layout(g.topk_idx, 8, 1, expert_alignment=align)
        x8, xs, h = ep.dispatch(x, g.topk_weights, lay, True)
        a8, a_s, ck, cs = ep.swiglu_fp8(ep.grouped_gemm_fp8(x8, xs, q1.codes, q1.scales, h), h, checkpoint=True)
        y = ep.grouped_gemm_fp8(a8, a_s, q2.codes, q2.scales, h)
        spoilt = torch.full((x8.shape[0], x.shape[1]), float("nan"), dtype=torch.bfloat16, device=x.device)
        del spoilt                                  # the allocator hands this memory out again
        gy, gw = ep.combine_backward(go, h, y=y)
        g8, gs = ep.quantize_rows(gy, h)
        gh, gh8, ghs = ep.swiglu_fp8_backward(ep.grouped_gemm_fp8(g8, gs, q2.codes_t, q2.scales_t, h), ck, cs, h)
        gx = ep.dispatch_backward(ep.grouped_gemm_fp8(gh8, ghs, q1.codes_t, q1.scales_t, h), h)
        f32 = torch.float32
        return (gx, gw, ep.grouped_wgrad_fp8(gh, x8, xs, h, out_dtype=f32),
                ep.grouped_wgrad_fp8(gy, a8, a_s, h, out_dtype=f32))

    for a, b in zip(grads(alignment), grads(1)):
        # the same rows in the same order, zeros behind them
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------
# arguments at the ends of their range
# ----------------------------------------------------------------------------

def test_expected_rows_at_the_largest_number():
    """The tile for many rows, also where rows + 255 pass 2^31 (EP_DEBUG is read once per
    process, so a child process makes the call)."""
    _dev()
    code = (
        "import sys; sys.path.insert(0, %r)\n"
        "import torch, combine_get_dispatch_scan_amd as ep\n"
        "d = torch.device('cuda:0')\n"
        "w = ep.quantize_weights(torch.randn((2, 256, 256), device=d))\n"
        "x, xs = ep.quantize_rows(torch.randn((64, 256), device=d).bfloat16())\n"
        "off = torch.tensor([0, 40, 64], dtype=torch.int32, device=d)\n"
        "for n in (100000, 2**31 - 1):\n"
        "    ep.grouped_gemm_fp8(x, xs, w.codes, w.scales, off, expected_rows=n)\n"
        "torch.cuda.synchronize()\n" % os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100,
                       env=dict(os.environ, EP_DEBUG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l.split()[1] for l in r.stderr.splitlines() if l.startswith("[moe_ep] grouped_gemm")]
    assert lines == ["grouped_gemm_tile"] * 2


# ----------------------------------------------------------------------------
# choice of a form
# ----------------------------------------------------------------------------

def _launches(calls):
    """What a child process prints of its expert-layer launches: (kernel, threads of a workgroup)."""
    _dev()
    code = (
        "import sys; sys.path.insert(0, %r)\n"
        "import torch, combine_get_dispatch_scan_amd as ep\n"
        "d = torch.device('cuda:0')\n"
        "def rows(r, k): return torch.zeros((r, k), dtype=torch.uint8, device=d), torch.zeros((r, k // 128), device=d)\n"
        "def off(g, m): return torch.arange(g + 1, dtype=torch.int32, device=d) * m\n"
        "%s\ntorch.cuda.synchronize()\n" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), calls))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100,
                       env=dict(os.environ, EP_DEBUG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    return [(l.split()[1], int(l.split("block=(")[1].split(",")[0])) for l in r.stderr.splitlines()
            if l.startswith("[moe_ep] grouped")]


def test_form_of_the_weight_gradient():
    """The smaller tile below 128 rows a group, and up to 128 tiles a group; from 512 rows on
    only below 512 tiles in all."""
    got = _launches(
        "for g, n, k, m in ((2, 2048, 4096, 600), (2, 2048, 4224, 600), (2, 2048, 4224, 127), (2, 2816, 4096, 128),\n"
        "                   (4, 2048, 4096, 511), (4, 2048, 4096, 512)):\n"
        "    x, xs = rows(g * m, k)\n"
        "    ep.grouped_wgrad_fp8(torch.zeros((g * m, n), dtype=torch.bfloat16, device=d), x, xs, off(g, m))\n")
    assert [b for _, b in got] == [256, 512, 256, 512, 256, 512]


@pytest.mark.parametrize("N,K", [(2944, 2944), (640, 16384), (16512, 384)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_weight_gradient_larger_tile(ep, N, K, dtype):
    """The larger tile (rows and tiles past the choice above), with partly filled tiles on
    both sides, stages of one row, groups without rows, and every way rows are laid out."""
    dt = getattr(torch, dtype)
    _check_wgrad(ep, [193, 0, 321], N, K, dt)
    _check_wgrad(ep, [300, 1], N, K, dt, column_major=True)
    _check_wgrad(ep, [130, 5], N, K, dt, stride=160)


def test_form_of_the_product():
    """By the typical rows of a group up to 16, then 64 x 64 tiles up to 512 of them."""
    got = _launches(
        "for g, n, m in ((4, 256, 8), (4, 256, 16), (4, 256, 17), (32, 512, 128), (32, 512, 129), (16, 4096, 32)):\n"
        "    x, xs = rows(g * m, 256)\n"
        "    w, ws = torch.zeros((g, n, 256), dtype=torch.uint8, device=d), torch.zeros((g, n // 128, 2), device=d)\n"
        "    for e in (m, 0):\n"
        "        ep.grouped_gemm_fp8(x, xs, w, ws, off(g, m), expected_rows=e)\n")
    # (the skinny forms share their name)
    want = ["grouped_gemm_skinny"] * 4 + ["grouped_gemm_tile"] * 2
    assert [k for k, _ in got] == [k for k in want for _ in (0, 1)]


# ----------------------------------------------------------------------------
# autograd
# ----------------------------------------------------------------------------

def test_training_steps_keep_no_memory(ep):
    """What is allocated after a step of gate and experts is what was before it."""
    import gc

    import combine_get_dispatch_scan_amd.autograd as A
    x, logits, w1, w2 = _layer_case(40, T=500)
    mask = torch.rand(500, generator=_gen(41), device=x.device) > 0.1
    params = [t.requires_grad_() for t in (logits, w1, w2)]

    def step(backward):
        g = A.gate(logits, 2, balance_coef=0.1, token_mask=mask)
        out = A.experts(x, g.topk_idx, g.topk_weights, w1, w2)
        if backward:
            (out.float().square().mean() + g.loss.sum()).backward()
            for p in params:
                p.grad = None

    sizes = []
    for i in range(8):
        step(backward=i % 2 == 0)
        gc.collect()
        sizes.append(torch.cuda.memory_allocated())
    assert len(set(sizes[1:])) == 1, sizes


def test_changes_between_forward_and_backward(ep):
    import combine_get_dispatch_scan_amd.autograd as A
    x, logits, w1, w2 = _layer_case(42)
    logits.requires_grad_()
    mask = torch.ones(len(x), dtype=torch.bool, device=x.device)
    for change in (lambda g: mask.fill_(0), lambda g: g.num_tokens_per_expert.zero_(), lambda g: g.topk_idx.fill_(0)):
        mask.fill_(1)
        g = A.gate(logits, 2, balance_coef=0.1, token_mask=mask)
        change(g)
        with pytest.raises(RuntimeError, match="inplace"):
            g.loss.sum().backward()
    mask.fill_(1)
    g = A.gate(logits, 2, balance_coef=0.1, token_mask=mask)
    g.loss.mul_(2.0).sum().backward()
    one = torch.ones(1, device=x.device)
    assert torch.equal(logits.grad, ep.gate_backward(logits.detach(), ep.gate(logits.detach(), 2, balance_coef=0.1),
                                                     None, 2 * one))
    # a second derivative is refused, the first one under create_graph is not
    out = A.experts(x.requires_grad_(), g.topk_idx, g.topk_weights.detach(), w1, w2)
    first, = torch.autograd.grad(out.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.float().square().sum().backward()


def test_inference_with_parameters(ep):
    """The same bits without gradients, and no more memory than the forward pass needs."""
    import combine_get_dispatch_scan_amd.autograd as A
    x, logits, w1, w2 = _layer_case(43, T=300)
    g = ep.gate(logits, 2)
    want = A.experts(x, g.topk_idx, g.topk_weights, w1, w2)
    w1, w2 = torch.nn.Parameter(w1), torch.nn.Parameter(w2)
    assert torch.equal(A.experts(x, g.topk_idx, g.topk_weights, w1, w2), want)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(A.experts(x, g.topk_idx, g.topk_weights, w1, w2), want)
