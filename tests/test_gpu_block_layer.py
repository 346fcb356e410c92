"""GPU checks of the operators around the expert layer together, as a model's blocks use
them: norms, gate, 8-bit dispatch, products with 4-bit weights, combine and the next
block's norms; in every layout, captured and replayed, on several streams, and with
gradients.

Tolerances count roundings: bf16 rounds by at most 2^-8, E4M3 by 2^-4 of a value.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF = torch.bfloat16
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


def _case(seed, T=70, H=256, inner=128, E=8):
    g = _gen(seed)
    c = dict(x=_randn(g, T, H).to(BF), y=(_randn(g, T, H) * 0.5).to(BF), logits=_randn(g, T, E))
    c["w1"], c["w2"] = _randn(g, E, 2 * inner, H) * 0.1, _randn(g, E, H, inner) * 0.1
    c["norm"], c["post"], c["gate"] = 1 + 0.1 * _randn(g, H), 1 + 0.1 * _randn(g, H), 0.5 + _randn(g, 1, H) * 0.1
    return c


def _experts(ep, x8, xs, h, q1, q2, column_major=False):
    y1 = ep.grouped_gemm_fp4(x8, xs, q1.codes, q1.scales, h, column_major_scales=column_major)
    a8, a_s, _, _ = ep.swiglu_fp8(y1, h)
    return ep.grouped_gemm_fp4(a8, a_s, q2.codes, q2.scales, h)


def _block(ep, c, q1, q2, K=2, aligned=1, column_major=False, static_cap=0):
    """A block of experts between two norms: the first one's 8-bit rows are what is dispatched (in the static layout
    dispatch quantises the norm's bf16 rows itself)."""
    E = q1.codes.shape[0]
    n = ep.block_norm(c["x"], c["y"], weight=c["norm"], quantize=True, residual_scale=0.75)
    g = ep.gate(c["logits"], K)
    if static_cap:
        x8, xs, lay = ep.low_latency_dispatch(n.h, g.topk_idx, g.topk_weights, E, 1, static_cap, True)
        h = lay.handle
    else:
        lay = ep.get_dispatch_layout(g.topk_idx, E, 1, expert_alignment=aligned)
        x8, xs, h = ep.dispatch(n.codes, g.topk_weights, lay, True, x_scales=n.scales, column_major_scales=column_major)
    out = ep.combine(_experts(ep, x8, xs, h, q1, q2, column_major), h)
    m = ep.block_norm(n.x, out, weight=c["norm"], y_norm=True, y_weight=c["post"], gate=c["gate"], quantize=True)
    return m, n, g, out


def _experts64(rows, g, d1, d2):
    inner = d2.shape[2]
    want = torch.zeros_like(rows)
    for t in range(rows.shape[0]):
        for k in range(g.topk_idx.shape[1]):
            e = int(g.topk_idx[t, k])
            if e < 0:
                continue
            y = d1[e] @ rows[t]
            want[t] += g.topk_weights[t, k].double() * (d2[e] @ (torch.nn.functional.silu(y[:inner]) * y[inner:]))
    return want


def _unit(v, eps=1e-6):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def test_block_in_every_layout(ep):
    """The same bits through the dense, aligned and column-major layouts, and the 64-bit block within what its roundings
    add up to."""
    c = _case(1)
    q1, q2 = ep.quantize_weights_fp4(c["w1"]), ep.quantize_weights_fp4(c["w2"])
    m, n, g, out = _block(ep, c, q1, q2)
    for kw in (dict(aligned=64), dict(column_major=True), dict(aligned=128, column_major=True)):
        other, _, _, o = _block(ep, c, q1, q2, **kw)
        assert torch.equal(out, o), kw
        assert torch.equal(m.x, other.x) and torch.equal(m.h, other.h) and torch.equal(m.scales, other.scales)
    # the static layout against a dense one that quantises the same bf16 rows
    lay = ep.get_dispatch_layout(g.topk_idx, 8, 1)
    x8, xs, h = ep.dispatch(n.h, g.topk_weights, lay, True)
    _, _, _, o = _block(ep, c, q1, q2, static_cap=70)
    assert torch.equal(o, ep.combine(_experts(ep, x8, xs, h, q1, q2), h))

    x1 = 0.75 * c["x"].double() + c["y"].double()
    want = _experts64(_unit(x1) * c["norm"].double(), g, ep.dequantize_weights_fp4(q1).double(), ep.dequantize_weights_fp4(q2).double())
    # two E4M3 roundings (the dispatched rows, SwiGLU's output) and bf16's, under the largest two of E4M3 can be
    assert float((out.double() - want).norm() / want.norm()) < 2 * 2.0 ** -4
    # the second norm from the first one's rounded stream and the experts' rounded output: bf16 stores alone
    v = n.x.double() + c["gate"].double() * _unit(out.double()) * c["post"].double()
    for got, want in ((m.x, v), (m.h, _unit(v) * c["norm"].double())):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8
    want = _unit(v) * c["norm"].double()
    got = m.codes.double() * m.scales.double().repeat_interleave(128, 1)
    assert float((got - want).norm() / want.norm()) < 2.0 ** -4


def test_block_with_tokens_no_expert_takes(ep):
    """Tokens whose mask leaves no expert: their block output is zero, their stream goes on unchanged by it."""
    c = _case(2)
    q1, q2 = ep.quantize_weights_fp4(c["w1"]), ep.quantize_weights_fp4(c["w2"])
    mask = torch.ones(70, dtype=torch.bool, device=_dev())
    mask[10:30] = False
    n = ep.block_norm(c["x"], c["y"], weight=c["norm"], quantize=True)
    for live in (mask, torch.zeros_like(mask)):
        g = ep.gate(c["logits"], 2, token_mask=live)
        lay = ep.get_dispatch_layout(g.topk_idx, 8, 1)
        x8, xs, h = ep.dispatch(n.codes, g.topk_weights, lay, True, x_scales=n.scales)
        out = ep.combine(_experts(ep, x8, xs, h, q1, q2), h)
        assert not out[~live].any() and torch.isfinite(out.float()).all()
        m = ep.block_norm(n.x, out, weight=c["norm"], y_norm=True, y_weight=c["post"], gate=c["gate"])
        assert torch.equal(m.x[~live], n.x[~live]) and torch.isfinite(m.h.float()).all()


def _step(ep, c, q, ws, static=True):
    """A block forward, its norms backward, and its weights into 4 bits and back."""
    E, T = 8, c["x"].shape[0]
    q1, q2 = ep.quantize_weights_fp4(c["w1"]), q
    n = ep.block_norm(c["x"], c["y"], weight=c["norm"], y_norm=True, y_weight=c["post"], gate=c["gate"], quantize=True)
    g = ep.gate(c["logits"], 2)
    if static:
        x8, xs, lay = ep.low_latency_dispatch(n.h, g.topk_idx, g.topk_weights, E, 1, T, True)
        h = lay.handle
    else:
        lay = ep.get_dispatch_layout(g.topk_idx, E, 1)
        x8, xs, h = ep.dispatch(n.codes, g.topk_weights, lay, True, x_scales=n.scales)
    out = ep.combine(_experts(ep, x8, xs, h, q1, q2), h)
    m = ep.block_norm(n.x, out, weight=c["norm"])
    p = ep.block_norm_backward(c["x"], c["y"], grad_x=m.x, grad_h=m.h, weight=c["norm"], y_norm=True, y_weight=c["post"],
                               gate=c["gate"], ws=ws)
    return [n.x, n.h, n.codes.view(torch.uint8), n.scales, out, m.x, m.h, p.x, p.y, p.weight, p.y_weight, p.gate,
            ep.dequantize_weights_fp4(q1)]


@pytest.mark.parametrize("static", [True, False])
def test_block_captured_and_replayed(ep, static):
    """Two graphs that share a workspace, replayed in turn on new inputs with eager work between the replays: each
    equals the eager calls."""
    c = _case(3, T=40)
    q2 = ep.quantize_weights_fp4(c["w2"])
    ws = torch.empty(ep.ep_block_norm_workspace_bytes(40, 256), dtype=torch.uint8, device=_dev())
    bufs = [{k: v.clone() for k, v in c.items()} for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for b in bufs:
            _step(ep, b, q2, ws, static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, got = [], []
    for b in bufs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(_step(ep, b, q2, ws, static))
    for i in range(6):
        new = _case(10 + i, T=40)
        want = [t.clone() for t in _step(ep, new, q2, None, static)]
        for k, v in new.items():
            bufs[i % 2][k].copy_(v)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got[i % 2], want)):
            assert torch.equal(a, b), (i, j)


def test_blocks_on_two_streams(ep):
    """Each stream with tensors and workspaces of its own."""
    cases = [_case(20, T=300), _case(21, T=300)]
    q2 = ep.quantize_weights_fp4(cases[0]["w2"])
    want = [[t.clone() for t in _step(ep, c, q2, None, False)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(_step(ep, cases[i % 2], q2, None, False))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a, b), i


def test_work_on_a_side_stream_is_ordered_there(ep):
    """The calls go to the stream that is current: inputs written there just before, outputs read there just after."""
    c = _case(22, T=2000, H=1024)
    want = ep.block_norm(c["x"], c["y"], weight=c["norm"], quantize=True)
    w4 = ep.quantize_weights_fp4(c["w1"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, y, w = torch.zeros_like(c["x"]), torch.zeros_like(c["y"]), torch.zeros_like(c["w1"])
        for _ in range(20):
            x.copy_(c["x"])
            y.copy_(c["y"])
            w.copy_(c["w1"])
        n = ep.block_norm(x, y, weight=c["norm"], quantize=True)
        q = ep.quantize_weights_fp4(w)
        kept = n.h.clone(), n.codes.clone(), q.codes.clone(), q.scales.clone()
        x.zero_()
        y.zero_()
        w.zero_()
    s.synchronize()
    for a, b in zip(kept, (want.h, want.codes, w4.codes, w4.scales)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


_FORMS = r"""
import torch
import combine_get_dispatch_scan_amd as ep
g = torch.Generator(device="cuda")
g.manual_seed(0)
for G, rows, N, K in ((4, 4, 128, 256), (4, 4, 128, 384), (2, 2, 128, 8192), (2, 2, 128, 8320), (8, 4096, 512, 1024), (2, 16384, 2048, 512)):
    x = torch.randn(rows, K, generator=g, device="cuda").to(torch.float8_e4m3fn)
    w = ep.quantize_weights_fp4(torch.randn(G, N, K, generator=g, device="cuda"))
    off = torch.arange(0, rows + 1, rows // G, device="cuda", dtype=torch.int32)
    ep.grouped_gemm_fp4(x, torch.ones(rows, K // 128, device="cuda"), w.codes, w.scales, off)
    torch.cuda.synchronize()
for T, H, xt in ((5, 512, torch.bfloat16), (5, 2048, torch.bfloat16), (3, 32768, torch.float32)):
    x = torch.randn(T, H, generator=g, device="cuda").to(xt)
    w = torch.ones(H, device="cuda")
    ep.block_norm(x, weight=w)
    ep.block_norm_backward(x, grad_h=x.bfloat16(), weight=w)
    torch.cuda.synchronize()
"""


def test_every_form_is_reached(ep):
    """EP_DEBUG is read once a process, hence another one: each size takes the kernel its rule names."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FORMS], cwd=root, capture_output=True, text=True, timeout=100,
                       env=dict(os.environ, EP_DEBUG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    got = [l.split()[1] for l in r.stderr.splitlines() if l.startswith("[moe_ep]")]
    assert [n for n in got if n.startswith("grouped")] == ["grouped_gemm_fp4_" + n
                                                           for n in ("small", "stream", "stream", "small", "small", "tile")]
    threads = [int(l.split("block=(")[1].split(",")[0]) for l in r.stderr.splitlines() if l.startswith("[moe_ep] block_norm ")]
    assert threads == [256, 256, 1024]
    assert [n for n in got if n.startswith("block_norm")] == ["block_norm", "block_norm_backward", "block_norm_reduce"] * 3


def test_codes_and_scales_of_other_types(ep):
    """Codes as pairs of E2M1, scales as bytes: the same bits mean the same weights."""
    g = _gen(30)
    x, xs = (_randn(g, 40, 256) * 50).to(F8), torch.rand(40, 2, generator=g, device=_dev()) + 0.1
    q = ep.quantize_weights_fp4(_randn(g, 2, 128, 256))
    off = torch.tensor([0, 15, 40], dtype=torch.int32, device=_dev())
    want = ep.grouped_gemm_fp4(x, xs, q.codes, q.scales, off)
    pairs = q.codes.view(torch.float4_e2m1fn_x2)
    assert torch.equal(want, ep.grouped_gemm_fp4(x, xs, pairs, q.scales.view(torch.uint8), off))
    assert torch.equal(want, ep.grouped_gemm_fp4(x.view(torch.uint8), xs, pairs, q.scales, off))
    back = ep.dequantize_weights_fp4(ep.Fp4Weights(pairs, q.scales.view(torch.uint8)))
    assert torch.equal(back, ep.dequantize_weights_fp4(q))


def test_product_refusals_on_the_gpu(ep):
    dev = _dev()
    x, xs = torch.zeros(4, 256, dtype=torch.uint8, device=dev).view(F8), torch.zeros(4, 2, device=dev)
    w, ws = torch.zeros(2, 128, 128, dtype=torch.uint8, device=dev), torch.zeros(2, 128, 8, dtype=torch.uint8, device=dev)
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    for kw, err, msg in [
        (dict(groups=off.long()), TypeError, "groups"), (dict(groups=off[:2]), ValueError, "groups"),
        (dict(groups=off.cpu()), ValueError, "one device"), (dict(w=w.view(F8)), TypeError, "w must"),
        (dict(w=w.cpu()), ValueError, "one device"), (dict(w_scales=ws.float()), TypeError, "w_scales"),
        (dict(w_scales=ws[:, :, :4]), ValueError, "w_scales"), (dict(w_scales=ws.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "w_scales"),
        (dict(x=x.float()), TypeError, "x must"), (dict(x_scales=xs.double()), TypeError, "x_scales"),
        (dict(out=torch.zeros(4, 256, dtype=BF, device=dev)), ValueError, "out must"),
        (dict(out=torch.zeros(4, 128, device=dev)), TypeError, "out"),
    ]:
        with pytest.raises(err, match=msg):
            ep.grouped_gemm_fp4(**{**dict(x=x, x_scales=xs, w=w, w_scales=ws, groups=off), **kw})
    e, es = torch.empty(0, 256, dtype=torch.uint8, device=dev).view(F8), torch.empty(0, 2, device=dev)
    assert ep.grouped_gemm_fp4(e, es, w, ws, off).shape == (0, 128)
    with pytest.raises(ValueError, match="contiguous"):
        ep.quantize_weights_fp4(torch.zeros(1, 256, 128, device=dev).transpose(1, 2))
    with pytest.raises(TypeError, match="dtype"):
        ep.dequantize_weights_fp4(ep.Fp4Weights(w, ws), torch.float16)


# ----------------------------------------------------------------------------
# gradients
# ----------------------------------------------------------------------------

NAMES = ("x", "y", "weight", "y_weight", "gate")


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("T,H,xt", [(1, 128, BF), (70, 520, torch.float32), (300, 2048, BF)])
def test_autograd_norm_is_the_plain_calls(ep, channel, T, H, xt):
    import combine_get_dispatch_scan_amd.autograd as A
    g = _gen(40)
    t = dict(x=_randn(g, T, H).to(xt), y=_randn(g, T, H).to(BF), weight=_randn(g, H), y_weight=_randn(g, H),
             gate=(_randn(g, 1, H) if channel else _randn(g, T, 1)).to(BF))
    o = dict(y_norm=True, residual_scale=0.5, y_scale=2.0, eps=1e-5, weight_offset=1.0)
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    gx, gh = _randn(g, T, H).to(xt), _randn(g, T, H).to(BF)
    n, plain = A.block_norm(**leaves, **o), ep.block_norm(**t, **o)
    assert torch.equal(n.x, plain.x) and torch.equal(n.h, plain.h)
    torch.autograd.backward([n.x, n.h], [gx, gh])
    want = ep.block_norm_backward(grad_x=gx, grad_h=gh, **t, **o)
    for k in NAMES:
        assert leaves[k].grad.dtype == t[k].dtype and torch.equal(leaves[k].grad, getattr(want, k)), k
    for outs, kw in (((0,), dict(grad_x=gx)), ((1,), dict(grad_h=gh))):
        leaves = {k: v.clone().requires_grad_(k != "x") for k, v in t.items()}
        n = A.block_norm(**leaves, **o)
        torch.autograd.backward([(n.x, n.h)[i] for i in outs], [(gx, gh)[i] for i in outs])
        want = ep.block_norm_backward(need=NAMES[1:], **kw, **t, **o)
        assert leaves["x"].grad is None
        for k in NAMES[1:]:
            assert torch.equal(leaves[k].grad, getattr(want, k)), k


def test_autograd_two_blocks(ep):
    """Norm, gate, experts and norm twice, with weights that both blocks share: every gradient within the 8-bit roundings
    of the 64-bit blocks'."""
    import combine_get_dispatch_scan_amd.autograd as A
    c = _case(50, T=48)
    K, E, T, H, I = 2, 8, 48, 256, 128
    g = _gen(51)
    router = _randn(g, H, E) * H ** -0.5
    go = _randn(g, T, H).to(BF)
    leaves = {k: c[k].clone().requires_grad_() for k in ("x", "w1", "w2", "norm", "post", "gate")}
    lr = router.clone().requires_grad_()
    ids = []
    s = A.block_norm(leaves["x"], weight=leaves["norm"])
    for _ in range(2):
        gt = A.gate(s.h.float() @ lr, K)
        ids.append(gt.topk_idx)
        y = A.experts(s.h, gt.topk_idx, gt.topk_weights, leaves["w1"], leaves["w2"])
        s = A.block_norm(s.x, y, weight=leaves["norm"], y_norm=True, y_weight=leaves["post"], gate=leaves["gate"])
    torch.autograd.backward([s.h], [go])

    d = {k: v.detach().double().requires_grad_() for k, v in leaves.items()}
    dr = router.double().requires_grad_()
    x, h = d["x"], _unit(d["x"]) * d["norm"]
    for i in range(2):
        p = torch.softmax(h @ dr, 1)
        sel = torch.gather(p, 1, ids[i])
        wt = sel / sel.sum(1, keepdim=True)
        rows = []
        for t in range(T):
            acc = 0
            for k in range(K):
                e = int(ids[i][t, k])
                u = d["w1"][e] @ h[t]
                acc = acc + wt[t, k] * (d["w2"][e] @ (torch.nn.functional.silu(u[:I]) * u[I:]))
            rows.append(acc)
        x = x + d["gate"] * _unit(torch.stack(rows)) * d["post"]
        h = _unit(x) * d["norm"]
    h.backward(go.double())
    # a block's chain holds at most six E4M3 roundings of 2^-4 (rows, two weights, SwiGLU's input and output, gradient
    # rows); two blocks, twice that
    for k, leaf in (*leaves.items(), ("router", lr)):
        want = (d[k] if k != "router" else dr).grad
        assert float((leaf.grad.double() - want).norm() / want.norm()) < 12 * 2.0 ** -4, k


def test_autograd_norm_refuses_to_be_captured(ep):
    """The forward call refuses before anything is launched into the graph."""
    import combine_get_dispatch_scan_amd.autograd as A
    x = _randn(_gen(60), 4, 256).to(BF).requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="cannot be captured"):
            A.block_norm(x)
        n = ep.block_norm(x.detach())
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n.h, ep.block_norm(x.detach()).h)
