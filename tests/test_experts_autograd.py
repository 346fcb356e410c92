"""CPU checks of how the expert layer's binding and autograd functions hold their
tensors: the library's calls are replaced by stand-ins on CPU tensors, everything
around them is the code that runs on the GPU."""
import contextlib
import dataclasses
import gc
import weakref

import pytest

import combine_get_dispatch_scan_amd as ep

torch = pytest.importorskip("torch")


@pytest.fixture
def binding(monkeypatch):
    """The tensor forms of the gate's calls on CPU tensors: the C calls return success
    and write nothing."""
    from combine_get_dispatch_scan_amd import experts
    monkeypatch.setattr(experts, "_on", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(experts, "_stream", lambda t: 0)
    monkeypatch.setattr(experts, "_ptr", lambda t, *a, **k: None if t is None else t.data_ptr())
    monkeypatch.setattr(experts, "ep_gate", lambda *a: 0)
    monkeypatch.setattr(experts, "ep_gate_backward", lambda *a: 0)
    return experts


def test_gate_outputs_own_their_storage(binding):
    """A loss that is kept holds four bytes, not the workspace; changing one output in
    place does not count as a change of another."""
    g = binding.gate(torch.zeros(16384, 256), 8)
    small = (g.num_tokens_per_expert, g.num_valid, g.loss)
    assert [t.untyped_storage().nbytes() for t in small] == [4 * 256, 4, 4]
    assert all(not t._is_view() for t in small)
    g.num_tokens_per_expert.zero_()
    assert g.loss._version == 0 and g.num_valid._version == 0


def _stand_in_gate(logits, K, *, score="softmax", normalize=True, scale=1.0, balance_coef=0.0, token_mask=None):
    """The gate (softmax, normalised) in torch."""
    T, E = logits.shape
    live = torch.ones(T) if token_mask is None else token_mask.float()
    p = torch.softmax(logits, 1) * live[:, None]
    w, idx = p.topk(K, 1)
    idx = torch.where(live[:, None] > 0, idx, -1)
    n = torch.stack([(idx == e).sum() for e in range(E)]).to(torch.int32)
    V = live.sum()
    loss = balance_coef * (E * n / (K * V) * p.sum(0) / V).sum().reshape(1)
    if token_mask is not None and token_mask.dtype == torch.bool:
        token_mask = token_mask.view(torch.uint8)
    return ep.Gate(idx, w / w.sum(1, keepdim=True), n, V.to(torch.int32).reshape(1), loss, 0, normalize, scale,
                   balance_coef, token_mask)


def _stand_in_gate_backward(logits, g, grad_weights=None, grad_loss=None):
    """The gradient of the loss alone."""
    if grad_loss is None:
        return torch.zeros_like(logits)
    live = torch.ones(len(logits)) if g.token_mask is None else g.token_mask.float()
    with torch.enable_grad():
        x = logits.clone().requires_grad_()
        p = torch.softmax(x, 1) * live[:, None]
        E, K, V = x.shape[1], g.topk_idx.shape[1], g.num_valid
        (g.balance_coef * (E * g.num_tokens_per_expert / (K * V) * p.sum(0) / V).sum()).backward()
    return x.grad * grad_loss


class _Handle:
    """Of a dense layout whose pair count the host has not read."""
    num_recv = None

    class c:
        static_cap, expert_alignment = 0, 1


def _stand_in_layer(monkeypatch, A):
    """Dispatch, products, SwiGLU and combine as calls on CPU tensors that only keep the
    shapes (values are copies of the inputs); returns the list of what was called, with
    what was asked of it."""
    log = []

    def wide(x, n):
        return x[:, :1].float().expand(-1, n).contiguous()

    def scales(x):
        return torch.ones(len(x), x.shape[1] // 128)

    def dispatch(x, w, layout, fp8, *a):
        log.append(("dispatch", None))
        x = x.repeat_interleave(2, 0)
        return x, scales(x) if fp8 else None, _Handle()

    def weights(w, transposed=False):
        log.append(("weights", transposed))
        t = w.transpose(1, 2).contiguous()
        return ep.Fp8Weights(w, w[:, ::128, ::128], *((t, t[:, ::128, ::128]) if transposed else (None, None)))

    def product(x, xs, w, ws, h):
        y = wide(x, w.shape[1])
        log.append(("product", weakref.ref(y)))
        return y

    def swiglu(h, handle, checkpoint=False):
        log.append(("swiglu", checkpoint))
        a = wide(h, h.shape[1] // 2)
        return (a, scales(a)) + ((wide(h, h.shape[1]), scales(h)) if checkpoint else (None, None))

    def combine(y, h, w=None):
        return wide(y[::2], y.shape[1])

    def combine_backward(go, h, y=None, topk_weights=None, grad_y=None):
        log.append(("combine_backward", y is not None))
        return go.repeat_interleave(2, 0), None if y is None else torch.ones(len(go), 2)

    def wgrad(dy, x, xs, h, out_dtype=None):
        log.append(("wgrad", out_dtype))
        return torch.ones(4, dy.shape[1], x.shape[1], dtype=out_dtype)

    def swiglu_backward(da, ck, cs, h, quantize=True):
        log.append(("swiglu_backward", quantize))
        return (wide(da, ck.shape[1]),) + ((wide(da, ck.shape[1]), cs) if quantize else (None, None))

    class Layout:
        handle = _Handle()

    for name, f in (("_get_dispatch_layout", lambda *a: Layout()), ("_dispatch", dispatch),
                    ("quantize_weights", weights), ("grouped_gemm_fp8", product), ("swiglu_fp8", swiglu),
                    ("_combine", combine), ("_combine_backward", combine_backward), ("grouped_wgrad_fp8", wgrad),
                    ("quantize_rows", lambda x, h: (x, scales(x))), ("swiglu_fp8_backward", swiglu_backward),
                    ("_dispatch_backward", lambda g, h: wide(g[::2], g.shape[1]))):
        monkeypatch.setattr(A, name, f)
    return log


@pytest.fixture
def autograd(monkeypatch):
    import combine_get_dispatch_scan_amd.autograd as A
    monkeypatch.setattr(A, "_on", lambda *t: contextlib.nullcontext(), raising=False)
    monkeypatch.setattr(A, "_eager_only", lambda what: None)
    monkeypatch.setattr(A, "_gate_call", _stand_in_gate)
    monkeypatch.setattr(A, "_gate_backward", _stand_in_gate_backward)
    return A


@pytest.mark.parametrize("backward", [True, False])
def test_gate_keeps_nothing_alive(autograd, backward):
    """A node that holds its own outputs is never freed: after a step nothing of it is left."""
    kept = []
    for i in range(4):
        logits = torch.randn(6, 8, requires_grad=True)
        g = autograd.gate(logits, 2, balance_coef=0.1)
        if backward:
            (g.loss.sum() + g.topk_weights.square().sum()).backward()
        kept += [weakref.ref(t) for t in (logits, g.topk_idx, g.topk_weights, g.num_tokens_per_expert, g.num_valid, g.loss)]
        del logits, g
    gc.collect()
    assert [r() is None for r in kept] == [True] * len(kept)


def test_gate_refuses_changed_ids_and_counts(autograd):
    """What backward reads of the outputs is guarded by torch's version check; the loss,
    which it does not read, may be changed."""
    for name in ("topk_idx", "num_tokens_per_expert"):
        logits = torch.randn(6, 8, requires_grad=True)
        g = autograd.gate(logits, 2, balance_coef=0.1)
        getattr(g, name).zero_()
        with pytest.raises(RuntimeError, match="inplace"):
            g.loss.sum().backward()
    logits = torch.randn(6, 8, requires_grad=True)
    autograd.gate(logits, 2, balance_coef=0.1).loss.mul_(3.0).sum().backward()
    once = logits.grad.clone()
    logits.grad = None
    (3.0 * autograd.gate(logits, 2, balance_coef=0.1).loss.sum()).backward()
    assert torch.equal(once, logits.grad) and once.any()


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
def test_gate_refuses_changed_mask_and_token_count(autograd, dtype):
    for change in (lambda g, mask: mask.fill_(1), lambda g, mask: g.num_valid.fill_(6)):
        logits, mask = torch.randn(6, 8, requires_grad=True), torch.tensor([1, 1, 0, 1, 0, 1]).to(dtype)
        g = autograd.gate(logits, 2, balance_coef=0.1, token_mask=mask)
        change(g, mask)
        with pytest.raises(RuntimeError, match="inplace"):
            g.loss.sum().backward()
    logits, mask = torch.randn(6, 8, requires_grad=True), torch.tensor([1, 1, 0, 1, 0, 1]).to(dtype)
    autograd.gate(logits, 2, balance_coef=0.1, token_mask=mask).loss.sum().backward()
    assert logits.grad[0].any() and not logits.grad[2].any() and not logits.grad[4].any()


def test_second_derivatives_are_refused(autograd, monkeypatch):
    """The backward passes are kernels without a derivative of their own: differentiating
    through them raises instead of dropping terms."""
    logits = torch.randn(6, 8, requires_grad=True)
    plain, = torch.autograd.grad(autograd.gate(logits, 2, balance_coef=0.1).loss.sum(), logits)
    first, = torch.autograd.grad(autograd.gate(logits, 2, balance_coef=0.1).loss.sum(), logits, create_graph=True)
    assert torch.equal(plain, first) and not plain.requires_grad
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.square().sum().backward()
    _stand_in_layer(monkeypatch, autograd)
    x, w = torch.randn(6, 128, requires_grad=True), torch.rand(6, 2, requires_grad=True)
    w1, w2 = torch.randn(4, 256, 128), torch.randn(4, 128, 128)
    out = autograd.experts(x, torch.zeros(6, 2, dtype=torch.int64), w, w1, w2)
    first, = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.square().sum().backward()
    recv, handle = autograd.dispatch(x, torch.zeros(6, 2, dtype=torch.int64), w, 4, 1)
    first, = torch.autograd.grad(recv.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.square().sum().backward()
    y = torch.randn(12, 128, requires_grad=True)
    first, = torch.autograd.grad(autograd.combine(y, handle, w).square().sum(), y, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.square().sum().backward()


def _layer_inputs(dtype=torch.float32):
    return (torch.randn(6, 128), torch.zeros(6, 2, dtype=torch.int64), torch.rand(6, 2),
            torch.randn(4, 256, 128), torch.randn(4, 128, 128))


def test_experts_without_gradients_does_no_training_work(autograd, monkeypatch):
    """Inference with parameters writes no transposed weights and no checkpoint."""
    log = _stand_in_layer(monkeypatch, autograd)
    x, idx, w, w1, w2 = _layer_inputs()
    w1, w2 = torch.nn.Parameter(w1), torch.nn.Parameter(w2)
    for mode in (torch.no_grad, torch.inference_mode):
        log.clear()
        with mode():
            out = autograd.experts(x, idx, w, w1, w2)
        assert not out.requires_grad
        assert [v for k, v in log if k == "weights"] == [False, False]
        assert [v for k, v in log if k == "swiglu"] == [False]
    log.clear()
    out = autograd.experts(x, idx, w, w1, w2)
    assert [v for k, v in log if k == "swiglu"] == [True] and out.requires_grad
    out.sum().backward()
    assert w1.grad is not None and w2.grad is not None


@pytest.mark.parametrize("need", [(a, b, c, d) for a in (0, 1) for b in (0, 1) for c in (0, 1) for d in (0, 1)
                                  if a or b or c or d])
def test_experts_keeps_what_backward_reads(autograd, monkeypatch, need):
    """The second product's bf16 output is kept only for the gradient of the gate's weights,
    and each 8-bit tensor only where a gradient reads it."""
    log = _stand_in_layer(monkeypatch, autograd)
    x, idx, w, w1, w2 = _layer_inputs()
    for t, n in zip((x, w, w1, w2), need):
        t.requires_grad_(bool(n))
    want_x, want_w, want_1, want_2 = map(bool, need)
    out = autograd.experts(x, idx, w, w1, w2)
    products = [v for k, v in log if k == "product"]
    gc.collect()
    assert products[0]() is None and (products[1]() is not None) == want_w
    assert [v for k, v in log if k == "weights"] == [want_x, want_x or want_1]
    assert [v for k, v in log if k == "swiglu"] == [want_x or want_1]
    saved = out.grad_fn.saved_tensors
    assert sum(t is not None for t in saved) == 2 * (want_1 + want_2 + (want_x or want_1)) + want_w + \
        2 * (want_x + (want_x or want_1))
    out.sum().backward()
    assert [t.grad is not None for t in (x, w, w1, w2)] == [want_x, want_w, want_1, want_2]
    assert [v for k, v in log if k == "combine_backward"] == [want_w]
    assert sum(k == "wgrad" for k, _ in log) == want_1 + want_2


def test_experts_runs_on_its_tensors_device(autograd, monkeypatch):
    """Every call of the layer, the layout's included, is made with the tensors' device
    current, and all five tensors have to be on it."""
    _stand_in_layer(monkeypatch, autograd)
    given, depth = [], [0]

    @contextlib.contextmanager
    def on(*tensors):
        given.append(tensors)
        depth[0] += 1
        yield
        depth[0] -= 1

    monkeypatch.setattr(autograd, "_on", on)
    for name in ("_get_dispatch_layout", "_dispatch", "quantize_weights", "grouped_gemm_fp8", "swiglu_fp8", "_combine",
                 "_eager_only"):
        def call(*a, f=getattr(autograd, name), **k):
            assert depth[0] == 1
            return f(*a, **k)
        monkeypatch.setattr(autograd, name, call)
    x, idx, w, w1, w2 = _layer_inputs()
    autograd.experts(x, idx, w, w1, w2)
    assert [[id(t) for t in g] for g in given] == [[id(t) for t in (x, idx, w, w1, w2)]]
    assert depth == [0]


def test_experts_refuses_cpu_tensors():
    import combine_get_dispatch_scan_amd.autograd as A
    with pytest.raises(ValueError, match="expected GPU tensors"):
        A.experts(*_layer_inputs())
    with pytest.raises(ValueError, match="expected GPU tensors"):
        A.gate(torch.zeros(4, 8), 2)


def test_experts_refuses_choices_that_do_not_fit(autograd, monkeypatch):
    """Dispatch reads a row of x and a weight for every choice: fewer rows or weights than
    choices are refused before any call."""
    log = _stand_in_layer(monkeypatch, autograd)
    x, idx, w, w1, w2 = _layer_inputs()
    for bad in ((x[:5], idx, w), (x, idx[:5], w), (x, idx, w[:5]), (x, idx, w[:, :1]), (x, idx[:, 0], w[:, 0]),
                (x[0], idx, w), (x[None], idx, w)):
        with pytest.raises(ValueError, match="do not fit"):
            autograd.experts(*bad, w1, w2)
    for a, b in ((w1[0], w2), (w1, w2[0]), (w1[:3], w2), (w1[:, :128], w2), (w1[:, :, :64], w2), (w1, w2[:, :64])):
        with pytest.raises(ValueError, match="do not fit"):
            autograd.experts(x, idx, w, a, b)
    assert not log


def test_gate_backward_refuses_a_gate_that_does_not_fit(binding):
    logits = torch.zeros(6, 8)
    g = binding.gate(logits, 2, token_mask=torch.ones(6, dtype=torch.bool))
    binding.gate_backward(logits, g)
    one = torch.zeros(1, dtype=torch.int32)
    for name, bad in (("topk_idx", g.topk_idx[:5]), ("num_tokens_per_expert", one), ("num_valid", one[:0]),
                      ("token_mask", g.token_mask[:5])):
        with pytest.raises(ValueError, match=name):
            binding.gate_backward(logits, dataclasses.replace(g, **{name: bad}))


def test_backward_is_not_captured_either(autograd, monkeypatch):
    """A backward pass captured while its forward pass was eager is refused before any call."""
    log = _stand_in_layer(monkeypatch, autograd)
    x, idx, w, w1, w2 = _layer_inputs()
    out = autograd.experts(x.requires_grad_(), idx, w, w1, w2)
    logits = torch.randn(6, 8, requires_grad=True)
    g = autograd.gate(logits, 2, balance_coef=0.1)

    def capturing(what):
        raise RuntimeError(f"{what} cannot be captured into a graph")

    monkeypatch.setattr(autograd, "_eager_only", capturing)
    n = len(log)
    with pytest.raises(RuntimeError, match="cannot be captured"):
        out.sum().backward()
    with pytest.raises(RuntimeError, match="cannot be captured"):
        g.loss.sum().backward()
    assert len(log) == n and x.grad is None and logits.grad is None
