"""CPU checks of how the expert layer's binding and autograd functions hold their
tensors: the library's calls are replaced by stand-ins on CPU tensors, everything
around them is the code that runs on the GPU."""
import contextlib
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


@pytest.fixture
def autograd(monkeypatch):
    import combine_get_dispatch_scan_amd.autograd as A
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
