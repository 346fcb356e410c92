"""CPU checks of block_norm under autograd: the two calls of the library are replaced by
their formulas in torch on CPU tensors, everything around them is the code that runs on
the GPU."""
import contextlib
import gc
import weakref

import pytest

import combine_get_dispatch_scan_amd as ep

torch = pytest.importorskip("torch")

NAMES = ("x", "y", "weight", "y_weight", "gate")


def _formula(x, y, weight, y_weight, gate, norm, y_norm, residual_scale, y_scale, eps, weight_offset):
    def unit(t):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + eps)

    v = x
    if y is not None:
        z = unit(y) if y_norm else y
        z = z if y_weight is None else z * (weight_offset + y_weight)
        v = residual_scale * x + y_scale * z * (1.0 if gate is None else gate)
    h = None
    if norm:
        h = unit(v) if weight is None else unit(v) * (weight_offset + weight)
    return v, h


@pytest.fixture
def autograd(monkeypatch):
    import combine_get_dispatch_scan_amd.autograd as A
    log = []

    def forward(x, y=None, **o):
        assert not any(t is not None and t.requires_grad for t in (x, y, o["weight"], o["y_weight"], o["gate"]))
        with torch.no_grad():
            v, h = _formula(x, y, **o)
        return ep.BlockNorm(x if y is None else v, h)

    def backward(x, y=None, *, grad_x, grad_h, need, **o):
        assert all(t is None or t.is_contiguous() for t in (grad_x, grad_h))
        log.append((tuple(need), grad_x is not None, grad_h is not None))
        given = dict(x=x, y=y, **{n: o.pop(n) for n in NAMES[2:]})
        with torch.enable_grad():
            leaves = {n: None if t is None else t.detach().clone().requires_grad_(n in need) for n, t in given.items()}
            outs = [(t, g) for t, g in zip(_formula(**leaves, **o), (grad_x, grad_h)) if t is not None and g is not None]
            torch.autograd.backward([t for t, _ in outs], [g for _, g in outs])
        return ep.BlockNormGrads(**{n: leaves[n].grad if leaves[n] is not None else None for n in NAMES})

    monkeypatch.setattr(A, "_on", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(A, "_eager_only", lambda what: None)
    monkeypatch.setattr(A, "_block_norm_call", forward)
    monkeypatch.setattr(A, "_block_norm_backward", backward)
    A.log = log
    yield A
    del A.log


def _inputs(channel=False, **skip):
    torch.manual_seed(5)
    t = dict(x=torch.randn(6, 16), y=torch.randn(6, 16), weight=torch.rand(16), y_weight=torch.rand(16),
             gate=torch.rand(1, 16) if channel else torch.rand(6, 1))
    return {n: None if n in skip else v.double().requires_grad_() for n, v in t.items()}


OPTIONS = dict(y_norm=True, residual_scale=0.5, y_scale=2.0, eps=1e-3, weight_offset=1.0)


@pytest.mark.parametrize("channel", [False, True])
def test_gradients_are_differences(autograd, channel):
    t = _inputs(channel)

    def f(*tensors):
        n = autograd.block_norm(**dict(zip(NAMES, tensors)), **OPTIONS)
        return n.x, n.h

    assert torch.autograd.gradcheck(f, [t[n] for n in NAMES])
    only_h = lambda x, w: autograd.block_norm(x, weight=w).h  # noqa: E731
    assert torch.autograd.gradcheck(only_h, [t["x"], t["weight"]])
    only_x = lambda x, y, g: autograd.block_norm(x, y, gate=g, norm=False).x  # noqa: E731
    assert torch.autograd.gradcheck(only_x, [t["x"], t["y"], t["gate"]])


def test_outputs_and_what_backward_is_asked_for(autograd):
    t = _inputs()
    n = autograd.block_norm(t["x"], weight=t["weight"])
    assert n.x is t["x"] and n.codes is None
    n = autograd.block_norm(t["x"], t["y"], norm=False)
    assert n.h is None and n.x.requires_grad
    for need in range(1, 32):
        for name, bit in zip(NAMES, range(5)):
            t[name].requires_grad_(bool(need >> bit & 1)).grad = None
        wanted = tuple(n for n in NAMES if t[n].requires_grad)
        n = autograd.block_norm(**t, **OPTIONS)
        autograd.log.clear()
        n.h.sum().backward()
        # what no output needs does not arrive as zeros
        assert autograd.log == [(wanted, False, True)]
        assert all((t[name].grad is not None) == (name in wanted) for name in NAMES)
    n = autograd.block_norm(**t, **OPTIONS)
    autograd.log.clear()
    n.x.t().sum().backward()          # an expanded gradient
    assert autograd.log == [(NAMES, True, False)]


def test_without_gradients_nothing_is_kept(autograd):
    t = _inputs()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            n = autograd.block_norm(**t, **OPTIONS)
        assert not n.x.requires_grad and not n.h.requires_grad


def test_nothing_is_kept_alive(autograd):
    kept = []
    for i in range(3):
        t = _inputs()
        n = autograd.block_norm(**t, **OPTIONS)
        if i:
            (n.x.sum() + n.h.sum()).backward()
        kept += [weakref.ref(v) for v in (*t.values(), n.x, n.h)]
        del t, n
    gc.collect()
    assert [r() is None for r in kept] == [True] * len(kept)


def test_changed_inputs_are_refused(autograd):
    for name in NAMES:
        t = _inputs()
        n = autograd.block_norm(**t, **OPTIONS)
        with torch.no_grad():
            t[name].mul_(2.0)
        with pytest.raises(RuntimeError, match="inplace"):
            n.h.sum().backward()


def test_second_derivatives_are_refused(autograd):
    t = _inputs()
    first, = torch.autograd.grad(autograd.block_norm(**t, **OPTIONS).h.sum(), t["x"], create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        first.square().sum().backward()


def test_capture_is_refused(autograd, monkeypatch):
    t = _inputs()
    n = autograd.block_norm(**t, **OPTIONS)

    def capturing(what):
        raise RuntimeError(f"{what} cannot be captured into a graph")

    monkeypatch.setattr(autograd, "_eager_only", capturing)
    with pytest.raises(RuntimeError, match="the backward pass of block_norm cannot be captured"):
        n.h.sum().backward()
    with pytest.raises(RuntimeError, match="block_norm cannot be captured"):
        autograd.block_norm(**t, **OPTIONS)
    assert not autograd.log and t["x"].grad is None


def test_cpu_tensors_are_refused():
    import combine_get_dispatch_scan_amd.autograd as A
    with pytest.raises(ValueError, match="expected GPU tensors"):
        A.block_norm(torch.zeros(4, 8))
