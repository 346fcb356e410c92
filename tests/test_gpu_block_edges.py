"""GPU checks of the norms around a block at the ends of their values' range, and of many
rows a workgroup."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_block import BF, _check_norm, _check_norm_backward, _dev, _gen, _norm_case, _randn  # noqa: E402

F32 = torch.float32


# a wave, workgroups with one and two vectors, with factors read again, with four vectors; not powers of two among them
@pytest.mark.parametrize("H", [8, 1000, 1032, 7168, 16384, 32768])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("gate", ["token", "channel"])
def test_block_norm_of_large_values(ep, H, xt, gate):
    """Rows whose mean squares fp32 still holds (values just below 2^63), where the sum of the squares would be infinite."""
    o = _norm_case(H, 6, H, xt, F32, gate=gate)
    g = _gen(H + 1)
    top = 2.0 ** 63 * (1 - 2.0 ** -8)
    large = lambda: (1 - torch.rand(6, H, generator=g, device=_dev()) / 4) * (_randn(g, 6, H).sign() * top)  # noqa: E731
    o["x"], o["y"] = large().to(xt), large().to(BF)
    o["residual_scale"] = 1.0
    # x' = x + (at most a few): its mean square is below 2^126
    n = _check_norm(ep, o, quantize=H % 128 == 0)
    assert n.h.abs().amax(1).gt(0.1).all() and torch.isfinite(n.h.float()).all()
    _check_norm_backward(ep, o, H)
    # y without a norm of its own, and alone
    o["residual_scale"], o["y_norm"], o["y_weight"] = 0.25, False, None
    o["gate"] = o["gate"].clamp(-0.5, 0.5)
    _check_norm(ep, o)
    _check_norm_backward(ep, o, H + 1)
    _check_norm(ep, dict(o, y=None, gate=None, residual_scale=1.0))


# NaNs as arithmetic makes them, with every bit set (memory filled with 0xFF), and signalling
@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, -1, 0x7FFF8000, 0x7F800001])
@pytest.mark.parametrize("H", [256, 2048, 8320])
def test_block_norm_keeps_every_nan(ep, bits, H):
    """A NaN of any bits in the 32-bit stream, its gradient, a weight or a gate is a NaN in all outputs it reaches."""
    def at(shape, *where):
        t = _randn(g, *shape)
        t.view(torch.int32)[where] = bits
        return t

    g = _gen(H)
    x, y, w = _randn(g, 5, H), _randn(g, 5, H).to(BF), _randn(g, H)
    bad = at((5, H), 2, 7)
    live = [0, 1, 3, 4]
    for n in (ep.block_norm(bad, quantize=True), ep.block_norm(bad, y, weight=w, quantize=True)):
        assert torch.isnan(n.x[2, 7]) and int(torch.isnan(n.x).sum()) == 1
        assert torch.isnan(n.h[2]).all() and torch.isnan(n.codes[2].float()).all()
        assert torch.isfinite(n.h[live].float()).all() and torch.isfinite(n.codes[live].float()).all()
    n = ep.block_norm(x, weight=at((H,), 9), quantize=True)
    assert torch.isnan(n.h[:, 9]).all() and int(torch.isnan(n.h).sum()) == 5 and torch.isnan(n.codes[:, 9].float()).all()
    n = ep.block_norm(x.to(BF), y, gate=at((5, 1), 3, 0))
    assert torch.isnan(n.x[3]).all() and torch.isnan(n.h[3]).all() and int(torch.isnan(n.x).sum()) == H
    # the bf16 gradients of y and of bf16 parameters
    o = dict(weight=w.to(BF), y_norm=True, y_weight=w.to(BF), gate=w[None].to(BF))
    q = ep.block_norm_backward(x, y, grad_x=bad, grad_h=y, **o)
    assert torch.isnan(q.y[2]).all() and torch.isnan(q.y_weight[7]) and torch.isnan(q.gate[0, 7])
    assert torch.isfinite(q.y[live].float()).all() and torch.isfinite(q.x[live]).all()
    q = ep.block_norm_backward(bad, y, grad_x=x, grad_h=y, **o)
    assert torch.isnan(q.x[2]).all() and torch.isnan(q.y[2]).all() and torch.isnan(q.weight).all()
    q = ep.block_norm_backward(x, y, grad_x=bad, norm=False, gate=_randn(g, 5, 1).to(BF))
    assert torch.isnan(q.gate[2, 0]) and torch.isfinite(q.gate[live].float()).all()


def test_autograd_of_gradients_at_odd_offsets(ep):
    """Outputs joined with something of an odd length: their gradients are dense and begin anywhere."""
    import combine_get_dispatch_scan_amd.autograd as A
    T, H, E, I = 24, 256, 4, 128
    g = _gen(5)
    w1, w2 = _randn(g, E, 2 * I, H) * 0.1, _randn(g, E, H, I) * 0.1
    idx = torch.stack([torch.randperm(E, generator=g, device=_dev())[:2] for _ in range(T)])
    start = torch.ones(1, dtype=BF, device=_dev())

    def grads(f, go, *leaves):
        leaves = [t.clone().requires_grad_() for t in leaves]
        got = []
        for odd in (False, True):
            outs = f(*leaves)
            if odd:
                torch.cat([start, *(o.flatten() for o in outs)]).backward(torch.cat([start, *(t.flatten() for t in go)]))
            else:
                torch.autograd.backward(outs, go)
            got.append([t.grad for t in leaves])
            for t in leaves:
                t.grad = None
        for a, b in zip(*got):
            assert a.any() and torch.equal(a, b)

    x, y = _randn(g, T, H).to(BF), _randn(g, T, H).to(BF)
    go = [_randn(g, T, H).to(BF) for _ in range(2)]

    def norm(x, y):
        n = A.block_norm(x, y, y_norm=True)
        return n.x, n.h

    grads(norm, go, x, y)
    wt = torch.rand(T, 2, generator=g, device=_dev()) + 0.1
    grads(lambda x, wt, w1, w2: [A.experts(x, idx, wt, w1, w2)], go[:1], x, wt, w1, w2)

    def there_and_back(x, wt):
        recv, h = A.dispatch(x, idx, wt.detach(), E, 1)
        return [A.combine(recv, h, wt)]

    grads(there_and_back, go[:1], x, wt)
    grads(lambda x: [A.dispatch(x, idx, wt, E, 1)[0]], [_randn(g, 2 * T, H).to(BF)], x)


def test_tensors_of_the_caller_that_are_written_count_as_changed(ep):
    """A stream updated in place and a product's reused buffer, while a backward pass still needs what they held."""
    import combine_get_dispatch_scan_amd.autograd as A
    g = _gen(6)
    x, y = _randn(g, 8, 256).to(BF), _randn(g, 8, 256).to(BF)
    w = _randn(g, 256).requires_grad_()
    q = ep.quantize_weights_fp4(_randn(g, 1, 256, 256))
    x8, xs, off = _randn(g, 8, 256).to(torch.float8_e4m3fn), torch.ones(8, 2, device=_dev()), torch.tensor([0, 8], dtype=torch.int32, device=_dev())

    def in_place():
        ep.block_norm(x, y, x_out=x)

    def reused():
        ep.grouped_gemm_fp4(x8, xs, q.codes, q.scales, off, out=y)

    for change in (in_place, reused):
        n = A.block_norm(x, y, weight=w)
        change()
        with pytest.raises(RuntimeError, match="inplace"):
            n.h.sum().backward()
        n = A.block_norm(x, y, weight=w)
        before = x._version, y._version
        ep.block_norm(x, y)
        ep.grouped_gemm_fp4(x8, xs, q.codes, q.scales, off)
        assert before == (x._version, y._version)
        n.h.sum().backward()
    with torch.inference_mode():          # such tensors have no counter
        a = x.clone()
        want = ep.block_norm(x, y)
        n = ep.block_norm(a, y, x_out=a)
        assert n.x is a and torch.equal(a, want.x)
        out = torch.empty(8, 256, dtype=BF, device=_dev())
        assert ep.grouped_gemm_fp4(x8, xs, q.codes, q.scales, off, out=out) is out


# widths of the workgroup forms: one vector a lane, two, factors read again and sums in LDS, four vectors
@pytest.mark.parametrize("H", [1032, 2048, 2056, 7168, 8200, 16384, 16392])
@pytest.mark.parametrize("gate", ["token", "channel"])
@pytest.mark.parametrize("xt", [BF, F32])
def test_block_norm_of_many_rows_a_workgroup(ep, H, gate, xt):
    """256 to 768 workgroups share 1700 rows, so each takes several and some one more than others: rows fetched ahead, the
    slots that reductions use in turn, and the sums over a workgroup's rows; and up to twelve sums a share afterwards (256
    workgroups with seven rows, or 768 with three: fewer roundings in all than the tolerance's depth counts)."""
    o = _norm_case(H + 7, 1700, H, xt, F32 if gate == "token" else BF, gate=gate, gt=F32 if gate == "token" else BF)
    _check_norm(ep, o, quantize=H % 128 == 0)
    _check_norm_backward(ep, o, H)


@pytest.mark.parametrize("H", [2048, 7168, 8320, 16512])
def test_block_norm_alone_of_many_rows(ep, H):
    for xt in (BF, F32):
        o = _norm_case(H, 1300, H, xt, F32, y=False)
        _check_norm(ep, o, quantize=True)
        _check_norm_backward(ep, o, H)
    o = _norm_case(H, 1300, H, y_norm=False, y_weight=False, gate="none")     # a plain residual addition
    _check_norm(ep, o)
    _check_norm_backward(ep, o, H)
    o = _norm_case(H, 1300, H, weight=False, gate="channel", gt=F32)          # and no norm behind it
    _check_norm(ep, o, norm=False)
    _check_norm_backward(ep, o, H, norm=False)
