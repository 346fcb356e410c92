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
