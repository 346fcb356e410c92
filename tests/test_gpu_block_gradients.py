"""GPU check of gradients through two whole blocks (norm, gate, experts, norm, ... with weights
that both share), close enough to see that a block's part is missing."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_block_layer import BF, _case, _gen, _randn, _unit  # noqa: E402

K, E, T, H, I = 2, 8, 48, 256, 128

# An E4M3 rounding is off by up to half a step of 2^-3 of the power of two below the value, evenly spread: 2^-3 / sqrt(12)
# of it in the mean square, where values spread evenly over the binade's logarithm are sqrt(3 / (2 ln 2)) of it.
E4M3 = 2.0 ** -3 / math.sqrt(12) / math.sqrt(3 / (2 * math.log(2)))
# A gradient of two blocks has at most twelve of them in its chain (rows, two weights, SwiGLU's input and output and the
# gradient's rows, a block), independent of each other, so they add up in the mean square.  Where two factors carry an
# error (SwiGLU and its gradient, products of weights and rows, the norms' factors) it is passed on twice, so each counts
# up to five times in the square: 12 * 5 <= 64 = 8^2.
BOUND = 8 * E4M3


@pytest.mark.parametrize("seed", [50, 60, 70])
def test_autograd_of_two_blocks_closely(ep, seed):
    import combine_get_dispatch_scan_amd.autograd as A
    c = _case(seed, T=T)
    g = _gen(seed + 1)
    c["router"] = _randn(g, H, E) * H ** -0.5
    go = _randn(g, T, H).to(BF)
    names = ("w1", "w2", "norm", "post", "gate", "router")
    leaves = {k: c[k].clone().requires_grad_() for k in ("x", *names)}
    ids = []
    s = A.block_norm(leaves["x"], weight=leaves["norm"])
    for _ in range(2):
        gt = A.gate(s.h.float() @ leaves["router"], K)
        ids.append(gt.topk_idx)
        y = A.experts(s.h, gt.topk_idx, gt.topk_weights, leaves["w1"], leaves["w2"])
        s = A.block_norm(s.x, y, weight=leaves["norm"], y_norm=True, y_weight=leaves["post"], gate=leaves["gate"])
    s.h.backward(go)

    # in 64 bits, with a copy of each shared weight for each place that uses it
    use = {k: [c[k].double().requires_grad_() for _ in range(3 if k == "norm" else 2)] for k in names}
    x0 = c["x"].double().requires_grad_()
    x, h = x0, _unit(x0) * use["norm"][0]
    for i in range(2):
        sel = torch.gather(torch.softmax(h @ use["router"][i], 1), 1, ids[i])
        wt = sel / sel.sum(1, keepdim=True)
        rows = []
        for t in range(T):
            acc = 0
            for k in range(K):
                e = int(ids[i][t, k])
                u = use["w1"][i][e] @ h[t]
                acc = acc + wt[t, k] * (use["w2"][i][e] @ (torch.nn.functional.silu(u[:I]) * u[I:]))
            rows.append(acc)
        x = x + use["gate"][i] * _unit(torch.stack(rows)) * use["post"][i]
        h = _unit(x) * use["norm"][i + 1]
    h.backward(go.double())

    def off(got, want):
        return float((got - want).norm() / want.norm())

    got = {k: v.grad.double() for k, v in leaves.items()}
    assert off(got["x"], x0.grad) < BOUND
    for k in names:
        want = sum(v.grad for v in use[k])
        assert off(got[k], want) < BOUND, (k, off(got[k], want))
        for i, v in enumerate(use[k]):        # and it would not be, were one place's part missing
            assert off(got[k] - v.grad, want) > BOUND, (k, i)
