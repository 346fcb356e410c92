"""CPU checks of the binding around the expert layer: what torch lacks, workspaces of every
width, gradients at any offset."""
import pytest

import combine_get_dispatch_scan_amd as ep

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("missing", [("float4_e2m1fn_x2",), ("float8_e8m0fnu",), ("float4_e2m1fn_x2", "float8_e8m0fnu")])
def test_types_that_torch_lacks_concern_their_own_calls_only(monkeypatch, missing):
    monkeypatch.setattr(ep, "_KINDS", {})
    for name in missing:
        monkeypatch.delattr(torch, name)
    kinds = ep._kinds()
    assert kinds["bf16"] == (torch.bfloat16,) and kinds["fp8"] == (torch.float8_e4m3fn, torch.uint8)
    assert kinds["f32"] == (torch.float32,) and kinds["i64"] == (torch.int64,) and kinds["i32"] == (torch.int32,)
    assert kinds["u8"] == (torch.uint8,) and torch.uint8 in kinds["fp4"] and torch.uint8 in kinds["e8m0"]


def test_types_of_this_torch():
    assert ep._kinds()["fp4"] == (torch.uint8, torch.float4_e2m1fn_x2)
    assert ep._kinds()["e8m0"] == (torch.float8_e8m0fnu, torch.uint8)


def test_gradients_at_odd_offsets(monkeypatch):
    """Outputs joined with something of an odd length hand back gradients that are dense and begin anywhere."""
    import contextlib
    import combine_get_dispatch_scan_amd.autograd as A
    got = []

    def backward(x, y=None, *, grad_x, grad_h, need, **o):
        got.append([None if t is None else (t.is_contiguous() and t.data_ptr() % 16 == 0, t.clone()) for t in (grad_x, grad_h)])
        return ep.BlockNormGrads(x=torch.zeros_like(x), y=torch.zeros_like(y))

    monkeypatch.setattr(A, "_on", lambda *t: contextlib.nullcontext())
    monkeypatch.setattr(A, "_eager_only", lambda what: None)
    monkeypatch.setattr(A, "_block_norm_call", lambda x, y, **o: ep.BlockNorm(x + y, (x + y).bfloat16()))
    monkeypatch.setattr(A, "_block_norm_backward", backward)
    x, y = (torch.randn(4, 16).bfloat16().requires_grad_() for _ in range(2))
    for first in (1, 3, 8):
        n = A.block_norm(x, y)
        g = torch.randn(first + 128).bfloat16()
        torch.cat([torch.ones(first).bfloat16(), n.x.flatten(), n.h.flatten()]).backward(g)
        (x_fits, gx), (h_fits, gh) = got.pop()
        assert x_fits and h_fits
        assert torch.equal(gx.flatten(), g[first:first + 64]) and torch.equal(gh.flatten(), g[first + 64:])


@pytest.mark.parametrize("width,most", [(8, 512), (512, 512), (1024, 512), (1032, 768), (2048, 768), (2056, 512), (4096, 512),
                                        (4104, 256), (7168, 256), (16384, 256), (16392, 256), (32768, 256)])
def test_norm_workspace_of_every_team(width, most):
    """Two sums of a row for each workgroup: at most three a CU (of 256) with one vector a lane, two with up to 256 threads,
    else one; at least one where there are no rows."""
    for rows in (0, 1, 5, 300, 1500, 1 << 20, 0x7FFFFF00):
        teams = -(-rows // 4) if width <= 1024 else rows
        want = max(1, min(teams, most)) * 2 * width * 4
        assert ep.ep_block_norm_workspace_bytes(rows, width) == -(-want // 256) * 256
