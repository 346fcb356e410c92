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
