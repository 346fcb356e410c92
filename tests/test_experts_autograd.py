"""CPU checks of how the expert layer's binding and autograd functions hold their
tensors: the library's calls are replaced by stand-ins on CPU tensors, everything
around them is the code that runs on the GPU."""
import contextlib

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
