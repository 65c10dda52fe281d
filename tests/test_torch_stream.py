"""The binding's torch stream of a raw handle (no GPU needed: torch's streams are stood in for)."""
import pytest
import torch

from selective_state_space_03_amd import binding


@pytest.mark.parametrize("handle,want", [(None, "default"), (0, "default"), (0x1000, 0x1000)])
def test_a_null_handle_is_the_default_stream(handle, want, monkeypatch):
    def external(ptr, device=None):
        assert ptr, "torch answers a null handle with a stream of its pool"
        return ptr

    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    assert binding._torch_stream(handle, torch.device("cuda", 0)) == want
