"""The binding's short ways into torch (the raw stream, the current device) are not part of torch's public
interface: on a torch without them the public ones answer.  CPU only."""
import pytest

PRIVATE = ["_cuda_getDevice", "_cuda_getCurrentRawStream"]


@pytest.mark.parametrize("missing", [PRIVATE[:1], PRIVATE[1:], PRIVATE], ids=str)
def test_public_calls_stand_in(missing, monkeypatch):
    import torch
    import int8_group_quantized_gb300 as dgq

    class Stream:
        cuda_stream = 0x500

    def raw(device):
        assert device == 3
        return 0x700
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    assert dgq._device() == 3
    assert dgq._stream(None) == (0x500 if PRIVATE[1] in missing else 0x700)
