"""A call runs on the current device: tensors of another one are refused on the host."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda


class On:
    """What the checks ask of a tensor, of one that is on another GPU than there may be."""

    is_cuda = True

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.meta, self.device = torch.empty(*shape, dtype=dtype, device="meta"), device

    def __getattr__(self, name):
        return getattr(self.meta, name)

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 4096


def test_tensors_of_another_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    calls = (lambda device: kda._checked_arg(On(device, 4, 8), torch.bfloat16, 32, "x", "[4, 8]"),
             lambda device: kda._gdn_rows(kda.dims(1), On(device, 4, 384), 4),
             lambda device: kda._space(On(device, 4096, dtype=torch.uint8))[0],
             lambda device: kda._probs(On(device, 2, 3, 100), torch.bfloat16, "p", 2, 3)[0],
             lambda device: kda._pages(On(device, 2, 3, 1, 128)).base)
    for call in calls:
        assert call(0) == 4096
        with pytest.raises(ValueError, match="current device, cuda:0 .got cuda:1"):
            call(1)


def test_native_place():
    kda.load()
    assert all(kda._place(t) is None for t in (torch.zeros(3), On(0, 3), torch.empty(3, device="meta"), None, 7))


@pytest.mark.gpu
def test_native_place_on_the_device():
    kda.load()
    x = torch.zeros(6, 8, device="cuda")
    assert kda._place(x) == x.data_ptr() and kda._place(x.t()[2:]) == x.t()[2:].data_ptr() == kda._here(x.t()[2:])


def test_logits_of_another_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    kda.load()
    with pytest.raises(ValueError, match="current device"):
        kda.kda_token_logprobs(On(1, 4, 100, dtype=torch.float32), torch.zeros(4, dtype=torch.int32), torch.zeros(4))
