"""The Python names of the training and 8-bit operators refuse a stream of another device than the tensors' (no GPU needed:
the refusal comes before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")

from mixture_experts_layer_token_amd import api  # noqa: E402


class Stream:
    cuda_stream = 0

    def __init__(self, device_index):
        self.device_index = device_index


class OnDevice:
    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_launch_on_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []

    def f(*args):
        calls.append(args)
        return 0

    with pytest.raises(ValueError):
        api._launch(f, (1, 2), (OnDevice(0), None, OnDevice(0)), Stream(1))
    with pytest.raises(ValueError):
        api._launch(f, (1, 2), (OnDevice(0), OnDevice(1)), Stream(0))
    assert not calls
    api._launch(f, (1, 2), (OnDevice(0), None, OnDevice(0)), Stream(0))
    assert calls == [(1, 2, 0)]


def test_no_workspace_is_made_for_a_stream_of_another_device():
    with pytest.raises(ValueError):
        api._grouped_ws(None, 0, None, torch.device("cuda", 0), Stream(1))


def test_torch_streams_name_their_device_so():
    assert hasattr(torch.cuda.Stream, "device_index")
