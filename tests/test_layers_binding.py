"""The token-sum layers' binding: what it refuses of a stream, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_layers_abi import On  # noqa: E402


class Stream:
    cuda_stream = 0x1234

    def __init__(self, device):
        self.device_index = device


@pytest.fixture
def gb(monkeypatch):
    """The binding over a library that takes every call and notes its stream."""
    import gradient_all_reduce_amd as lib

    class Library:
        streams = []

        def __getattr__(self, name):
            return lambda *args: self.streams.append(args[-1]) or 0

    monkeypatch.setattr(lib, "_lib", Library())
    monkeypatch.setattr(lib, "_current_device", lambda: 0)
    return lib


def test_a_stream_of_another_device_is_refused(gb):
    """Its kernels would run there, on memory of the tensors' device."""
    x, v, ids = On(torch, (4, 8), torch.float32), On(torch, (8,), torch.float32), On(torch, (4,), torch.int64)
    rows = On(torch, (4,), torch.float32)
    calls = [lambda s: gb.gb_layer_norm_forward(x, x, stream=s),
             lambda s: gb.gb_layer_norm_backward(x, v, v, x, x, rows, rows, stream=s),
             lambda s: gb.gb_embedding_forward(x, x, ids, stream=s),
             lambda s: gb.gb_embedding_backward(x, x, ids, stream=s)]
    for n, call in enumerate(calls):
        with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
            call(Stream(1))
        assert len(gb._lib.streams) == n
        call(Stream(0))
        assert gb._lib.streams[-1] == 0x1234
