"""SsdLayer on the GPU: streams, errors of device-side waits, residual types, single tokens of the W8A8 path, the mean
correction, states and weights that do not fit."""
import pytest

from tests.test_gpu_layer import D, _hidden, _layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _same(a, b):
    return all(x.equal(y) for x, y in zip(a[:2], b[:2])) and all(a[2][k].equal(b[2][k]) for k in b[2])


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_prefill_on_a_stream_that_is_not_the_current_one(torch_cuda, path):
    """A stream, its handle, the default stream's: the bits of a call on the current one, also where the current stream
    allocates and writes while the other one works."""
    torch = torch_cuda
    layer = _layer(torch, path)
    hidden = _hidden(torch, 8, 4, 300, D)
    ref = layer.prefill(hidden)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        got = layer.prefill(hidden, stream=stream)
        waste = [torch.full((1 << n,), 1.0, device="cuda") for n in range(8, 22)]
        torch.cuda.synchronize()
        assert _same(got, ref) and len(waste) == 14
