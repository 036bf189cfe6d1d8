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


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_check_raises_an_expired_wait(torch_cuda, monkeypatch, path):
    """The word that an expired wait leaves in the scan's workspace, or in the products' status, written here from the
    host's side after a call that succeeded."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    layer = _layer(torch, path)
    hidden = _hidden(torch, 8, 2, 40, D)
    name = "ssd_scan_fwd_bf16_from_state" if path == "bf16" else "ssd_scan_fwd_i8_from_state"
    scan, words = getattr(iq.ssd, name), []

    def call(*a):
        scan(*a)
        if words:
            a[-1].view(torch.int32)[:1].fill_(words.pop())

    monkeypatch.setattr(iq.ssd, name, call)
    layer.prefill(hidden)
    layer.check()
    words.append(5)
    ref = layer.prefill(hidden)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.use_deterministic_algorithms(True)
    try:
        got = layer.prefill(hidden, stream=side)
    finally:
        torch.use_deterministic_algorithms(False)
    with pytest.raises(iq.SsdError) as err:
        layer.check(side)
    assert err.value.status == 5 and _same(got, ref)
    layer.check()
    layer.status.fill_(5)
    with pytest.raises(iq.SsdError):
        layer.check()
    layer.check()
    layer.prefill(hidden[:0])                          # no rows: no scan, and no word of one
    layer.prefill(hidden[:, :0])
    layer.check()


def test_status_is_kept_by_a_captured_prompt(torch_cuda):
    torch = torch_cuda
    layer = _layer(torch, "w8a8")
    hidden = _hidden(torch, 8, 2, 40, D)
    ref = layer.prefill(hidden)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer.prefill(hidden)
    for _ in range(2):
        g.replay()
        layer.check()
        assert _same(got, ref)


@pytest.mark.parametrize("T,N", [(40, 700), (1, 8), (1500, 2048), (1500, 2053)])
def test_product_of_a_slice_of_tokens_and_channels(torch_cuda, T, N):
    """Tokens from the second on, channels from the fourth on, one of several status words: what the whole call gives."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = torch.Generator(device="cuda").manual_seed(N)
    q = torch.randint(-127, 128, (T + 1, 256), generator=g, device="cuda", dtype=torch.int8)
    Wq = torch.randint(-127, 128, (N + 3, 256), generator=g, device="cuda", dtype=torch.int8)
    s_t, s_w = torch.rand(T + 1, generator=g, device="cuda"), torch.rand(N + 3, generator=g, device="cuda")
    words = torch.zeros(6, dtype=torch.int32, device="cuda")
    whole, part = torch.empty(T + 1, N + 3, device="cuda").bfloat16(), torch.empty(T, N, device="cuda").bfloat16()
    iq.ssd_matmul_i8(q, s_t, Wq, s_w, None, whole, words[:1])
    iq.ssd_matmul_i8(q[1:], s_t[1:], Wq[3:], s_w[3:], None, part, words[5:])
    assert torch.equal(part, whole[1:, 3:])
    assert iq.ssd_workspace_status(words[5:]) == 0 and not words.any()


def test_residual_of_another_type_is_refused(torch_cuda):
    torch = torch_cuda
    import int8_quant_b200 as iq
    layer = _layer(torch, "bf16")
    hidden, res = _hidden(torch, 1, 2, 3, D), torch.zeros(2, 3, D, device="cuda", dtype=torch.float16)
    with pytest.raises(iq.SsdError, match="residual"):
        layer.prefill(hidden, res)
    with pytest.raises(iq.SsdError, match="residual"):
        layer.decoder(layer.zero_state(2)).step(hidden[:, 0].contiguous(), res[:, 0].contiguous())


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
@pytest.mark.parametrize("lo", [1, 39])
def test_prompts_that_are_slices_of_longer_ones(torch_cuda, path, lo):
    """Up to a single token of a longer batch, its residual too, from a state: the bits of dense copies."""
    torch = torch_cuda
    layer = _layer(torch, path)
    hidden, res = _hidden(torch, 2, 3, 40, D), _hidden(torch, 3, 3, 40, D).float()
    state = layer.prefill(_hidden(torch, 4, 3, 9, D))[2]
    ref = layer.prefill(hidden[:, lo:].contiguous(), res[:, lo:].contiguous(), state)
    assert _same(layer.prefill(hidden[:, lo:], res[:, lo:], state), ref)
