"""SsdLayer's and its decoder's host side (no GPU): where their calls go, with the library's functions replaced by
recorders and torch's current device and stream by fakes."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from int8_quant_b200 import runner, ssd  # noqa: E402

H, P, G, N, D, W = 2, 16, 1, 16, 32, 4
HP, CH = H * P, H * P + 2 * G * N
CALLS = ("ssd_add_rmsnorm_i8", "ssd_matmul_i8", "ssd_conv_fwd_bf16", "ssd_conv_step_bf16", "ssd_gated_rmsnorm_i8",
         "ssd_quantize_inputs", "ssd_scan_fwd_bf16_from_state", "ssd_scan_fwd_i8_from_state", "ssd_decode_step_bf16",
         "ssd_decode_step_i8")


def make_weights():
    E = HP + CH + 8
    return {"norm": torch.ones(D), "gate_norm": torch.ones(HP), "in_q": torch.zeros(E, D, dtype=torch.int8),
            "in_s": torch.ones(E), "out_q": torch.zeros(D, HP, dtype=torch.int8), "out_s": torch.ones(D),
            "conv_w": torch.zeros(W, CH), "dt_bias": torch.zeros(H), "A": -torch.ones(H), "D": torch.ones(H)}


def make_scales():
    return {"s_B": torch.ones(G), "s_C": torch.ones(G), "s_x": torch.ones(HP), "s_s": torch.ones(HP)}


def make_layer(path):
    return runner.SsdLayer(make_weights(), (H, P, G, N), path, 64, make_scales() if path == "w8a8" else None)


class World:
    """A current device and stream, and the calls made under them."""

    def __init__(self, monkeypatch):
        self.device, self.stream, self.calls = 0, "device 0's", []

        @contextlib.contextmanager
        def device(index):
            was, self.device, self.stream = (self.device, self.stream), index, f"device {index}'s"
            yield
            self.device, self.stream = was

        @contextlib.contextmanager
        def stream(s):
            was, self.stream = self.stream, s.cuda_stream
            yield
            self.stream = was

        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        for name in CALLS:
            monkeypatch.setattr(ssd, name, lambda *a, _n=name, **k: self.calls.append((_n, self.device, self.stream)))


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
@pytest.mark.parametrize("current", [0, 1])
def test_every_call_runs_on_the_layers_device(world, path, current):
    """The scan and its step launch on the current device: a layer on another one makes its own the current one, and
    leaves the caller's as it was."""
    layer = make_layer(path)
    layer.index = 1
    world.device, world.stream = current, f"device {current}'s"
    layer.prefill(torch.zeros(1, 3, D, dtype=torch.bfloat16))
    assert len(world.calls) == (7 if path == "w8a8" else 6)
    layer.decoder(layer.zero_state(1)).step(torch.zeros(1, D, dtype=torch.bfloat16))
    assert {c[1:] for c in world.calls} == {(1, "device 1's")}
    assert (world.device, world.stream) == (current, f"device {current}'s")


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_a_prompts_buffers_belong_to_its_stream(world, path):
    """With a stream given, the calls and the allocations around them are that stream's: memory that a call gives back
    is used again in the order of the stream it was used on."""
    class Side:
        cuda_stream = "side"

    layer = make_layer(path)
    layer.index = 0
    made = []
    new = layer.new
    layer.new = lambda *a, **k: made.append(world.stream) or new(*a, **k)
    layer.prefill(torch.zeros(1, 3, D, dtype=torch.bfloat16), stream=Side())
    assert set(made) == {"side"} and {c[2] for c in world.calls} == {"side"}
    assert world.stream == "device 0's"


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_an_expired_wait_of_the_scan_outlives_its_workspace(world, monkeypatch, path):
    """The scan's error word lies in a workspace that ends with the call: check() raises it, also after later calls
    without an error, and then is clear again."""
    layer = make_layer(path)
    words = iter([0, 5, 0])
    scan = "ssd_scan_fwd_bf16_from_state" if path == "bf16" else "ssd_scan_fwd_i8_from_state"
    monkeypatch.setattr(ssd, scan, lambda *a: a[-1].view(torch.int32)[:1].fill_(next(words)))

    def status(word, stream=None):
        bad = int(word)
        word.zero_()
        return bad

    monkeypatch.setattr(ssd, "ssd_workspace_status", status)
    hidden = torch.zeros(1, 3, D, dtype=torch.bfloat16)
    layer.prefill(hidden)
    layer.check()
    layer.prefill(hidden)
    layer.prefill(hidden)
    with pytest.raises(ssd.SsdError) as err:
        layer.check()
    assert err.value.status == 5
    layer.check()


def _wrong_states(path, b):
    good, other = (torch.float32, torch.int8) if path == "bf16" else (torch.int8, torch.float32)
    z = lambda *s, t=good: torch.zeros(s, dtype=t)  # noqa: E731
    return [z(b, H, P, N, t=other), z(b, H, P, N, t=torch.bfloat16), z(b - 1, H, P, N), z(b, H, P, N - 1),
            z(b, H, P * N), z(b, H, N, P).transpose(2, 3), torch.zeros(b, H, P, N, dtype=good, device="meta")]


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_states_that_the_scan_would_read_past_are_refused(world, path):
    """Another path's state, another batch's, one of other strides or elsewhere: nothing is launched."""
    layer = make_layer(path)
    hidden = torch.zeros(3, 2, D, dtype=torch.bfloat16)
    for wrong in _wrong_states(path, 3):
        state = {**layer.zero_state(3), "ssd": wrong}
        with pytest.raises(ssd.SsdError) as err:
            layer.prefill(hidden, None, state)
        assert err.value.status == 1 and 'state["ssd"]' in str(err.value)
        with pytest.raises(ssd.SsdError):
            layer.decoder(state)
    assert not world.calls
    layer.prefill(hidden, None, layer.zero_state(3))
    layer.decoder(layer.zero_state(3))


@pytest.mark.parametrize("name,wrong", [("A", torch.ones(H, dtype=torch.float64)), ("A", torch.ones(H - 1)),
                                        ("D", torch.ones(2 * H)[::2]), ("s_B", torch.ones(G + 1)),
                                        ("s_C", torch.ones(G, dtype=torch.bfloat16)), ("s_x", torch.ones(H)),
                                        ("s_s", torch.ones(H, P))])
def test_scan_parameters_of_other_sizes_are_refused(name, wrong):
    w, scales = make_weights(), make_scales()
    (w if name in w else scales)[name] = wrong
    with pytest.raises(ValueError, match=name):
        runner.SsdLayer(w, (H, P, G, N), "w8a8", 64, scales)


def test_a_residual_of_another_type_reaches_the_calls_own_check(world, monkeypatch):
    """... which refuses it with its reason, from the prompt and from the step."""
    layer, seen = make_layer("bf16"), []
    layer.index = 0
    monkeypatch.setattr(ssd, "ssd_add_rmsnorm_i8", lambda x, res, *a, **k: seen.append(res.dtype))
    res = torch.zeros(2, D, dtype=torch.float16)
    layer.prefill(torch.zeros(2, 1, D, dtype=torch.bfloat16), res[:, None])
    layer.decoder(layer.zero_state(2)).step(torch.zeros(2, D, dtype=torch.bfloat16), res)
    assert seen == [torch.float16] * 2


@pytest.mark.parametrize("lo,hi", [(0, 5), (2, 4), (4, 5), (0, 1), (5, 5)])
def test_prompts_that_are_slices_arrive_dense(world, monkeypatch, lo, hi):
    layer, seen = make_layer("bf16"), []
    layer.index = 0
    monkeypatch.setattr(ssd, "ssd_add_rmsnorm_i8", lambda x, res, *a, **k: seen.extend((x, res)))
    hidden = torch.randn(3, 5, 2 * D).bfloat16()[..., D:]
    res = torch.randn(3, 5, D)
    layer.prefill(hidden[:, lo:hi], res[:, lo:hi])
    assert all(t.is_contiguous() for t in seen)
    assert torch.equal(seen[0], hidden[:, lo:hi].reshape(-1, D)) and torch.equal(seen[1], res[:, lo:hi].reshape(-1, D))
