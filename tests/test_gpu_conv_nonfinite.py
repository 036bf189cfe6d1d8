"""Infinities and NaN in live tokens of the causal convolution: each reaches the tokens whose window holds it, as the
formula has it (a sum of -inf gives -inf / (1 + inf) = NaN), and nothing else; the state keeps the raw inputs."""
import numpy as np
import pytest

from oracle import layer as O
from tests.gpu_common import host
from tests.test_gpu_layer_ops import E, H, _conv_case, _np, _run_conv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _same_kind(got, ref):
    """Where the formula is not finite: the same infinity, or NaN."""
    bad = ~np.isfinite(ref)
    np.testing.assert_array_equal(got[bad], ref[bad])
    assert np.isfinite(got[~bad]).all()
    return ~bad


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("padded", [False, True])
def test_values_that_are_not_finite(torch_cuda, W, padded):
    torch = torch_cuda
    import int8_quant_b200 as iq
    inf, nan = float("inf"), float("nan")
    lengths = [70, 66, 9] if padded else None
    c = _conv_case(torch, W, 3, 70, 4, 16, 2, 16, W, True, True, lengths)
    # the first and last tokens, both ends of a tile of 64, two infinities in one window, every output part
    for b, t, ch, v in [(0, 0, 0, inf), (0, 69, 1, -inf), (0, 63, 2, nan), (0, 64, 3, inf), (0, 30, 64, inf),
                        (0, 31, 64, -inf), (1, 5, 70, -inf), (1, 65, 100, nan), (1, 20, 127, inf), (2, 8, 127, nan),
                        (2, 3, 96, -inf)]:
        c["xbc"][b, t, ch] = v
    for b, t, h, v in [(0, 0, 0, inf), (0, 7, 1, -inf), (1, 9, 2, nan), (2, 8, 3, -inf)]:
        c["dt_raw"][b, t, h] = v
    c["init"][0, 0, 5], c["init"][1, -1, 6] = nan, -inf
    _run_conv(c)
    with np.errstate(invalid="ignore"):
        ref = O.conv(_np(torch, c["xbc"]), _np(torch, c["weight"]), _np(torch, c["bias"]), _np(torch, c["init"]),
                     lengths, _np(torch, c["dt_raw"]), _np(torch, c["dt_bias"]))
    got = np.concatenate([_np(torch, c[k]).reshape(3, 70, -1) for k in ("x", "B", "C")], axis=2)
    ok = _same_kind(got, ref["out"])
    lim = (H * (1 + 2.0 ** -10) + 2 * (5 + 1.2 * np.abs(ref["u"])) * E) * np.abs(ref["out"]) + 1.2 * 5 * E * ref["mag"]
    assert (np.abs(got[ok] - ref["out"][ok]) <= lim[ok]).all()
    dt = _np(torch, c["dt"])
    ok = _same_kind(dt, ref["dt"])
    live = np.isfinite(ref["v"]) & ok
    assert (np.abs(dt[live] - ref["dt"][live]) <= ref["dt"][live] * (12 + np.abs(ref["v"][live])) * E).all()
    assert not dt[ok & ~live].any()                       # softplus of -inf, and padding
    np.testing.assert_array_equal(_np(torch, c["final"]), ref["state"])

    # the one-token form over the first row's tokens: the same bits
    state = c["init"][:1].clone()
    bits = lambda t: host(t.contiguous().view(torch.int16 if t.dtype is torch.bfloat16 else torch.int32))  # noqa: E731
    for t in range(70):
        o = {k: torch.empty_like(c[k][:1, t]) for k in ("x", "B", "C", "dt")}
        iq.ssd_conv_step_bf16(c["xbc"][:1, t], c["dt_raw"][:1, t], c["weight"], c["bias"], c["dt_bias"], state, o["x"],
                              o["dt"], o["B"], o["C"])
        for k in o:
            a, b = o[k], c[k][:1, t]
            assert (torch.isnan(a) == torch.isnan(b)).all() and (bits(a.nan_to_num(7.0)) == bits(b.nan_to_num(7.0))).all()
    np.testing.assert_array_equal(_np(torch, state), ref["state"][:1])
