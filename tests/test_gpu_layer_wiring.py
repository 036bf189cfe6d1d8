"""SsdLayer's wiring on the GPU, where an argument that went astray would show: single tokens of the W8A8 path with a
decay shift of their own, residual streams in bf16, the output projection's correction, a layer of the 2.7B model's width.

Tolerances, relative norms.  Codes of step s are off by a uniform error of s / sqrt(12) root mean square, so a quantised
row u by s sqrt(n / 12) / |u|: e1 for in_proj's, e2 for out_proj's, computed from the definition's own rows (1% where the
largest value is 5 times the root mean square; gated rows of thousands of features have values of 20 times it, 4%).  e2 is
carried by a linear map.  e1 reaches the gated row four times, independently: through x, B and C, whose product y is, and
through z: sqrt(4) e1.  With the scan's own 5e-3 (bf16) or 5e-2 (W8A8) and four roundings to bf16 (rows, x | B | C, y,
output; 2^-9 each at most, root mean square): 2 e1 + e2 + scan + 4 * 2^-9.  Between a prompt and single tokens of 256
features: 1e-2 for the scans' y, 2 * 1.1e-2 for the codes behind it, as in test_gpu_layer.py.  A correction c is added
in fp32 before the one rounding to bf16, so outputs with and without it differ by c within half a step of each, 2^-8 of
their values (the fp32 roundings, 2^-23 of |output| + |c|, are in the 2% on top).
"""
import numpy as np
import pytest

from oracle import layer as O
from oracle import ssd_fp64 as F
from oracle import ssd_w8a8 as W
from oracle.ssd_fp64 import rel_l2
from tests.gpu_common import bf16_to_np, host

pytestmark = pytest.mark.gpu

SMALL = (4, 64, 2, 128, 256)               # heads, head size, groups, state size, features
WIDE = (80, 64, 1, 128, 2560)              # the 2.7B model's layer
TAPS, EPS = 4, 1e-5
SCAN = {"bf16": 5e-3, "w8a8": 5e-2}


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _layer(torch, path, dims=SMALL, corr=0.0, shift=7, seed=0):
    from int8_quant_b200.runner import SsdLayer
    H, P, G, N, d = dims
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    hp, ch = H * P, H * P + 2 * G * N
    E = (hp + ch + H + 7) // 8 * 8
    w = {"norm": 1 + 0.1 * rn(d), "gate_norm": 1 + 0.1 * rn(hp), "conv_w": 0.5 * rn(TAPS, ch), "conv_b": 0.1 * rn(ch),
         "A": -torch.exp(rn(H)), "D": rn(H), "dt_bias": -3 + rn(H)}
    for k, (n, m) in {"in": (E, d), "out": (d, hp)}.items():
        v = rn(n, m) / m ** 0.5
        s = v.abs().amax(1) / 127
        w[k + "_q"], w[k + "_s"] = torch.round(v / s[:, None]).to(torch.int8), s.contiguous()
    c = rn(d)
    if corr:
        w["out_corr"] = corr * c
    scales = None
    if path == "w8a8":
        # every channel and group a scale of its own
        one = lambda n, v: v * torch.linspace(0.8, 1.2, n, device="cuda")  # noqa: E731
        scales = {"s_B": one(G, 5 / 127), "s_C": one(G, 5.5 / 127), "s_x": one(hp, 1.5 / 127), "s_s": one(hp, 12 / 127)}
    return SsdLayer(w, (H, P, G, N), path, 64, scales, shift)


def _hidden(torch, seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _definition(layer, v):
    """The layer's output and final state, float64, of the residual stream v [b, L, d], and the tolerance on the output."""
    H, P, G, N, hp, ch = layer.H, layer.P, layer.G, layer.N, layer.hp, layer.ch
    w = {k: host(t).astype(np.float64) for k, t in layer.w.items()}
    b, L, d = v.shape
    n1 = O.norm_codes(v.reshape(-1, d), w["norm"])
    rows = n1["u"] @ (w["in_q"] * w["in_s"][:, None]).T
    c = O.conv(rows[:, hp:hp + ch].reshape(b, L, ch), w["conv_w"], w["conv_b"], None, None,
               rows[:, hp + ch:hp + ch + H].reshape(b, L, H), w["dt_bias"])
    x = c["out"][..., :hp].reshape(b, L, H, P)
    B, C = (c["out"][..., lo:lo + G * N].reshape(b, L, G, N) for lo in (hp, hp + G * N))
    y, fin = F.ssd_sequential(x, c["dt"], w["A"], B, C, w["D"])
    n2 = O.norm_codes(O.gate(y.reshape(-1, hp), rows[:, :hp]), w["gate_norm"])
    e1, e2 = (np.sqrt((n["scale"] ** 2).sum() * n["u"].shape[1] / 12 / (n["u"] ** 2).sum()) for n in (n1, n2))
    out = n2["u"] @ (w["out_q"] * w["out_s"][:, None]).T + w.get("out_corr", 0.0)
    return out.reshape(b, L, d), fin, 2 * e1 + e2 + SCAN[layer.path] + 4 * 2.0 ** -9


@pytest.mark.parametrize("shift,dims", [(7, SMALL), (6, SMALL), (9, SMALL), (7, WIDE)])
def test_w8a8_steps_follow_the_integer_oracle(torch_cuda, shift, dims):
    """The state's codes after each of the decoder's steps, from the x, dt, B and C that it formed."""
    torch = torch_cuda
    layer = _layer(torch, "w8a8", dims, shift=shift)
    _, _, state = layer.prefill(_hidden(torch, 3, 3, 64, dims[-1]))
    dec = layer.decoder(state)
    w, sc = {k: host(layer.w[k]) for k in ("A", "D")}, {k: host(v) for k, v in layer.scales.items()}
    ref = host(state["ssd"]).copy()
    assert np.abs(ref).max() > 20                         # the state is there to decay
    for t in range(6):
        dec.step(_hidden(torch, 50 + t, 3, dims[-1]))
        torch.cuda.synchronize()
        Bq, Cq = W.quantize_inputs(bf16_to_np(dec.B).astype(np.float32)[:, None],
                                   bf16_to_np(dec.C).astype(np.float32)[:, None], sc["s_B"], sc["s_C"])
        r = W.decode_step_i8(bf16_to_np(dec.x).astype(np.float32), host(dec.dt), w["A"], Bq[:, 0], Cq[:, 0], w["D"],
                             sc["s_B"], sc["s_C"], sc["s_x"], sc["s_s"], ref, k=shift)
        np.testing.assert_array_equal(host(state["ssd"]), r["state8"])
        assert rel_l2(bf16_to_np(dec.ssd.y), r["y"]) <= 1e-2
        ref = r["state8"]


@pytest.mark.parametrize("shift", [7, 5])
@pytest.mark.parametrize("residual", ["fp32", "bf16", "none"])
def test_w8a8_steps_equal_prompts_of_one_token(torch_cuda, shift, residual):
    """A prompt of one token that goes on from the state forms the same chunk: the state's codes, the convolution's state
    and the residual are the same bits."""
    torch = torch_cuda
    layer = _layer(torch, "w8a8", shift=shift, corr=1.0)
    _, _, state = layer.prefill(_hidden(torch, 3, 2, 64, 256))
    mine = {k: v.clone() for k, v in state.items()}
    dec = layer.decoder(mine)
    for t in range(5):
        h, res = _hidden(torch, 20 + t, 2, 1, 256), None
        if residual != "none":
            res = (_hidden(torch, 70 + t, 2, 1, 256) * 2).to(torch.float32 if residual == "fp32" else torch.bfloat16)
        out, kept, state = layer.prefill(h, res, state)
        o, r = dec.step(h[:, 0], None if res is None else res[:, 0])
        assert torch.equal(r, kept[:, 0]) and r.dtype == kept.dtype
        assert torch.equal(mine["ssd"], state["ssd"]) and torch.equal(mine["conv"], state["conv"])
        assert rel_l2(bf16_to_np(o), bf16_to_np(out[:, 0])) <= 3.2e-2


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
@pytest.mark.parametrize("L", [1, 70])
def test_bf16_residual_stream(torch_cuda, path, L):
    """The sum is stored rounded to bf16, and normalised as it is stored; prompt and step alike."""
    torch = torch_cuda
    layer = _layer(torch, path, corr=1.0)
    hidden, res = _hidden(torch, L, 2, L, 256), (_hidden(torch, 9, 2, L, 256) * 3)
    out, kept, state = layer.prefill(hidden, res)
    v = (hidden.float() + res.float()).bfloat16()
    assert kept.dtype is torch.bfloat16 and torch.equal(kept, v)
    ref, fin, tol = _definition(layer, bf16_to_np(v))
    assert rel_l2(bf16_to_np(out), ref) <= tol, rel_l2(bf16_to_np(out), ref)
    if path == "bf16":
        assert rel_l2(host(state["ssd"]), fin) <= tol
    if L == 1:
        o, r = layer.decoder(layer.zero_state(2)).step(hidden[:, 0], res[:, 0])
        assert torch.equal(r, v[:, 0])
        assert rel_l2(bf16_to_np(o), ref[:, 0]) <= tol
    layer.check()


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_correction_is_added_to_every_output(torch_cuda, path):
    torch = torch_cuda
    plain, corrected = _layer(torch, path), _layer(torch, path, corr=1.0)
    c = host(corrected.w["out_corr"]).astype(np.float64)
    hidden = _hidden(torch, 4, 2, 33, 256)

    def check(a, b):
        a, b = bf16_to_np(a), bf16_to_np(b)
        assert (np.abs(b - (a + c)) <= 1.02 * 2.0 ** -8 * (np.abs(a) + np.abs(b)) + 2.0 ** -20).all()

    assert np.abs(c).max() > 2
    a, b = plain.prefill(hidden), corrected.prefill(hidden)
    check(a[0], b[0])
    token = _hidden(torch, 5, 2, 256)
    check(plain.decoder(a[2]).step(token)[0], corrected.decoder(b[2]).step(token)[0])


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_a_wide_layer(torch_cuda, path):
    """80 heads, 2560 features: against the definition, in two parts and in single tokens."""
    torch = torch_cuda
    layer = _layer(torch, path, WIDE, corr=1.0)
    hidden = _hidden(torch, 6, 2, 70, 2560)
    out, kept, state = layer.prefill(hidden)
    ref, fin, tol = _definition(layer, bf16_to_np(hidden))
    assert rel_l2(bf16_to_np(out), ref) <= tol, (rel_l2(bf16_to_np(out), ref), tol)
    a, _, st = layer.prefill(hidden[:, :64])
    dec = layer.decoder({k: v.clone() for k, v in st.items()})
    steps = torch.stack([dec.step(hidden[:, t].contiguous())[0].clone() for t in range(64, 70)], 1)
    z, _, st = layer.prefill(hidden[:, 64:], None, st)
    assert torch.equal(torch.cat([a, z], 1), out)
    assert torch.equal(st["conv"], state["conv"]) and torch.equal(st["ssd"], state["ssd"])
    assert torch.equal(dec.state["conv"], state["conv"])
    if path == "bf16":                                    # (the integer state's steps: the integer oracle, above)
        assert rel_l2(bf16_to_np(steps), ref[:, 64:]) <= tol, (rel_l2(bf16_to_np(steps), ref[:, 64:]), tol)
    layer.check()
