"""The layer's operators run together: SsdLayer (prompts) and its decoder (single tokens).

* Against the layer's definition in float64 (weights as their codes' values, activations unquantised): the two
  quantisations of activations are off by a uniform error of a step of max / 127, relatively max / (127 sqrt(12) rms),
  1.1% for rows whose largest value is 5 times their root mean square; each is carried by a linear map, the first also
  through the scan and the norm behind it (taken as twice itself).  With the scan's own 5e-3 (bf16) or 5e-2 (W8A8 y)
  and a handful of bf16 roundings (2^-9 root mean square each): 4e-2 and 9e-2.
* Prompt against single tokens (bf16 scan): in_proj's rows, and so the convolution's state, are the same bits, as every
  operator ahead of the scan forms a token's values in one way; y differs by the two scans' 5e-3 each, and a code by at
  most a step where it does: 1e-2 + 2 * 1.1e-2.
* Rows of a padded batch, a prompt split on a chunk boundary, calls that overlap their predecessors' ends, graphs: the
  same bits.
"""
import numpy as np
import pytest

from oracle import layer as O
from oracle import ssd_fp64 as F
from oracle.ssd_fp64 import rel_l2
from tests.gpu_common import bf16_to_np, host

pytestmark = pytest.mark.gpu

H, P, G, N, D, W = 4, 64, 2, 128, 256, 4


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _layer(torch, path, seed=0, corr=True):
    from int8_quant_b200.runner import SsdLayer
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    hp, ch = H * P, H * P + 2 * G * N
    E = (hp + ch + H + 7) // 8 * 8
    w = {"norm": 1 + 0.1 * rn(D), "gate_norm": 1 + 0.1 * rn(hp), "conv_w": 0.5 * rn(W, ch), "conv_b": 0.1 * rn(ch),
         "A": -torch.exp(rn(H)), "D": rn(H), "dt_bias": -3 + rn(H)}
    for k, (n, m) in {"in": (E, D), "out": (D, hp)}.items():
        v = rn(n, m) / m ** 0.5
        s = v.abs().amax(1) / 127
        w[k + "_q"], w[k + "_s"] = torch.round(v / s[:, None]).to(torch.int8), s.contiguous()
    if corr:
        w["out_corr"] = 0.01 * rn(D)
    scales = None
    if path == "w8a8":
        one = lambda n, v: torch.full((n,), v, device="cuda")  # noqa: E731
        scales = {"s_B": one(G, 5 / 127), "s_C": one(G, 5 / 127), "s_x": one(hp, 1.5 / 127), "s_s": one(hp, 12 / 127)}
    return SsdLayer(w, (H, P, G, N), path, 64, scales)


def _hidden(torch, seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _definition(layer, hidden, residual):
    w = {k: host(v).astype(np.float64) for k, v in layer.w.items()}
    b, L, _ = hidden.shape
    T, hp, ch = b * L, H * P, H * P + 2 * G * N
    v = hidden.reshape(T, D) + (0 if residual is None else residual.reshape(T, D))
    u = O.norm_codes(v, w["norm"])["u"]
    rows = u @ (w["in_q"] * w["in_s"][:, None]).T
    c = O.conv(rows[:, hp:hp + ch].reshape(b, L, ch), w["conv_w"], w["conv_b"], None, None,
               rows[:, hp + ch:hp + ch + H].reshape(b, L, H), w["dt_bias"])
    x = c["out"][..., :hp].reshape(b, L, H, P)
    B, C = (c["out"][..., lo:lo + G * N].reshape(b, L, G, N) for lo in (hp, hp + G * N))
    y, fin = F.ssd_sequential(x, c["dt"], w["A"], B, C, w["D"])
    ug = O.norm_codes(O.gate(y.reshape(T, hp), rows[:, :hp]), w["gate_norm"])["u"]
    out = ug @ (w["out_q"] * w["out_s"][:, None]).T + w.get("out_corr", 0.0)
    return out.reshape(b, L, D), v.reshape(b, L, D), fin


@pytest.mark.parametrize("path,tol", [("bf16", 4e-2), ("w8a8", 9e-2)])
@pytest.mark.parametrize("L", [1, 130])
@pytest.mark.parametrize("residual", ["fp32", "none"])
def test_prefill_against_the_definition(torch_cuda, path, tol, L, residual):
    torch = torch_cuda
    layer = _layer(torch, path)
    hidden = _hidden(torch, L, 2, L, D)
    res = None if residual == "none" else _hidden(torch, 9, 2, L, D).float() * 2
    out, kept, state = layer.prefill(hidden, res)
    ref, v, fin = _definition(layer, bf16_to_np(hidden), None if res is None else host(res).astype(np.float64))
    np.testing.assert_array_equal(host(kept), v.astype(np.float32))
    assert rel_l2(bf16_to_np(out), ref) <= tol, rel_l2(bf16_to_np(out), ref)
    if path == "bf16":
        assert rel_l2(host(state["ssd"]), fin) <= tol
    import int8_quant_b200 as iq
    assert iq.ssd_workspace_status(layer.status) == 0


def test_steps_follow_a_prompt(torch_cuda):
    torch = torch_cuda
    layer = _layer(torch, "bf16")
    hidden = _hidden(torch, 3, 3, 70, D)
    out, kept, state = layer.prefill(hidden)
    _, _, st = layer.prefill(hidden[:, :60].contiguous())
    dec = layer.decoder(st)
    got = []
    for t in range(60, 70):
        o, r = dec.step(hidden[:, t].contiguous())
        got.append(o.clone())
        assert torch.equal(r, kept[:, t])
    assert torch.equal(st["conv"], state["conv"])
    assert rel_l2(bf16_to_np(torch.stack(got, 1)), bf16_to_np(out[:, 60:])) <= 3.2e-2
    assert rel_l2(host(st["ssd"]), host(state["ssd"])) <= 1e-2


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_prompts_without_tokens_leave_the_state(torch_cuda, path):
    """No tokens at all, and a padded batch of rows that are all padding."""
    torch = torch_cuda
    layer = _layer(torch, path)
    start = {"conv": _hidden(torch, 6, 2, W - 1, H * P + 2 * G * N), "ssd": layer.zero_state(2)["ssd"].random_(-100, 100)}
    for state in (None, start):
        want = layer.zero_state(2) if state is None else start
        out, kept, got = layer.prefill(_hidden(torch, 1, 2, 0, D), None, state)
        assert out.shape == kept.shape == (2, 0, D) and kept.dtype == torch.float32
        assert all(torch.equal(got[k], want[k]) for k in want)
        _, _, got = layer.prefill(_hidden(torch, 1, 2, 9, D), None, state,
                                  torch.zeros(2, dtype=torch.int32, device="cuda"))
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_padded_batch_equals_its_rows(torch_cuda, path):
    torch = torch_cuda
    layer = _layer(torch, path)
    lens = [70, 1, 64, 33]
    hidden = _hidden(torch, 5, 4, 70, D)
    for r, n in enumerate(lens):
        hidden[r, n:] = float("nan")
    start = {"conv": _hidden(torch, 6, 4, W - 1, H * P + 2 * G * N), "ssd": layer.zero_state(4)["ssd"]}
    if path == "bf16":
        start["ssd"].normal_()
    else:
        start["ssd"].random_(-100, 100)
    out, kept, state = layer.prefill(hidden, None, start, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for r, n in enumerate(lens):
        o, k, s = layer.prefill(hidden[r:r + 1, :n].contiguous(), None, {q: v[r:r + 1].contiguous() for q, v in start.items()})
        assert torch.equal(out[r, :n], o[0]) and torch.equal(kept[r, :n], k[0])
        assert torch.equal(state["conv"][r], s["conv"][0]) and torch.equal(state["ssd"][r], s["ssd"][0])


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_prompt_split_on_a_chunk_boundary(torch_cuda, path):
    torch = torch_cuda
    layer = _layer(torch, path)
    hidden = _hidden(torch, 7, 2, 150, D)
    out, kept, state = layer.prefill(hidden)
    a, _, st = layer.prefill(hidden[:, :64].contiguous())
    z, _, st = layer.prefill(hidden[:, 64:].contiguous(), None, st)
    assert torch.equal(torch.cat([a, z], 1), out)
    assert torch.equal(st["conv"], state["conv"]) and torch.equal(st["ssd"], state["ssd"])


@pytest.mark.parametrize("path", ["bf16", "w8a8"])
def test_steps_without_a_wait_between_and_in_graphs(torch_cuda, path):
    """Every kernel of the chain reads what the one ahead of it wrote.  The device waited for after each token, not at
    all, and two decoders' graphs on two streams at a time: the same bits."""
    torch = torch_cuda
    layer = _layer(torch, path)
    tokens = [_hidden(torch, 100 + t, 5, D) for t in range(24)]
    _, _, st0 = layer.prefill(_hidden(torch, 1, 5, 65, D))
    copy = lambda st: {k: v.clone() for k, v in st.items()}  # noqa: E731

    def run(wait):
        st, outs = copy(st0), []
        dec = layer.decoder(st)
        for h in tokens:
            o, r = dec.step(h)
            o2, r2 = dec.step(o.clone(), r.clone())     # a second layer's worth on the same state
            outs += [o2.clone(), r2.clone()]
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, st

    ref, st_ref = run(True)
    for _ in range(5):
        got, st = run(False)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        assert all(torch.equal(st[k], st_ref[k]) for k in st)

    graphs = []
    for _ in range(2):
        st, h = copy(st0), torch.empty_like(tokens[0])
        dec = layer.decoder(st)
        o, r = dec.step(h)                               # warm up, then the state again
        for k in st:
            st[k].copy_(st0[k])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, r = dec.step(h)
            mid_o, mid_r = o.clone(), r.clone()
            o, r = dec.step(mid_o, mid_r)
        for k in st:
            st[k].copy_(st0[k])
        graphs.append((g, st, h, o, r))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for t, token in enumerate(tokens):
        for (g, st, h, o, r), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                h.copy_(token)
                g.replay()
        torch.cuda.synchronize()
        for g, st, h, o, r in graphs:
            assert torch.equal(o, ref[2 * t]) and torch.equal(r, ref[2 * t + 1])
    for g, st, h, o, r in graphs:
        assert all(torch.equal(st[k], st_ref[k]) for k in st)


def test_prefill_on_a_side_stream_and_of_no_tokens(torch_cuda):
    torch = torch_cuda
    layer = _layer(torch, "w8a8", corr=False)
    hidden = _hidden(torch, 8, 2, 40, D)
    out, kept, state = layer.prefill(hidden)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o, k, s = layer.prefill(hidden, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(k, kept) and torch.equal(s["ssd"], state["ssd"])
    o, k, s = layer.prefill(hidden[:, :0], None, state)
    torch.cuda.synchronize()
    assert o.shape == (2, 0, D) and torch.equal(s["ssd"], state["ssd"]) and torch.equal(s["conv"], state["conv"])


def test_layer_refuses_unaligned_rows(torch_cuda):
    torch = torch_cuda
    from int8_quant_b200.runner import SsdLayer
    layer = _layer(torch, "bf16")
    w = dict(layer.w, in_q=layer.w["in_q"][:-4].contiguous(), in_s=layer.w["in_s"][:-4].contiguous())
    with pytest.raises(ValueError):
        SsdLayer(w, (H, P, G, N), "bf16")
