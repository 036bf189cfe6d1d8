"""GPU parity of the layer operators around the scan: norms with INT8 codes, the INT8 product,
the causal convolution and its one-token step, against the float64 oracle.

Tolerances, by the arithmetic of the kernels (e = 2^-24, half a step of fp32; h = 2^-8, half a
step of bf16; documented bounds: ex2.approx 2^-22 relative, rcp.approx 1 ulp, rsqrtf 2 ulp, expf
and log1pf 2 ulp, an ulp at most 2 e relative).  SiLU of u, u / (1 + exp(-u)): the exponent's
two roundings move the exponential by at most 2|u| e, ex2 4 e, the addition e, the reciprocal
2 e, the product e: within 2 (5 + 1.2|u|) e.

* residual_out: one fp32 addition, so bit for bit; in bf16 one more rounding.
* a norm's v after the gate: one more product, GATE(z) = (2 (5 + 1.2|z|) + 1) e.
* codes: p = v w, 127 / top, their product (and top itself): 4 e relative on a position of at
  most 127, and twice the gate's, so |code - pos| <= 1/2 + 127 (4 e + 2 GATE).
* scale: top (e + GATE), the sum of squares (at most 64 additions in a row and 12 in the
  tree, halved by the root, and 2 GATE / 2), rsqrtf 4 e, three products: (48 + 2 GATE / e) e.
* product: the sums are exact; fp32(sum), s_t s_w, their product and the bias's addition, 4 e of
  |product| + |bias|, then bf16.
* convolution: 5 fused steps on Σ|w s| + |bias| (5 e), SiLU's slope at most 1.1, its value's
  error 2 (5 + 1.2|u|) e relative, then bf16.
* dt: one addition (e |v|, and |d dt/dv| <= dt), expf and log1pf: dt (12 + |v|) e.
"""
import numpy as np
import pytest

from oracle import layer as O
from tests.gpu_common import bf16_to_np, host

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
H = 2.0 ** -8


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(torch, g, *shape, scale=1.0, dtype=None):
    t = torch.randn(*shape, generator=g, device="cuda") * scale
    return t if dtype is None else t.to(dtype)


def _np(torch, t):
    if t is None:
        return None
    return bf16_to_np(t) if t.dtype is torch.bfloat16 else host(t).astype(np.float64)


# ---------------------------------------------------------------- norms

def _check_codes(q, scale, v, weight, eps, gate_err=0.0):
    ref = O.norm_codes(v, weight, eps)
    off = np.abs(q.astype(np.float64) - ref["pos"])
    assert off.max(initial=0) <= 0.5 + 127 * (4 * E + 2 * gate_err), off.max()
    rel = np.abs(scale - ref["scale"]) / ref["scale"]
    assert rel.max(initial=0) <= 48 * E + 2 * gate_err, rel.max()


NORM_SIZES = [(1, 16), (3, 48), (1, 8192), (130, 2560), (5, 8208), (2, 16400), (2, 32768), (1025, 2048), (3001, 512)]


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("residual", ["fp32", "bf16", "none"])
@pytest.mark.parametrize("weighted,in_place", [(True, False), (False, True)])
def test_add_rmsnorm(torch_cuda, T, d, residual, weighted, in_place):
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, T * 7 + d)
    x = _randn(torch, g, T, d, dtype=torch.bfloat16)
    x[:, ::5] *= 8
    res = None if residual == "none" else _randn(torch, g, T, d, scale=3.0, dtype=torch.float32 if residual == "fp32"
                                                 else torch.bfloat16)
    w = _randn(torch, g, d) * 0.2 + 1.0 if weighted else None
    x0, res0 = x.clone(), None if res is None else res.clone()
    out = (res if res is not None else x) if in_place else torch.empty_like(x if res is None else res)
    q = torch.full((T, d), -128, dtype=torch.int8, device="cuda")
    scale = torch.full((T,), -7.0, device="cuda")
    iq.ssd_add_rmsnorm_i8(x, res, w, 1e-5, out, q, scale)
    torch.cuda.synchronize()
    if res is None:
        assert torch.equal(out, x0)
    elif residual == "fp32":
        assert torch.equal(out, x0.float() + res0)
    else:
        assert torch.equal(out, (x0.float() + res0.float()).bfloat16())
    _check_codes(host(q), host(scale).astype(np.float64), _np(torch, out), _np(torch, w), 1e-5)
    if not in_place:                       # without residual_out, and with values, the codes are the same
        q2, s2, values = torch.empty_like(q), torch.empty_like(scale), torch.full_like(x, float("nan"))
        iq.ssd_add_rmsnorm_i8(x, res, w, 1e-5, None, q2, s2, values)
        assert torch.equal(q, q2) and torch.equal(scale, s2)
        assert torch.equal(values, (q.float() * scale[:, None]).bfloat16())
    if residual == "none":                 # the start of an fp32 residual stream
        kept = torch.full((T, d), float("nan"), device="cuda")
        iq.ssd_add_rmsnorm_i8(x0, None, w, 1e-5, kept, q, scale)
        assert torch.equal(kept, x0.float())


@pytest.mark.parametrize("T,d", NORM_SIZES)
@pytest.mark.parametrize("pad", [0, 40])
def test_gated_rmsnorm(torch_cuda, T, d, pad):
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, T + 3 * d)
    y = _randn(torch, g, T, d, dtype=torch.bfloat16)
    zrows = _randn(torch, g, T, d + pad, scale=2.0, dtype=torch.bfloat16)
    z = zrows[:, pad // 2 // 8 * 8:][:, :d]
    w = _randn(torch, g, d) * 0.2 + 1.0
    q = torch.full((T, d), -128, dtype=torch.int8, device="cuda")
    scale = torch.full((T,), -7.0, device="cuda")
    iq.ssd_gated_rmsnorm_i8(y, z, w, 1e-5, q, scale)
    zn = _np(torch, z)
    gate_err = (2 * (5 + 1.2 * np.abs(zn).max()) + 1) * E
    _check_codes(host(q), host(scale).astype(np.float64), O.gate(_np(torch, y), zn), _np(torch, w), 1e-5, gate_err)
    q2, s2, values = torch.empty_like(q), torch.empty_like(scale), torch.full_like(y, float("nan"))
    iq.ssd_gated_rmsnorm_i8(y, z, w, 1e-5, q2, s2, values=values)
    assert torch.equal(q, q2) and torch.equal(scale, s2)
    assert torch.equal(values, (q.float() * scale[:, None]).bfloat16())


def test_gate_at_large_arguments(torch_cuda):
    torch = torch_cuda
    import int8_quant_b200 as iq
    d = 64
    z = torch.zeros(1, d, device="cuda")
    z[0, :8] = torch.tensor([100.0, -100.0, 1e30, -1e30, 3e38, -3e38, -88.0, 88.0])
    z[0, 4] = 1e18                                     # finite squares
    z[0, 2] = 1e17
    z, y = z.bfloat16(), torch.ones(1, d, device="cuda").bfloat16()
    q, s = torch.empty(1, d, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    iq.ssd_gated_rmsnorm_i8(y, z, None, 1e-5, q, s)
    ref = O.norm_codes(O.gate(_np(torch, y), _np(torch, z)))
    np.testing.assert_array_equal(host(q), np.rint(ref["pos"]))
    assert abs(float(s) / ref["scale"][0] - 1) < 1e-5


@pytest.mark.parametrize("d", [48, 2560, 16400])
def test_norm_rows_of_zeros_and_rows_that_are_not_finite(torch_cuda, d):
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, d)
    x = _randn(torch, g, 8, d, dtype=torch.bfloat16)
    x[1] = 0
    x[2, d // 2] = float("nan")
    x[3, d - 1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = 1e-38                                        # v * weight below 2^-100
    x[6, 3] = 3e38                                      # the square overflows
    w = torch.ones(d, device="cuda")
    q = torch.full((8, d), -128, dtype=torch.int8, device="cuda")
    s = torch.full((8,), -7.0, device="cuda")
    val = torch.empty_like(x)
    z = torch.full((8, d), 20.0, device="cuda").bfloat16()

    def check():
        qh, sh = host(q), host(s)
        vh = host(val.float())
        assert np.isnan(vh[[2, 3, 4, 6]]).all() and not vh[[1, 5]].any() and np.isfinite(vh[[0, 7]]).all()
        assert not qh[1:7].any()
        assert sh[1] == 1.0 and sh[5] == 1.0 and np.isnan(sh[[2, 3, 4, 6]]).all()
        assert np.abs(qh[0]).max() == 127 and np.abs(qh[7]).max() == 127 and np.isfinite(sh[[0, 7]]).all()

    iq.ssd_add_rmsnorm_i8(x, None, w, 1e-5, None, q, s, val)
    check()
    q.fill_(-128)
    iq.ssd_add_rmsnorm_i8(x, torch.zeros(8, d, device="cuda"), w, 1e-5, None, q, s, val)
    check()
    q.fill_(-128)
    iq.ssd_gated_rmsnorm_i8(x, z, w, 1e-5, q, s, val)
    check()


# ---------------------------------------------------------------- product

MM = [(1, 16, 1), (1, 2560, 10576), (8, 2560, 10576), (7, 5120, 2560), (33, 144, 130), (64, 1024, 257), (65, 512, 512),
      (128, 128, 128), (129, 2064, 1000), (300, 4096, 777), (257, 400, 2049), (1001, 1040, 600), (2000, 256, 4096),
      (2500, 272, 2305), (1001, 8192, 4096),
      (8001, 1024, 1025), (8001, 1024, 1026), (8001, 1024, 1031), (8001, 1024, 1100), (8001, 1024, 1064)]


@pytest.mark.parametrize("T,K,N", MM)
@pytest.mark.parametrize("biased", [True, False])
def test_matmul(torch_cuda, T, K, N, biased):
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, T + K + N)
    q = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    Wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    s_t = torch.rand(T, generator=g, device="cuda") + 0.1
    s_w = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-4
    bias = _randn(torch, g, N) if biased else None
    # rows behind the last one, to see that nothing is written there
    room = torch.full((T * N + 512,), float("nan"), device="cuda").bfloat16()
    out, st = room[:T * N].view(T, N), torch.zeros(1, dtype=torch.int32, device="cuda")
    iq.ssd_matmul_i8(q, s_t, Wq, s_w, bias, out, st)
    torch.cuda.synchronize()
    assert iq.ssd_workspace_status(st) == 0
    assert torch.isnan(room[T * N:]).all()
    ref = O.matmul(host(q), host(s_t), host(Wq), host(s_w), None if bias is None else host(bias))
    off = np.abs(_np(torch, out) - ref["out"])
    lim = H * np.abs(ref["out"]) * (1 + 2.0 ** -10) + 8 * E * ref["mag"] + 1e-38
    assert (off <= lim).all(), (off / lim).max()


def test_matmul_every_kernel_and_split_gives_the_same_bits(torch_cuda):
    """Sizes over the choices (tile heights, CTAs an SM, K splits, ragged ends): the exact sum, two fp32 products and
    one rounding, bit for bit."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    import random
    rng = random.Random(5)
    sizes = [(1, 8192, 9400), (20, 4096, 8500), (64, 8192, 18000), (3, 2064, 20000), (40, 3088, 21000), (9, 4464, 4480),
             (17, 5360, 2137), (5, 144, 3000), (50, 272, 9000), (64, 400, 64), (16, 4000, 2040), (100, 2928, 8647)]
    for _ in range(80):
        sizes.append((round(1500 ** rng.random()), 16 * round(400 ** rng.random()), round(20000 ** rng.random())))
    g, st = _gen(torch, 1), torch.zeros(1, dtype=torch.int32, device="cuda")
    for T, K, N in sizes:
        q = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
        Wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        s_t, s_w = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda") * 1e-3
        out = torch.full((T, N), float("nan"), device="cuda").bfloat16()
        iq.ssd_matmul_i8(q, s_t, Wq, s_w, None, out, st)
        acc = (q.double() @ Wq.double().T).float()                       # exact below 2^53, rounded once
        assert torch.equal(out, (acc * s_w * s_t[:, None]).bfloat16()), (T, K, N)
    assert iq.ssd_workspace_status(st) == 0


@pytest.mark.parametrize("code", [127, -128])
def test_matmul_extreme_sums_stay_exact(torch_cuda, code):
    """All codes the largest over the longest k: the sum 131056 * 128^2 fits INT32, the next k's would not."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    for T in (3, 200):
        K, N = 131056, 160
        q = torch.full((T, K), code, dtype=torch.int8, device="cuda")
        Wq = torch.full((N, K), 127 if code < 0 else -127, dtype=torch.int8, device="cuda")
        Wq[::2] = code
        one = lambda n: torch.full((n,), 2.0 ** -15, device="cuda")  # noqa: E731
        out, st = torch.empty(T, N, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda")
        iq.ssd_matmul_i8(q, one(T), Wq, one(N), None, out, st)
        want, other = K * code * code * 2.0 ** -30, -K * abs(code) * 127 * 2.0 ** -30
        got = _np(torch, out)
        assert np.abs(got[:, ::2] / want - 1).max() <= H and np.abs(got[:, 1::2] / other - 1).max() <= H


def test_matmul_carries_a_poisoned_scale(torch_cuda):
    torch = torch_cuda
    import int8_quant_b200 as iq
    q = torch.zeros(5, 64, dtype=torch.int8, device="cuda")
    s_t = torch.ones(5, device="cuda")
    s_t[2] = float("nan")
    Wq = torch.ones(40, 64, dtype=torch.int8, device="cuda")
    out, st = torch.empty(5, 40, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda")
    iq.ssd_matmul_i8(q, s_t, Wq, torch.ones(40, device="cuda"), None, out, st)
    bad = torch.isnan(out)
    assert bad[2].all() and not bad[[0, 1, 3, 4]].any()


# ---------------------------------------------------------------- convolution

def _conv_case(torch, seed, b, L, Hn, P, G, N, W, biased=True, from_state=False, lengths=None, extra=24):
    g = _gen(torch, seed)
    C, d = Hn * P + 2 * G * N, Hn * P
    rows = _randn(torch, g, b, L, d + C + (Hn + 7) // 8 * 8 + extra, dtype=torch.bfloat16)
    c = {"xbc": rows[:, :, d:d + C], "dt_raw": rows[:, :, d + C:d + C + Hn],
         "weight": _randn(torch, g, W, C, scale=0.6), "bias": _randn(torch, g, C, scale=0.3) if biased else None,
         "dt_bias": _randn(torch, g, Hn, scale=2.0) - 3.0,
         "init": _randn(torch, g, b, W - 1, C, dtype=torch.bfloat16) if from_state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    c["x"], c["B"], c["C"] = (nan(b, L, Hn, P).bfloat16(), nan(b, L, G, N).bfloat16(), nan(b, L, G, N).bfloat16())
    c["dt"], c["final"] = nan(b, L, Hn), nan(b, W - 1, C).bfloat16()
    return c


def _check_conv(torch, c):
    ref = O.conv(_np(torch, c["xbc"]), _np(torch, c["weight"]), _np(torch, c["bias"]), _np(torch, c["init"]),
                 None if c["lengths"] is None else host(c["lengths"]), _np(torch, c["dt_raw"]), _np(torch, c["dt_bias"]))
    b, L = c["x"].shape[:2]
    got = np.concatenate([_np(torch, c[k]).reshape(b, L, -1) for k in ("x", "B", "C")], axis=2)
    off = np.abs(got - ref["out"])
    lim = (H * (1 + 2.0 ** -10) + 2 * (5 + 1.2 * np.abs(ref["u"])) * E) * np.abs(ref["out"]) + 1.2 * 5 * E * ref["mag"]
    assert (off <= lim).all(), np.nanmax(off / np.maximum(lim, 1e-300))
    dt = _np(torch, c["dt"])
    assert (np.abs(dt - ref["dt"]) <= ref["dt"] * (12 + np.abs(ref["v"])) * E).all()
    np.testing.assert_array_equal(_np(torch, c["final"]), ref["state"])
    return ref


def _run_conv(c):
    import int8_quant_b200 as iq
    iq.ssd_conv_fwd_bf16(c["xbc"], c["dt_raw"], c["weight"], c["bias"], c["dt_bias"], c["lengths"], c["init"], c["x"],
                         c["dt"], c["B"], c["C"], c["final"])


CONV_LENGTHS = [(1, 1), (2, 2), (3, 3), (1, 31), (2, 32), (2, 33), (1, 63), (2, 64), (1, 65), (1, 130), (5, 257)]
CONV_FORMS = [(4, True, True), (4, False, False), (3, True, False), (2, True, True)]
CONV_CASES = [(b, L, dims, *form) for b, L in CONV_LENGTHS for dims in [(2, 64, 1, 128), (3, 24, 3, 8)]
              for form in CONV_FORMS] + [(b, L, (80, 64, 1, 128), 4, True, True) for b, L in [(1, 1), (2, 33), (1, 130)]]


@pytest.mark.parametrize("b,L,dims,W,biased,from_state", CONV_CASES)
def test_conv(torch_cuda, b, L, dims, W, biased, from_state):
    torch = torch_cuda
    c = _conv_case(torch, L * 11 + W, b, L, *dims, W, biased, from_state)
    _run_conv(c)
    _check_conv(torch, c)


@pytest.mark.parametrize("lengths", [[0, 1, 2, 3, 4, 70], [70, 69, 33, 32, 31, 64], [-5, 1000, 5, 0, 0, 0]])
@pytest.mark.parametrize("from_state", [True, False])
def test_conv_padded_batch(torch_cuda, lengths, from_state):
    torch = torch_cuda
    c = _conv_case(torch, 3, 6, 70, 4, 16, 2, 16, 4, True, from_state, lengths)
    live = np.clip(lengths, 0, 70)
    for r in range(6):                                   # what lies in the padding does not matter
        c["xbc"][r, live[r]:] = float("nan")
        c["dt_raw"][r, live[r]:] = float("inf")
    clean = dict(c, xbc=torch.nan_to_num(c["xbc"], nan=0.0), dt_raw=torch.nan_to_num(c["dt_raw"], posinf=0.0))
    _run_conv(c)
    _check_conv(torch, clean)


def test_conv_split_of_a_row_reproduces_it(torch_cuda):
    torch = torch_cuda
    c = _conv_case(torch, 9, 2, 50, 4, 64, 2, 128, 4)
    _run_conv(c)
    for cut in (1, 2, 3, 17, 49):
        state, parts = None, []
        for lo, hi in ((0, cut), (cut, 50)):
            p = dict(c, xbc=c["xbc"][:, lo:hi], dt_raw=c["dt_raw"][:, lo:hi], init=state, final=torch.empty_like(c["final"]))
            # slices of a longer batch are not evenly spaced: copy them into rows of their own
            rows = torch.cat([p["xbc"], p["dt_raw"], torch.zeros_like(p["dt_raw"])], 2)
            C, Hn = c["xbc"].shape[2], c["dt_raw"].shape[2]
            p["xbc"], p["dt_raw"] = rows[:, :, :C], rows[:, :, C:C + Hn]
            for k in ("x", "B", "C", "dt"):
                p[k] = torch.empty_like(c[k][:, lo:hi])
            _run_conv(p)
            state = p["final"]
            parts.append(p)
        for k in ("x", "B", "C", "dt"):
            assert torch.equal(torch.cat([p[k] for p in parts], 1), c[k]), (cut, k)
        assert torch.equal(state, c["final"])


@pytest.mark.parametrize("b", [1, 3, 129])
@pytest.mark.parametrize("dims", [(2, 64, 1, 128), (3, 24, 3, 8), (128, 64, 8, 128)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_step_equals_a_scan_of_one_token(torch_cuda, b, dims, W):
    torch = torch_cuda
    import int8_quant_b200 as iq
    c = _conv_case(torch, b + W, b, 1, *dims, W, True, True)
    _run_conv(c)
    if dims[0] < 128:
        _check_conv(torch, c)
    state = c["init"].clone()
    o = {k: torch.full_like(c[k][:, 0], float("nan")) for k in ("x", "B", "C", "dt")}
    iq.ssd_conv_step_bf16(c["xbc"][:, 0], c["dt_raw"][:, 0], c["weight"], c["bias"], c["dt_bias"], state, o["x"],
                          o["dt"], o["B"], o["C"])
    for k in o:
        assert torch.equal(o[k], c[k][:, 0]), k
    assert torch.equal(state, c["final"])


def test_conv_without_dt_and_without_a_final_state(torch_cuda):
    torch = torch_cuda
    import int8_quant_b200 as iq
    c = _conv_case(torch, 4, 2, 37, 4, 16, 1, 16, 4)
    _run_conv(c)
    x, B, C = (torch.empty_like(c[k]) for k in ("x", "B", "C"))
    iq.ssd_conv_fwd_bf16(c["xbc"], None, c["weight"], c["bias"], None, None, None, x, None, B, C, None)
    assert torch.equal(x, c["x"]) and torch.equal(B, c["B"]) and torch.equal(C, c["C"])


def test_conv_of_no_tokens_copies_the_state(torch_cuda):
    torch = torch_cuda
    for from_state in (True, False):
        c = _conv_case(torch, 4, 2, 0, 4, 16, 1, 16, 4, from_state=from_state)
        _run_conv(c)
        torch.cuda.synchronize()
        assert torch.equal(c["final"], c["init"] if from_state else torch.zeros_like(c["final"]))


# ---------------------------------------------------------------- long tensors

def test_rows_past_2_to_the_31_elements(torch_cuda):
    """The last rows of calls whose tensors have more than 2^31 elements, bit for bit those of a call on them alone."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, 5)
    T, d, last = 530000, 4096, 9                          # 2.17e9 features
    x = torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    tail = _randn(torch, g, last, d, dtype=torch.bfloat16)
    x.zero_()
    x[-last:] = tail
    q, s = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    q2, s2 = torch.empty(last, d, dtype=torch.int8, device="cuda"), torch.empty(last, device="cuda")
    iq.ssd_add_rmsnorm_i8(x, None, None, 1e-5, None, q, s)
    iq.ssd_add_rmsnorm_i8(tail, None, None, 1e-5, None, q2, s2)
    assert torch.equal(q[-last:], q2) and torch.equal(s[-last:], s2) and not q[:-last].any()
    iq.ssd_gated_rmsnorm_i8(x, x, None, 1e-5, q, s)
    iq.ssd_gated_rmsnorm_i8(tail, tail, None, 1e-5, q2, s2)
    assert torch.equal(q[-last:], q2) and torch.equal(s[-last:], s2)
    del x

    # product: codes and outputs, aligned rows and not
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    small = q2.contiguous()
    for n in (4100, 4104):
        W8 = torch.randint(-127, 128, (n, d), generator=g, device="cuda", dtype=torch.int8)
        sw = torch.rand(n, generator=g, device="cuda")
        out, out2 = torch.empty(T, n, device="cuda", dtype=torch.bfloat16), torch.empty(last, n, device="cuda").bfloat16()
        iq.ssd_matmul_i8(q, s, W8, sw, sw, out, st)
        iq.ssd_matmul_i8(small, s2, W8, sw, sw, out2, st)
        assert torch.equal(out[-last:], out2)
        assert torch.equal(out[:1], sw.bfloat16()[None])   # a token of zeros: the bias
        del out
    assert iq.ssd_workspace_status(st) == 0
    del q, s

    # convolution: two rows of a batch, the second beyond 2^31 elements
    c = _conv_case(torch, 3, 1, 70, 4, 64, 1, 128, 4)
    ch, L, ld = c["xbc"].shape[2], 1100000, 1024
    rows = torch.zeros(2, L, ld, device="cuda", dtype=torch.bfloat16)
    rows[1, -70:, :ch] = c["xbc"][0]
    rows[1, -70:, ch:ch + 4] = c["dt_raw"][0]
    big = {"x": (2, L, 4, 64), "B": (2, L, 1, 128), "C": (2, L, 1, 128)}
    big = {k: torch.empty(v, device="cuda", dtype=torch.bfloat16) for k, v in big.items()}
    dt, fin = torch.empty(2, L, 4, device="cuda"), torch.empty(2, 3, ch, device="cuda", dtype=torch.bfloat16)
    iq.ssd_conv_fwd_bf16(rows[:, :, :ch], rows[:, :, ch:ch + 4], c["weight"], c["bias"], c["dt_bias"], None, None,
                         big["x"], dt, big["B"], big["C"], fin)
    _run_conv(c)                                           # from zeros, as the long row's inputs ahead of it are
    for k in big:
        assert torch.equal(big[k][1, -70:], c[k][0]), k
    assert torch.equal(dt[1, -70:], c["dt"][0]) and torch.equal(fin[1], c["final"][0])


@pytest.mark.parametrize("N", [2048, 2050])
def test_product_of_a_token_does_not_depend_on_its_batch(torch_cuda, N):
    """Few tokens or many, K split or not: the same bits (exact sums, one way of scaling)."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, N)
    T, K = 1500, 1024
    q = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    W8 = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    s, sw, b = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda"), _randn(torch, g, N)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(T, N, device="cuda").bfloat16()
    iq.ssd_matmul_i8(q, s, W8, sw, b, out, st)
    for n in (1, 16, 24, 60, 120, 400):
        part = torch.empty(n, N, device="cuda").bfloat16()
        iq.ssd_matmul_i8(q[:n], s[:n], W8, sw, b, part, st)
        assert torch.equal(part, out[:n]), n


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses_wrong_tensors(torch_cuda):
    torch = torch_cuda
    import int8_quant_b200 as iq
    T, d = 4, 64
    x = torch.zeros(T, d, device="cuda").bfloat16()
    q, s = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    ok = dict(x=x, residual=None, weight=None, eps=1e-5, residual_out=None, q=q, scale=s)
    wrong = [dict(x=x.float()), dict(x=x.cpu()), dict(q=q[:, ::2]), dict(q=q[:2]), dict(scale=s.double()),
             dict(residual=torch.zeros(T, d + 1, device="cuda")), dict(weight=torch.ones(d + 1, device="cuda")),
             dict(residual=torch.zeros(T, d, device="cuda"), residual_out=torch.empty_like(x)),
             dict(residual=torch.zeros(T, d, device="cuda").half()), dict(eps=0.0), dict(x=x[0]),
             dict(x=torch.zeros(T, 2 * d, device="cuda").bfloat16()[:, ::2])]
    iq.ssd_add_rmsnorm_i8(**ok)
    for w in wrong:
        with pytest.raises(iq.SsdError) as err:
            iq.ssd_add_rmsnorm_i8(**{**ok, **w})
        assert err.value.status == 1
    with pytest.raises(iq.SsdError):                     # z's features not next to each other
        iq.ssd_gated_rmsnorm_i8(x, torch.zeros(T, 2 * d, device="cuda").bfloat16()[:, ::2], None, 1e-5, q, s)
    with pytest.raises(iq.SsdError):                     # rows 2-byte aligned
        iq.ssd_gated_rmsnorm_i8(x, torch.zeros(T, d + 8, device="cuda").bfloat16()[:, 1:d + 1], None, 1e-5, q, s)
    W8 = torch.zeros(8, d, dtype=torch.int8, device="cuda")
    out, st, sw = torch.empty(T, 8, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda"), \
        torch.ones(8, device="cuda")
    iq.ssd_matmul_i8(q, s, W8, sw, None, out, st)
    for a in ((q, s, W8[:, :48], sw, None, out, st), (q, s, W8, sw[:7], None, out, st), (q, s, W8, sw, sw[:3], out, st),
              (q, s, W8, sw, None, out.float(), st), (q, s, W8, sw, None, out, None or st.long()),
              (q, s[:3], W8, sw, None, out, st)):
        with pytest.raises(iq.SsdError):
            iq.ssd_matmul_i8(*a)
    c = _conv_case(torch, 1, 2, 8, 4, 16, 1, 16, 4, from_state=True)
    _run_conv(c)
    gaps = torch.zeros(2, 16, c["xbc"].shape[2], device="cuda").bfloat16()[:, :8]   # rows not evenly spaced
    for k, v in (("xbc", gaps), ("xbc", c["xbc"].float()), ("dt_raw", c["dt_raw"].contiguous()), ("dt", None),
                 ("final", c["init"]), ("init", c["init"][:, :2]), ("weight", c["weight"][:, :-8]),
                 ("lengths", torch.zeros(2, dtype=torch.int64, device="cuda")), ("B", c["B"].float())):
        with pytest.raises(iq.SsdError):
            _run_conv({**c, k: v})
    torch.cuda.synchronize()


# ---------------------------------------------------------------- streams and graphs

def test_from_four_threads_at_a_time(torch_cuda):
    """Four host threads, each with a stream and buffers of its own: the bits of one."""
    import threading
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, 1)
    x, z = _randn(torch, g, 40, 1024, dtype=torch.bfloat16), _randn(torch, g, 40, 1024, dtype=torch.bfloat16)
    W8 = torch.randint(-127, 128, (1500, 1024), generator=g, device="cuda", dtype=torch.int8)
    sw, status = torch.rand(1500, generator=g, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    results = {}

    def work(name, reps):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            q, s = torch.empty(40, 1024, dtype=torch.int8, device="cuda"), torch.empty(40, device="cuda")
            out = torch.empty(40, 1500, device="cuda").bfloat16()
            for _ in range(reps):
                iq.ssd_gated_rmsnorm_i8(x, z, None, 1e-5, q, s)
                iq.ssd_matmul_i8(q, s, W8, sw, None, out, status)
        stream.synchronize()
        results[name] = out

    work("ref", 1)
    threads = [threading.Thread(target=work, args=(i, 100)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(results[i], results["ref"]) for i in range(4))
    assert iq.ssd_workspace_status(status) == 0


def test_on_a_side_stream_and_in_two_graphs(torch_cuda):
    """Each operator on a stream of its own, then captured in two graphs that share every buffer but the outputs and
    are replayed on two streams at a time: the same bits each time."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = _gen(torch, 0)
    T, d, n = 96, 512, 1000
    x, z = _randn(torch, g, T, d, dtype=torch.bfloat16), _randn(torch, g, T, d, dtype=torch.bfloat16)
    Wq = torch.randint(-127, 128, (n, d), generator=g, device="cuda", dtype=torch.int8)
    s_w, status = torch.rand(n, generator=g, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    conv = _conv_case(torch, 2, 3, 40, 4, 64, 1, 128, 4, from_state=True)

    def outputs():
        o = {"q1": torch.empty(T, d, dtype=torch.int8, device="cuda"), "s1": torch.empty(T, device="cuda"),
             "q2": torch.empty(T, d, dtype=torch.int8, device="cuda"), "s2": torch.empty(T, device="cuda"),
             "o1": torch.empty(T, n, device="cuda").bfloat16(), "o2": torch.empty(5, n, device="cuda").bfloat16()}
        o.update({k: torch.empty_like(conv[k]) for k in ("x", "dt", "B", "C", "final")})
        return o

    def go(o):
        iq.ssd_add_rmsnorm_i8(x, None, None, 1e-5, None, o["q1"], o["s1"])
        iq.ssd_gated_rmsnorm_i8(x, z, None, 1e-5, o["q2"], o["s2"])
        iq.ssd_matmul_i8(o["q1"], o["s1"], Wq, s_w, None, o["o1"], status)
        iq.ssd_matmul_i8(o["q2"][:5], o["s2"][:5], Wq, s_w, None, o["o2"], status)
        iq.ssd_conv_fwd_bf16(conv["xbc"], conv["dt_raw"], conv["weight"], conv["bias"], conv["dt_bias"], None,
                             conv["init"], o["x"], o["dt"], o["B"], o["C"], o["final"])

    ref = outputs()
    go(ref)
    torch.cuda.synchronize()
    same = lambda o: all(torch.equal(o[k].view(torch.uint8), ref[k].view(torch.uint8)) for k in ref)  # noqa: E731
    side = torch.cuda.Stream()
    o = outputs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(o)
    torch.cuda.synchronize()
    assert same(o)
    graphs = []
    for _ in range(2):
        o, gr = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            go(o)
        graphs.append((gr, o))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for _, o in graphs:
            for t in o.values():
                t.zero_()
        torch.cuda.synchronize()
        for (gr, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert all(same(o) for _, o in graphs)
    assert iq.ssd_workspace_status(status) == 0
