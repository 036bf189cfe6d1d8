"""Host-side validation of the layer operators (no GPU): every call below fails before anything is launched, or
has nothing to do."""
import ctypes

import pytest

import int8_quant_b200 as iq

F = ctypes.c_void_p(0x10000)              # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10004)
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_add_rmsnorm_refusals():
    f = iq.library().ssd_add_rmsnorm_i8
    good = [4, 64, F, F, 1, F, 1e-5, F, F, F, None, None]
    for i, v, want in [(0, -1, INVALID), (1, 0, INVALID), (1, 40, UNSUPPORTED), (1, 32784, UNSUPPORTED),
                       (2, None, INVALID), (2, ODD, INVALID), (3, ODD, INVALID),
                       (5, ODD, INVALID), (6, 0.0, INVALID), (6, -1.0, INVALID), (6, float("nan"), INVALID),
                       (7, ODD, INVALID), (8, None, INVALID), (8, ODD, INVALID), (9, None, INVALID), (10, ODD, INVALID)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(0, 64, None, None, 0, None, 1e-5, None, None, None, None, None) == OK      # no tokens


def test_gated_rmsnorm_refusals():
    f = iq.library().ssd_gated_rmsnorm_i8
    good = [4, 64, F, F, 96, F, 1e-5, F, F, None, None]
    for i, v, want in [(0, -1, INVALID), (1, 24, UNSUPPORTED), (2, None, INVALID), (3, None, INVALID), (3, ODD, INVALID),
                       (4, 56, INVALID), (4, 100, INVALID), (6, 0.0, INVALID), (7, None, INVALID), (8, ODD, INVALID),
                       (9, ODD, INVALID)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(0, 64, None, None, 64, None, 1e-5, None, None, None, None) == OK


def test_matmul_refusals():
    f = iq.library().ssd_matmul_i8
    good = [4, 64, 8, F, F, F, F, F, F, F, None]
    for i, v, want in [(0, -1, INVALID), (1, 0, INVALID), (2, 0, INVALID), (1, 40, UNSUPPORTED),
                       (1, 131072, UNSUPPORTED), (0, 2 ** 30 + 1, UNSUPPORTED), (2, 2 ** 30 + 1, UNSUPPORTED),
                       (3, None, INVALID), (3, ODD, INVALID), (4, None, INVALID),
                       (5, None, INVALID), (6, None, INVALID), (7, ODD, INVALID), (8, None, INVALID), (8, ODD, INVALID),
                       (9, None, INVALID)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(0, 64, 8, None, None, None, None, None, None, None, None) == OK


def _shape(b=2, L=8, H=4, P=16, G=1, N=16):
    return ctypes.byref(iq.SsdShape.of(b, L, H, P, G, N, 64))


def test_conv_fwd_refusals():
    f = iq.library().ssd_conv_fwd_bf16
    far = ctypes.c_void_p(0x900000)
    good = [_shape(), 4, F, F, 104, F, F, F, F, F, F, F, F, F, far, None]
    for i, v, want in [(0, None, INVALID), (0, _shape(b=-1), INVALID), (0, _shape(H=3, G=2), INVALID),
                       (0, _shape(H=1, P=12, N=8), UNSUPPORTED), (0, _shape(N=4), UNSUPPORTED), (1, 1, UNSUPPORTED),
                       (1, 5, UNSUPPORTED), (0, _shape(b=2 ** 31 - 1, L=2 ** 31 - 1), UNSUPPORTED), (2, None, INVALID),
                       (2, ODD, INVALID), (3, None, INVALID), (3, ctypes.c_void_p(0x10001), INVALID), (4, 88, INVALID),
                       (4, 100, INVALID), (5, None, INVALID), (6, ODD, INVALID), (7, None, INVALID), (8, ODD, INVALID),
                       (9, ODD, INVALID), (10, None, INVALID), (11, None, INVALID), (12, None, INVALID),
                       (13, ODD, INVALID), (14, ODD, INVALID), (14, F, INVALID),
                       (14, ctypes.c_void_p(0x10000 + 2 * 2 * 3 * 96 - 16), INVALID)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(_shape(b=0), 4, None, None, 104, None, None, None, None, None, None, None, None, None, None, None) == OK
    assert f(_shape(L=0), 4, None, None, 104, None, None, None, None, None, None, None, None, None, None, None) == OK


def test_conv_step_refusals():
    f = iq.library().ssd_conv_step_bf16
    good = [_shape(L=1), 4, F, F, 104, F, F, F, F, F, F, F, F, None]
    for i, v, want in [(0, None, INVALID), (0, _shape(L=2), INVALID), (0, _shape(L=1, N=4), UNSUPPORTED),
                       (1, 0, UNSUPPORTED), (2, None, INVALID), (4, 8, INVALID), (5, ODD, INVALID), (7, None, INVALID),
                       (8, None, INVALID), (8, ODD, INVALID), (9, None, INVALID), (12, None, INVALID)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(_shape(b=0, L=1), 4, None, None, 104, None, None, None, None, None, None, None, None, None) == OK


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    q, s = torch.empty(2, 32, dtype=torch.int8), torch.empty(2)
    with pytest.raises(iq.SsdError) as err:
        iq.ssd_add_rmsnorm_i8(x, None, None, 1e-5, None, q, s)
    assert err.value.status == INVALID and "CUDA device" in str(err.value)
    with pytest.raises(iq.SsdError):
        iq.ssd_gated_rmsnorm_i8(x, x, None, 1e-5, q, s)
    with pytest.raises(iq.SsdError):
        iq.ssd_matmul_i8(q, s, q, s, None, x, s)
    y = torch.zeros(2, 1, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(iq.SsdError):
        iq.ssd_conv_fwd_bf16(x, None, s, None, None, None, None, y, None, y, y, None)
    with pytest.raises(iq.SsdError):
        iq.ssd_conv_step_bf16(x, None, s, None, None, x, y[:, 0], None, y[:, 0], y[:, 0])


def test_matmul_scales_and_status_need_their_elements_alignment():
    f = iq.library().ssd_matmul_i8
    good = [4, 64, 8, F, F, F, F, F, F, F, None]
    for i in (4, 6, 9):
        for p in (0x10002, 0x10001):
            a = list(good)
            a[i] = ctypes.c_void_p(p)
            assert f(*a) == INVALID, (i, p)
