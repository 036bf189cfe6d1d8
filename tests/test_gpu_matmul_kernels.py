"""Every kernel of the INT8 product, bit for bit: the exact sum, two fp32 products, the bias's addition fused into the
second, one rounding to bf16.  tests/matmul_sizes.py has the sizes; that they reach the kernels on the GPU at hand is
checked first."""
import numpy as np
import pytest

from tests import matmul_sizes as S
from tests.gpu_common import bf16_to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import int8_quant_b200 as iq
    iq.library()
    return torch


def _plan(torch, *a):
    import int8_quant_b200 as iq
    return iq.ssd_matmul_i8_plan(*a, torch.cuda.get_device_properties(0).multi_processor_count)


def _check(torch, T, K, N):
    """Codes of every value, -128 too; rows behind the last one and words beside the status stay as they were."""
    import int8_quant_b200 as iq
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    q = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    Wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    s_t, s_w = torch.rand(T, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda") * 1e-3
    bias = torch.randn(N, generator=g, device="cuda")
    room = torch.full((T * N + 512,), float("nan"), device="cuda").bfloat16()
    out, st = room[:T * N].view(T, N), torch.zeros(3, dtype=torch.int32, device="cuda")
    acc = torch.empty(T, N, device="cuda")
    for t in range(0, T, 1024):                          # exact in 64 bits, rounded once
        acc[t:t + 1024] = (q[t:t + 1024].double() @ Wq.double().T).float()
    iq.ssd_matmul_i8(q, s_t, Wq, s_w, None, out, st[1:2])
    assert torch.equal(out, (acc * s_w * s_t[:, None]).bfloat16())
    out.fill_(float("nan"))
    iq.ssd_matmul_i8(q, s_t, Wq, s_w, bias, out, st[1:2])
    # the product of two fp32 is exact in 64 bits; its sum with the bias is rounded to 64 and then to 32 bits, which
    # differs from the fused rounding for one value in 2^29, and that shows in bf16 (a tie 16 bits up) for one of 2^16
    want = ((acc * s_w).double() * s_t.double()[:, None] + bias.double()).float().bfloat16()
    assert torch.equal(out, want)
    assert torch.isnan(room[T * N:]).all() and not st.any()


@pytest.mark.parametrize("T,K,N", S.PAIRS)
def test_pairs(torch_cuda, T, K, N):
    assert _plan(torch_cuda, T, K, N).pair
    _check(torch_cuda, T, K, N)


@pytest.mark.parametrize("bn,split", S.FEW)
def test_clusters(torch_cuda, bn, split):
    a = S.FEW[bn, split]
    p = _plan(torch_cuda, *a)
    assert (p.pair, p.tile_tokens, p.split) == (0, bn, split)
    _check(torch_cuda, *a)


@pytest.mark.parametrize("code", [127, -128])
@pytest.mark.parametrize("T,N,pair", S.EXTREME)
def test_largest_sums(torch_cuda, T, N, pair, code):
    """All codes the largest over the longest k; scales are powers of two, so one rounding to fp32 and one to bf16."""
    torch = torch_cuda
    import int8_quant_b200 as iq
    K = S.LONGEST_K
    assert _plan(torch, T, K, N).pair == pair
    q = torch.full((T, K), code, dtype=torch.int8, device="cuda")
    Wq = torch.full((N, K), 127 if code < 0 else -127, dtype=torch.int8, device="cuda")
    Wq[::2] = code
    one = lambda n: torch.full((n,), 2.0 ** -15, device="cuda")  # noqa: E731
    out, st = torch.empty(T, N, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda")
    iq.ssd_matmul_i8(q, one(T), Wq, one(N), None, out, st)
    sums = torch.tensor([K * code * code, K * code * (127 if code < 0 else -127)], dtype=torch.float64)
    assert sums.abs().max() < 2 ** 31
    want = bf16_to_np((sums.float() * 2.0 ** -30).bfloat16())
    got = bf16_to_np(out)
    np.testing.assert_array_equal(got[:, ::2], np.broadcast_to(want[0], got[:, ::2].shape))
    np.testing.assert_array_equal(got[:, 1::2], np.broadcast_to(want[1], got[:, 1::2].shape))


@pytest.mark.parametrize("N", [4096, 4101])
def test_a_tokens_bits_on_pairs_and_clusters(torch_cuda, N):
    torch = torch_cuda
    import int8_quant_b200 as iq
    g = torch.Generator(device="cuda").manual_seed(N)
    T, K = 1500, 1040
    q = torch.randint(-127, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    Wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    s, sw, b = (torch.rand(n, generator=g, device="cuda") for n in (T, N, N))
    st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(T, N, device="cuda").bfloat16()
    assert _plan(torch, T, K, N).pair
    iq.ssd_matmul_i8(q, s, Wq, sw, b, out, st)
    for n in (1, 17, 64, 100):
        assert not _plan(torch, n, K, N).pair
        part = torch.empty(n, N, device="cuda").bfloat16()
        iq.ssd_matmul_i8(q[:n], s[:n], Wq, sw, b, part, st)
        assert torch.equal(part, out[:n]), n
