"""The widest matrices that the gradients of a W8A8 linear accept, 2^30 columns (about 20 GB), and
matrices of more than 2^31 values (up to about 35 GB) in the gradients and block-boundary norms."""
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from test_gpu_grad_gemm import _assert_close, _codes, _dequantized, _scales, _silu_reference, _tol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _normal(*shape, seed, std=1.0):
    """bf16, drawn on the device (in bf16, so nothing of twice the size is held)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)


@pytest.mark.parametrize("K", [1 << 30, (1 << 30) - 16])
def test_weight_gradient_of_the_widest_rows(K):
    """One token, so dw[n, k] = dy[n] s q[k], exact with powers of two; every column is looked at,
    the first ones among them (whose distance to the row's end, in bytes, passes 32 bits)."""
    N = 8
    dy = torch.tensor([[2.0 ** (n - 4) for n in range(N)]], dtype=torch.bfloat16, device="cuda")
    xq = torch.randint(-128, 128, (1, K), dtype=torch.int8, device="cuda")
    dw = torch.full((N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    w8.w8a8_gemm_wgrad(dy, xq, torch.tensor([0.5], device="cuda"), dw=dw)
    torch.cuda.synchronize()
    assert w8.w8a8_last_device_status() == 0
    for n in range(N):
        want = xq[0].to(torch.bfloat16).mul_(float(dy[0, n]) * 0.5)
        assert torch.equal(dw[n], want), n


FAR = 2 ** 31  # values; the last rows of each matrix below lie past it


@pytest.mark.parametrize("M,N,K", [(280_001, 8192, 512), (280_001, 512, 8192)])
def test_input_gradient_of_far_rows(M, N, K):
    """dy, then dx, of more than 2^31 values."""
    assert M * max(N, K) > FAR
    dy, q, s = _normal(M, N, seed=1, std=0.05), _codes((N, K), False, 2), _scales(N, 3)
    dx = w8.w8a8_gemm_dgrad(dy, q, s)
    b = _dequantized(q, s)
    for rows in (slice(0, 40), slice(M - 300, M)):
        ref = dy[rows].double() @ b
        _assert_close(dx[rows], ref, _tol(ref, dy[rows].double().abs() @ b.abs(), N))
    assert w8.w8a8_last_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(70_001, 512, 16384), (140_001, 8200, 8192)])
def test_gated_block_backward_of_far_rows(M, N, K):
    """gate|up and its gradient of more than 2^31 values, in both wide forms of the kernel."""
    assert 2 * M * K > FAR
    dy, q, s = _normal(M, N, seed=4, std=0.05), _codes((N, K), True, 5), _scales(N, 6)
    gate_up = _normal(M, 2 * K, seed=7, std=4.0)
    out = w8.w8a8_gemm_dgrad_silu_fp8(dy, q, s, gate_up)
    for rows in (slice(0, 40), slice(M - 300, M)):
        _assert_close(out[rows], *_silu_reference(dy[rows], q, s, gate_up[rows]))
    assert w8.w8a8_last_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(72, 280_008, 8192), (8200, 280_008, 512)])
def test_weight_gradient_of_far_rows(M, N, K):
    """dw, then dy, of more than 2^31 values; the codes converted ahead, then in the kernel."""
    assert N * max(M, K) > FAR
    dy, q, s = _normal(M, N, seed=8, std=0.05), _codes((M, K), False, 9), _scales(M, 10)
    dw = w8.w8a8_gemm_wgrad(dy, q, s)
    b = _dequantized(q, s)
    for rows in (slice(0, 40), slice(N - 300, N)):
        a = dy[:, rows].double().t()
        ref = a @ b
        _assert_close(dw[rows], ref, _tol(ref, a.abs() @ b.abs(), M))
    assert w8.w8a8_last_device_status() == 0


@pytest.mark.parametrize("M,K", [(270_001, 8192), (70_001, 32768)])
def test_norms_of_far_rows(M, K):
    """The last rows of a call of more than 2^31 values against a call of those rows alone."""
    assert M * K > FAR
    y, r = _normal(M, K, seed=11), _normal(M, K, seed=12)
    g = (1 + 0.1 * _normal(K, seed=13)).float()
    gate = torch.rand(M, 1, device="cuda")
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(y, r, g, 1e-5, gamma_post=g, gate=gate)
    last = slice(M - 50, M)
    want = w8.w8a8_sandwich_rmsnorm_quant(y[last], r[last], g, 1e-5, gamma_post=g, gate=gate[last])
    for a, b in zip((q, s, h), want):
        assert torch.equal(a[last], b)
    dy, dr, _, _, dgate = w8.w8a8_sandwich_rmsnorm_backward(r, y, h, g, 1e-5, gamma_post=g,
                                                            gate=gate)
    wy, wr, _, _, wg = w8.w8a8_sandwich_rmsnorm_backward(r[last], y[last], h[last], g, 1e-5,
                                                         gamma_post=g, gate=gate[last])
    assert torch.equal(dy[last], wy) and torch.equal(dr[last], wr)
    assert torch.equal(dgate[last], wg)
    assert w8.w8a8_last_device_status() == 0
