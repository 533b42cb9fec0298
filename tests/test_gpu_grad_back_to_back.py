"""The gradient calls launched one right after another, in every form of the kernels, code type and
epilogue: the load, convert and multiply rings run full and out of step, and each call gives the
first one's bits."""
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from test_gpu_grad_gemm import (_assert_close, _call, _codes, _dequantized, _dy, _scales,
                                _silu_reference, _tol)

pytestmark = pytest.mark.gpu

CALLS, REPLAYS = 24, 8

# (M, N, K): up to 128 rows; rows the kernel converts for in tiles of 256 and of 512; a pass ahead
DGRAD = [(16, 28672, 4096), (128, 14336, 4096), (512, 8192, 4096), (4096, 4096, 2048),
         (2048, 12288, 4096)]
SILU = [(16, 4096, 14336), (100, 4104, 4112), (512, 4096, 14336), (4096, 4096, 2048),
        (2048, 8192, 4096), (265, 7880, 4400)]
WGRAD = [(8192, 512, 4096), (8200, 2048, 4112), (2048, 4096, 4096), (777, 1032, 2064)]


def _repeat(call, ref):
    outs = [torch.empty_like(ref) for _ in range(CALLS)]
    for o in outs:
        call(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            call(o)
    for _ in range(REPLAYS):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
    assert w8.w8a8_last_device_status() == 0


@pytest.mark.parametrize("M,N,K", DGRAD)
def test_input_gradient_fp8(M, N, K):
    dy, q, s = _dy(M, N, 60), _codes((N, K), True, 61), _scales(N, 62)
    ref = w8.w8a8_gemm_dgrad_fp8(dy, q, s)
    b = _dequantized(q, s)
    want = dy.double() @ b
    _assert_close(ref, want, _tol(want, dy.double().abs() @ b.abs(), N))
    _repeat(lambda o: w8.w8a8_gemm_dgrad_fp8(dy, q, s, dx=o), ref)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("M,N,K", SILU)
def test_gated_block_backward(M, N, K, f8):
    dy, q, s = _dy(M, N, 63), _codes((N, K), f8, 64), _scales(N, 65)
    g = torch.Generator().manual_seed(66)
    gate_up = (torch.randn(M, 2 * K, generator=g) * 4).bfloat16().cuda()
    fn = _call("w8a8_gemm_dgrad_silu", f8)
    ref = fn(dy, q, s, gate_up)
    _assert_close(ref, *_silu_reference(dy, q, s, gate_up))
    _repeat(lambda o: fn(dy, q, s, gate_up, dgate_up=o), ref)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("M,N,K", WGRAD)
def test_weight_gradient(M, N, K, f8):
    dy, q, s = _dy(M, N, 67), _codes((M, K), f8, 68), _scales(M, 69)
    fn = _call("w8a8_gemm_wgrad", f8)
    ref = fn(dy, q, s)
    b = _dequantized(q, s)
    want = dy.double().t() @ b
    _assert_close(ref, want, _tol(want, dy.double().abs().t() @ b.abs(), M))
    _repeat(lambda o: fn(dy, q, s, dw=o), ref)
