"""Calls from host threads that have made no CUDA call before, as the threads of PyTorch's backward
pass are."""
import threading

import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from test_gpu_grad_gemm import _codes, _dy, _scales

pytestmark = pytest.mark.gpu

M, N, K = 300, 512, 528


def _calls():
    """Every kind of call that describes its operands to the copy engine."""
    dy, wq, sc = _dy(M, N, 1), _codes((N, K), False, 2), _scales(N, 3)
    xq, st = _codes((M, K), False, 4), _scales(M, 5)
    gate_up = torch.randn(M, 2 * K, device="cuda").bfloat16()
    w8q, x8q = _codes((N, K), True, 6), _codes((M, K), True, 7)
    return {
        "dgrad": lambda: w8.w8a8_gemm_dgrad(dy, wq, sc),
        "dgrad, few rows": lambda: w8.w8a8_gemm_dgrad(dy[:16], wq, sc),
        "dgrad_fp8": lambda: w8.w8a8_gemm_dgrad_fp8(dy, w8q, sc),
        "dgrad_silu": lambda: w8.w8a8_gemm_dgrad_silu(dy, wq, sc, gate_up),
        "wgrad": lambda: w8.w8a8_gemm_wgrad(dy, xq, st),
        "dequant": lambda: w8.w8a8_gemm_dequant(xq, st, wq, sc),
        "dequant, few rows": lambda: w8.w8a8_gemm_dequant(xq[:8], st[:8], wq, sc),
        "dequant_fp8": lambda: w8.w8a8_gemm_dequant_fp8(x8q, st, w8q, sc),
        "norm": lambda: w8.w8a8_sandwich_rmsnorm_quant(dy, dy, sc, 1e-5)[2],
    }


def test_calls_from_new_threads():
    for name, call in _calls().items():
        want = call().clone()
        again = call()  # so that the thread's outputs come from memory that is there already
        del again
        torch.cuda.synchronize()
        got = []

        def work():
            try:
                got.append(call())
                torch.cuda.synchronize()
            except Exception as e:  # noqa: BLE001 (reported by the main thread)
                got.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert isinstance(got[0], torch.Tensor), (name, got[0])
        assert torch.equal(got[0], want), name


class _Linear(torch.autograd.Function):
    """A frozen W8A8 linear whose input has a gradient."""

    @staticmethod
    def forward(ctx, x, wq, sc):
        ctx.save_for_backward(wq, sc)
        q, s = w8.w8a8_quantize_rows(x)
        return w8.w8a8_gemm_dequant(q, s, wq, sc)

    @staticmethod
    def backward(ctx, dy):
        return w8.w8a8_gemm_dgrad(dy.contiguous(), *ctx.saved_tensors), None, None


def test_an_autograd_function_calls_the_gradients():
    wq, sc, dy = _codes((N, K), False, 8), _scales(N, 9), _dy(M, N, 10)
    x = _dy(M, K, 11).requires_grad_()
    for _ in range(2):
        x.grad = None
        _Linear.apply(x, wq, sc).backward(dy)
        assert torch.equal(x.grad, w8.w8a8_gemm_dgrad(dy, wq, sc))
