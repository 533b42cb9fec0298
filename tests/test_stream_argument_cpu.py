"""The stream argument of the gradient calls and block-boundary norms, as the other calls have it."""
import inspect

import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8

CALLS = ["w8a8_sandwich_rmsnorm_quant", "w8a8_sandwich_rmsnorm_quant_fp8",
         "w8a8_sandwich_rmsnorm_backward", "w8a8_gemm_dgrad", "w8a8_gemm_dgrad_fp8",
         "w8a8_gemm_dgrad_silu", "w8a8_gemm_dgrad_silu_fp8", "w8a8_gemm_wgrad",
         "w8a8_gemm_wgrad_fp8"]


@pytest.mark.parametrize("name", CALLS + ["w8a8_gemm_dequant", "w8a8_silu_mul_quant"])
def test_stream_is_the_last_parameter(name):
    last = list(inspect.signature(getattr(w8, name)).parameters.values())[-1]
    assert last.name == "stream" and last.default is None


@pytest.mark.parametrize("name", CALLS)
def test_stream_by_position_and_by_name(name):
    """Taken either way (the call then refuses the CPU tensor), but not both."""
    fn = getattr(w8, name)
    args = [None] * len(inspect.signature(fn).parameters)
    args[0] = torch.zeros(4, 64, dtype=torch.bfloat16)
    if "gate_up" in inspect.signature(fn).parameters:
        args[3] = args[0]
    stream = object()
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args[:-1], stream)
    with pytest.raises(ValueError, match="CUDA"):
        fn(*args[:-1], stream=stream)
    with pytest.raises(TypeError, match="multiple values"):
        fn(*args[:-1], stream, stream=stream)
    with pytest.raises(TypeError):
        fn(*args, stream)
