"""The widest matrices that the gradients of a W8A8 linear accept: 2^30 columns (about 20 GB)."""
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1 << 30, (1 << 30) - 16])
def test_weight_gradient_of_the_widest_rows(K):
    """One token, so dw[n, k] = dy[n] s q[k], exact with powers of two; every column is looked at,
    the first ones among them (whose distance to the row's end, in bytes, passes 32 bits)."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
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
    del dw, xq, want
    torch.cuda.empty_cache()
