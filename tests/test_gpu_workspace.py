"""One Workspace through a whole tuning step: GEMMs that need its flag words zero, and gradients
that leave any contents behind, in turn."""
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from int8_w8a8_quantized_smoothed_b200 import prep

pytestmark = pytest.mark.gpu

M, H, I = 16, 4096, 2048


def _inputs():
    g = torch.Generator().manual_seed(5)

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()

    def scales(n):
        return (torch.rand(n, generator=g) * 1e-3 + 1e-4).cuda()

    def values(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()

    return dict(xq=codes(M, H), st=scales(M), w=codes(H, H), sc=scales(H), gu=codes(2 * I, H),
                sgu=scales(2 * I), down=codes(H, I), sd=scales(H), res=values(M, H),
                dy=values(M, H), gate_up=values(M, 2 * I), gamma=torch.ones(H).cuda())


def _forward(t, ws):
    """Every kind of call that counts on the flag words."""
    il = prep.interleave_gate_up(t["gu"], t["sgu"])
    y = w8.w8a8_gemm_dequant_ex(t["xq"], t["st"], t["w"], t["sc"], variant=2, workspace=ws)
    a = w8.w8a8_gemm_silu_quant(t["xq"], t["st"], *il, workspace=ws)
    n = w8.w8a8_gemm_rmsnorm_quant(t["xq"], t["st"], t["w"], t["sc"], t["res"], t["gamma"], 1e-5,
                                   workspace=ws, one_launch=True)
    return [y, *a, *n]


def _gradients(t, ws):
    """Every kind of call that leaves its partial results behind."""
    dx = w8.w8a8_gemm_dgrad(t["dy"], t["w"], t["sc"], workspace=ws)
    dgu = w8.w8a8_gemm_dgrad_silu(t["dy"], t["down"], t["sd"], t["gate_up"], workspace=ws)
    dw = w8.w8a8_gemm_wgrad(t["dy"], t["xq"], t["st"], workspace=ws)
    b = w8.w8a8_sandwich_rmsnorm_backward(t["dy"], t["res"], t["res"], t["gamma"], 1e-5,
                                          gamma_post=t["gamma"], workspace=ws)
    return [dx, dgu, dw, *b[:4]]


def test_one_workspace_serves_forward_and_gradient_calls():
    assert w8.w8a8_gemm_workspace_size_ex(M, H, H, 2) > 0
    assert w8.w8a8_gemm_dgrad_workspace_size(M, H, H) > 0
    t = _inputs()
    want_f, want_g = _forward(t, w8.Workspace()), _gradients(t, None)
    ws = w8.Workspace()
    for _ in range(3):
        for got, want in zip(_gradients(t, ws), want_g):
            assert torch.equal(got, want)
        for got, want in zip(_forward(t, ws), want_f):
            assert torch.equal(got, want)
    assert w8.w8a8_last_device_status() == 0


def test_stream_by_position():
    t = _inputs()
    want = w8.w8a8_gemm_dgrad(t["dy"], t["w"], t["sc"])
    wq, ws, wh = w8.w8a8_sandwich_rmsnorm_quant(t["dy"], t["res"], t["gamma"], 1e-5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = w8.w8a8_gemm_dgrad(t["dy"], t["w"], t["sc"], None, None, side)
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(t["dy"], t["res"], t["gamma"], 1e-5, None, None, None,
                                             1.0, None, None, None, side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(q, wq) and torch.equal(h, wh)
    assert torch.equal(s, ws)
