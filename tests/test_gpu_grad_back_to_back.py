"""The gradient calls launched one right after another, in every form of the kernels, code type and
epilogue: the load, convert and multiply rings run full and out of step, and each call gives the
first one's bits."""
import threading

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


def _step(t, stream=None):
    """A linear's forward call and every gradient around it, one reading the other's output."""
    kw = dict(stream=stream)
    y = w8.w8a8_gemm_dequant(t["xq"], t["st"], t["w"], t["sc"], workspace=t["ws"], **kw)
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(y, t["res"], t["g"], 1e-5, gamma_post=t["g"], **kw)
    b = w8.w8a8_sandwich_rmsnorm_backward(t["res"], y, h, t["g"], 1e-5, gamma_post=t["g"],
                                          workspace=t["ws"], **kw)
    dw = w8.w8a8_gemm_wgrad(b[0], t["xq"], t["st"], workspace=t["ws"], **kw)
    dx = w8.w8a8_gemm_dgrad(b[0], t["w"], t["sc"], workspace=t["ws"], **kw)
    dgu = w8.w8a8_gemm_dgrad_silu(dx, t["w2"], t["sc2"], t["gate_up"], workspace=t["ws"], **kw)
    return [y, q, s, h, *b[:4], dw, dx, dgu]


def _step_inputs(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def values(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    return dict(xq=_codes((M, K), False, seed), st=_scales(M, seed + 1),
                w=_codes((N, K), False, seed + 2), sc=_scales(N, seed + 3),
                w2=_codes((K, 1040), False, seed + 4), sc2=_scales(K, seed + 5),
                res=values(M, N), gate_up=values(M, 2 * 1040),
                g=1 + 0.1 * torch.randn(N, generator=g, device="cuda"), ws=w8.Workspace())


@pytest.mark.parametrize("M,N,K", [(16, 4096, 4096), (300, 4096, 4112)])
def test_overlap_modes_give_the_same_bits(M, N, K):
    t = _step_inputs(M, N, K, 70)
    want = [x.clone() for x in _step(t)]
    before = w8.w8a8_get_overlap()
    try:
        for mode in (0, 1, 2):
            w8.w8a8_set_overlap(mode)
            for _ in range(10):
                got = _step(t)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), mode
    finally:
        w8.w8a8_set_overlap(before)
    assert w8.w8a8_last_device_status() == 0


def test_two_threads_on_their_own_streams():
    """Calls at once from two threads, each with its inputs, stream and workspace."""
    sets = [_step_inputs(16, 4096, 4096, 80), _step_inputs(300, 4096, 4112, 90)]
    want = [[x.clone() for x in _step(t)] for t in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(t, ref):
        try:
            stream = torch.cuda.Stream()
            for i in range(40):
                got = _step(t, stream)
                if i % 8 == 0:
                    stream.synchronize()
                    wrong.extend(k for k, (a, b) in enumerate(zip(got, ref)) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(sets, want)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert w8.w8a8_last_device_status() == 0
