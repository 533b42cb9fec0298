"""The gradients of a W8A8 linear and of the gated feed-forward block against their formulas in
binary64.

The dequantized operand is reproduced exactly (the scale as two bf16 parts, bf16(q hi + bf16(q
lo))), so the only differences are the tensor cores' binary32 additions and the output's rounding. A k = 16 instruction adds its sixteen exact products to the accumulator
with an error of at most one unit in the last place of the largest partial sum, 2^-23 of
sum |products|; over R terms R / 16 + 1 instructions, and up to 74 parts of a split sum."""
import numpy as np
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from int8_w8a8_quantized_smoothed_b200 import synth
from grad_reference import HALF_BF16
from helpers import bf16_out

pytestmark = pytest.mark.gpu

# (M, N, K): single tokens, the smallest sides, sides that end inside a tile and inside a k-block,
# sums split over the SMs (few tiles), whole waves of tiles with and without a remainder; rows that
# the kernel dequantizes itself, in tiles of 256 and of 512 of them, and that a pass before it does
# (4096 and more, sums of fewer than 8192)
SHAPES = [(1, 8, 16), (1, 4096, 4096), (16, 6144, 512), (3, 72, 48), (64, 64, 64), (65, 56, 272),
          (300, 264, 528), (257, 1032, 4112), (2304, 512, 2304), (2304, 1024, 2304),
          (1000, 2056, 1040), (129, 14336, 256), (4100, 264, 528), (4100, 8200, 272),
          (33, 4104, 4112), (100, 6144, 528), (128, 1000, 2064), (20, 640, 19072),
          (769, 8200, 4112), (265, 7880, 4400), (263, 7576, 4416), (1309, 2504, 4112),
          (3345, 2568, 4432), (3139, 10256, 528), (1282, 3976, 4656), (2570, 1312, 4112),
          (2499, 3176, 4640)]


def _codes(shape, f8, seed):
    q = torch.from_numpy(synth.int8_codes(shape, seed)).cuda()
    if not f8:
        return q
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=g) * 60).clamp(-448, 448)
    return x.cuda().to(w8.FP8)


def _round_bf16(x):
    """Binary64 values rounded to eight significant bits, ties to even, in one step."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e - 8)


def _dequantized(q, s):
    """The bf16 operand s q as the kernels form it, in binary64: q hi + bf16(q lo), rounded."""
    hi = s.bfloat16().float()
    lo = (s - hi).bfloat16().float()
    v = q.float().double()
    return _round_bf16(v * hi.double()[:, None] + _round_bf16(v * lo.double()[:, None]))


def _dy(M, N, seed):
    return torch.from_numpy(synth.normal_bf16((M, N), seed, std=0.05).view(np.int16)).view(
        torch.bfloat16).cuda()


def _scales(n, seed):
    return torch.from_numpy(synth.scales(n, seed, 1e-4, 1e-2)).cuda()


def _tol(ref, mag, R):
    acc = (R / 16 + 1 + 74) * 2.0 ** -23 * mag
    return acc + HALF_BF16 * (ref.abs() + acc) + 2.0 ** -133


def _assert_close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def _call(name, f8):
    return getattr(w8, name + ("_fp8" if f8 else ""))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_input_gradient(M, N, K, f8):
    dy, q, s = _dy(M, N, 1), _codes((N, K), f8, 2), _scales(N, 3)
    dx, check = bf16_out((M, K))
    _call("w8a8_gemm_dgrad", f8)(dy, q, s, dx=dx)
    torch.cuda.synchronize()
    check()
    assert w8.w8a8_last_device_status() == 0
    b = _dequantized(q, s)
    ref = dy.double() @ b
    _assert_close(dx, ref, _tol(ref, dy.double().abs() @ b.abs(), N))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES + [(63, 520, 528), (2000, 264, 272)])
def test_weight_gradient(M, N, K, f8):
    dy, q, s = _dy(M, N, 4), _codes((M, K), f8, 5), _scales(M, 6)
    dw, check = bf16_out((N, K))
    _call("w8a8_gemm_wgrad", f8)(dy, q, s, dw=dw)
    torch.cuda.synchronize()
    check()
    assert w8.w8a8_last_device_status() == 0
    b = _dequantized(q, s)
    ref = dy.double().t() @ b
    _assert_close(dw, ref, _tol(ref, dy.double().abs().t() @ b.abs(), M))


def _silu_reference(dy, q, s, gate_up):
    b = _dequantized(q, s)
    I = b.shape[1]
    da, mag = dy.double() @ b, dy.double().abs() @ b.abs()
    g, u = gate_up.double()[:, :I], gate_up.double()[:, I:]
    e = torch.exp(-g.abs())
    sig = torch.where(g >= 0, 1 / (1 + e), e / (1 + e))
    rest = torch.where(g >= 0, e / (1 + e), 1 / (1 + e))
    acc = (dy.shape[1] / 16 + 1 + 74) * 2.0 ** -23 * mag
    ref = torch.cat([da * u * sig * (1 + g * rest), da * g * sig], 1)
    # binary32 evaluation: exp of -|g| is within 2^-21 + |g| 2^-23 relative (its argument is
    # rounded once), the logistic function's two halves and the products around them add less than
    # 16 roundings more; 1 + g (1 - sig) is taken with absolute values, as it can cancel
    rel = 2.0 ** -19 + g.abs() * 2.0 ** -22
    size = torch.cat([u.abs() * sig * (1 + g.abs() * rest), g.abs() * sig], 1)
    err = torch.cat([acc + rel * (da.abs() + acc)] * 2, 1) * size
    return ref, err + HALF_BF16 * (ref.abs() + err) + 2.0 ** -133


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated_block_backward(M, N, K, f8):
    dy, q, s = _dy(M, N, 7), _codes((N, K), f8, 8), _scales(N, 9)
    gate_up = (torch.randn(M, 2 * K, generator=torch.Generator().manual_seed(10)) * 4).bfloat16()
    gate_up[0, :4] = torch.tensor([-200.0, 200.0, 0.0, -88.5])  # exp overflow and underflow
    gate_up = gate_up.cuda()
    out, check = bf16_out((M, 2 * K))
    _call("w8a8_gemm_dgrad_silu", f8)(dy, q, s, gate_up, dgate_up=out)
    torch.cuda.synchronize()
    check()
    assert w8.w8a8_last_device_status() == 0
    _assert_close(out, *_silu_reference(dy, q, s, gate_up))


def test_against_the_unrounded_definition():
    """The operand's own rounding included: at most 2^-8 of each product, and 2^-15 before it."""
    M, N, K = 200, 1024, 512
    dy, q, s = _dy(M, N, 11), _codes((N, K), False, 12), _scales(N, 13)
    b = q.double() * s.double()[:, None]
    ref, mag = dy.double() @ b, dy.double().abs() @ b.abs()
    tol = _tol(ref, mag, N) + (2.0 ** -8 + 2.0 ** -15) * mag
    _assert_close(w8.w8a8_gemm_dgrad(dy, q, s), ref, tol)


def test_extreme_codes_and_zero_scales():
    """Every int8 value as a code, rows with scale 0, a whole dy row of zeros."""
    N, K = 256, 256
    q = torch.arange(-128, 128, dtype=torch.int8, device="cuda").repeat(N, 1).contiguous()
    s = torch.full((N,), 0.5, device="cuda")  # exact: dx is sum of small integers / 2
    s[10] = 0.0
    dy = torch.zeros(2, N, dtype=torch.bfloat16, device="cuda")
    dy[0, 3], dy[0, 10] = 1.0, 7.0
    got = w8.w8a8_gemm_dgrad(dy, q, s)
    assert torch.equal(got[0].float(), torch.arange(-128, 128, device="cuda") * 0.5)
    assert not got[1].any()
    # every finite E4M3 value, subnormals among them, times a power of two
    codes = torch.arange(256, device="cuda").to(torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0  # NaN
    q8 = codes.view(w8.FP8).repeat(N, 1).contiguous()
    got = w8.w8a8_gemm_dgrad_fp8(dy, q8, s)
    assert torch.equal(got[0].float(), codes.view(w8.FP8).float() * 0.5)


@pytest.mark.parametrize("name,M,N,K", [("dgrad", 16, 256, 272), ("dgrad", 200, 256, 272),
                                        ("dgrad", 4100, 256, 272), ("wgrad", 64, 256, 272)])
def test_a_broken_scale_or_gradient_is_not_hidden(name, M, N, K):
    """A NaN (any payload) or infinite scale makes NaN of every sum it is in, in each form of the
    kernel; a NaN in dy of its own row's sums only."""
    rows = M if name == "wgrad" else N
    fn = getattr(w8, "w8a8_gemm_" + name)
    dy, q, s = _dy(M, N, 50), _codes((rows, K), False, 51), _scales(rows, 52)
    for bits in (0x7FFFFFFF, 0x7FC00000, -1, 0x7F800000):
        bad = s.clone()
        bad.view(torch.int32)[7] = bits
        assert fn(dy, q, bad).isnan().all()
    dy[3, 5] = float("nan")
    got = fn(dy, q, s).isnan()
    hit = 5 if name == "wgrad" else 3
    assert got[hit].all() and int(got.sum()) == K


@pytest.mark.parametrize("name,M,N,K", [("dgrad", 40, 4096, 512), ("wgrad", 2100, 264, 272),
                                        ("dgrad_silu", 40, 4096, 512),
                                        ("dgrad_silu", 4100, 8200, 272),
                                        ("dgrad_silu", 4100, 8184, 272),
                                        ("dgrad", 265, 7880, 4400), ("dgrad_silu", 3139, 10256, 528),
                                        ("dgrad", 300, 4096, 512)])
def test_repeatable_streams_and_graphs(name, M, N, K):
    """The same bits on every call (split sums included), on a side stream, with the caller's
    workspace, and from a captured call replayed on new inputs beside another capture."""
    rows = M if name == "wgrad" else N
    fn = getattr(w8, "w8a8_gemm_" + name)

    def inputs(seed):
        t = [_dy(M, N, seed), _codes((rows, K), False, seed + 1), _scales(rows, seed + 2)]
        if name == "dgrad_silu":
            t.append(torch.randn(M, 2 * K, device="cuda").bfloat16())
        return t

    a, b = inputs(20), inputs(30)
    first, other = fn(*a), fn(*b)
    torch.cuda.synchronize()
    assert torch.equal(fn(*a), first)
    size = getattr(w8, f"w8a8_gemm_{name.replace('_silu', '')}_workspace_size")(M, N, K)
    assert size > 0  # the shapes are split
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # any contents: NaN here
    assert torch.equal(fn(*a, workspace=ws), first)
    with pytest.raises(w8.W8A8Error, match="WORKSPACE"):
        fn(*a, workspace=ws[:size - 16].contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = fn(*a, stream=side)
    side.synchronize()
    assert torch.equal(x, first)
    static = [[t.clone() for t in a] for _ in range(2)]
    graphs, outs = [], []
    for st in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fn(*st))
        graphs.append(g)
    for x, y in zip(static[1], b):
        x.copy_(y)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], other)


@pytest.mark.parametrize("M,N,K", [(16, 28672, 4096), (128, 14336, 4096), (512, 8192, 4096),
                                   (4096, 4096, 2048), (2048, 12288, 4096)])
def test_many_calls_back_to_back(M, N, K):
    """Long sums, one launch right after another (from a graph too): every form's load, convert
    and multiply rings run full and out of step, and each call gives the first one's bits."""
    dy, q, s = _dy(M, N, 40), _codes((N, K), False, 41), _scales(N, 42)
    ref = w8.w8a8_gemm_dgrad(dy, q, s)
    b = _dequantized(q, s)
    want = dy.double() @ b
    _assert_close(ref, want, _tol(want, dy.double().abs() @ b.abs(), N))
    outs = [torch.empty_like(ref) for _ in range(25)]
    for o in outs:
        w8.w8a8_gemm_dgrad(dy, q, s, dx=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            w8.w8a8_gemm_dgrad(dy, q, s, dx=o)
    for _ in range(4):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
    assert w8.w8a8_last_device_status() == 0


def test_gradients_through_a_gated_block_match_the_formula():
    """The run a tuning step makes: forward codes by the row kernels and the GEMM, then the norms
    after the block, and every gradient back to the block's input and its weights."""
    M, H, I = 96, 512, 1024
    gen = torch.Generator().manual_seed(3)
    eps = 1e-5
    x = torch.randn(M, H, generator=gen).bfloat16().cuda()
    res = torch.randn(M, H, generator=gen).bfloat16().cuda()
    gamma, gpost = (1 + 0.1 * torch.randn(2, H, generator=gen)).cuda()
    wgu = (torch.randn(2 * I, H, generator=gen) * 0.05).bfloat16().cuda()
    wdn = (torch.randn(H, I, generator=gen) * 0.05).bfloat16().cuda()
    (qgu, sgu), (qdn, sdn) = w8.w8a8_quantize_rows(wgu), w8.w8a8_quantize_rows(wdn)
    q3, s3 = w8.w8a8_smooth_rmsnorm_quant(x, gamma, eps)
    gate_up = w8.w8a8_gemm_dequant(q3, s3, qgu, sgu)
    q4, s4 = w8.w8a8_silu_mul_quant(gate_up)
    y = w8.w8a8_gemm_dequant(q4, s4, qdn, sdn)
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(y, res, gamma, eps, gamma_post=gpost, res_scale=0.5)
    dz = (torch.randn(M, H, generator=gen) * 0.02).bfloat16().cuda()
    dh = (torch.randn(M, H, generator=gen) * 0.02).bfloat16().cuda()
    dy, dres, dgamma, dgpost, _ = w8.w8a8_sandwich_rmsnorm_backward(
        dz, y, h, gamma, eps, dh=dh, gamma_post=gpost, res_scale=0.5)
    dgu = w8.w8a8_gemm_dgrad_silu(dy, qdn, sdn, gate_up)
    dwdn = w8.w8a8_gemm_wgrad(dy, q4, s4)
    dx3 = w8.w8a8_gemm_dgrad(dgu, qgu, sgu)
    dwgu = w8.w8a8_gemm_wgrad(dgu, q3, s3)
    torch.cuda.synchronize()
    # the same path differentiated in binary64, from the values the forward calls stored
    x3 = (q3.double() * s3.double()[:, None]).requires_grad_()
    wg = (qgu.double() * sgu.double()[:, None]).requires_grad_()
    wd = (qdn.double() * sdn.double()[:, None]).requires_grad_()
    a4 = q4.double() * s4.double()[:, None]
    gu = x3 @ wg.t()
    gu.data.copy_(gate_up.double())
    a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
    a.data.copy_(a4)
    yy = a @ wd.t()
    yy.data.copy_(y.double())
    gp, gm = gpost.double().requires_grad_(), gamma.double().requires_grad_()
    n = yy * torch.rsqrt(yy.square().mean(1, keepdim=True) + eps) * gp
    rr = res.double().requires_grad_()
    hh = 0.5 * rr + n
    hh.data.copy_(h.double())
    z = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + eps) * gm
    (z * dz.double()).sum().add((hh * dh.double()).sum()).backward()
    # each stored gradient and each dequantized operand is rounded to bf16 once: 2^-8 at most and
    # 2^-8 / sqrt(3) in the 2-norm, over at most four such steps in a row that add at most linearly
    for got, want in ((dres, rr.grad), (dgamma, gm.grad), (dgpost, gp.grad), (dwdn, wd.grad),
                      (dx3, x3.grad), (dwgu, wg.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 4 * 2 * HALF_BF16 / 3 ** 0.5, rel


def test_argument_errors():
    dy, q, s = _dy(4, 64, 1), _codes((64, 128), False, 2), _scales(64, 3)
    with pytest.raises(ValueError, match="wq must be"):
        w8.w8a8_gemm_dgrad(_dy(4, 72, 1), q, s)
    with pytest.raises(TypeError, match="int8"):
        w8.w8a8_gemm_dgrad(dy, q.to(torch.float32), s)
    with pytest.raises(ValueError, match="contiguous"):
        w8.w8a8_gemm_dgrad(dy, q.t().contiguous().t(), s)
    with pytest.raises(TypeError, match="gate_up"):
        w8.w8a8_gemm_dgrad_silu(dy, q, s, None)
    with pytest.raises(ValueError, match="gate_up must have shape"):
        w8.w8a8_gemm_dgrad_silu(dy, q, s, torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w8.W8A8Error, match="UNSUPPORTED_SHAPE"):
        w8.w8a8_gemm_dgrad(_dy(4, 12, 1), _codes((12, 128), False, 2), _scales(12, 3))
    with pytest.raises(ValueError, match="xq must be"):
        w8.w8a8_gemm_wgrad(dy, q, s)
