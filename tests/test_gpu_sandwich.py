"""Parity of the block-boundary norms: h bit for bit against the formula's binary32 operations,
codes and scales against the oracle's RMSNorm + quantization of that h, and the backward pass
against the binary64 formula within the bound that its magnitudes give."""
import numpy as np
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
import oracle
from int8_w8a8_quantized_smoothed_b200 import synth
from grad_reference import HALF_BF16, U, backward
from helpers import (assert_rms_rows_match, bf16_out, dev, dev_bf16, f32_out, host, host_bf16,
                     i8_out)

pytestmark = pytest.mark.gpu

EPS, EPS_POST = 1e-5, 1e-3
SHAPES = [(1, 16), (1, 4096), (3, 48), (37, 4096), (5, 8192), (7, 4112), (33, 1040), (2, 14336),
          (2, 32768), (700, 272)]
# enough values for the kernel in which one, two or four warps share a row
MANY = [(1600, 1040), (400, 4096), (400, 4112)]
GATES = ["none", "token", "channel", "full"]


def _gate(kind, M, K, seed):
    """(numpy values for the formula, device tensor)."""
    rng = np.random.default_rng(seed)
    if kind == "none":
        return None, None
    shape = {"token": (M, 1), "channel": (1, K), "full": (M, K)}[kind]
    g = rng.normal(size=shape).astype(np.float32)
    if kind != "full":
        return g, dev(g)
    b = oracle.f32_to_bf16(g).reshape(shape)
    return oracle.bf16_to_f32(b).reshape(shape), dev_bf16(b)


def _rstd32(x, eps):
    """1 / sqrt(ms + eps) in binary32, ms the mean of squares summed with 64 bits and rounded."""
    ms = (x.astype(np.float64) ** 2).astype(np.longdouble).sum(axis=1) / x.shape[1]
    return np.float32(1.0) / np.sqrt(ms.astype(np.float32) + np.float32(eps))


def _h_reference(y, res, gp, gate, rs):
    v = y
    if gp is not None:
        v = (y * _rstd32(y, EPS_POST)[:, None]) * gp
    if gate is not None:
        v = gate * v
    h = np.float32(rs) * res + v
    return oracle.f32_to_bf16(h.astype(np.float32)).reshape(h.shape)


def _inputs(M, K, post, seed):
    y, res = synth.activation(M, K, seed), synth.activation(M, K, seed + 1)
    gs = synth.gamma(K, seed + 2).astype(np.float32)
    gp = synth.gamma(K, seed + 3).astype(np.float32) if post else None
    return y, res, gs, gp


def _f(b):
    return oracle.bf16_to_f32(b).reshape(b.shape)


@pytest.mark.parametrize("M,K", SHAPES + MANY)
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("f8", [False, True])
def test_forward_matches_oracle(M, K, kind, post, f8):
    y, res, gs, gp = _inputs(M, K, post, seed=5 * M + K)
    gate, dgate = _gate(kind, M, K, M + K)
    rs = 0.75
    ref_h = _h_reference(_f(y), _f(res), gp, gate, rs)
    h, ch = bf16_out((M, K))
    s, cs = f32_out((M,))
    kw = dict(gamma_post=None if gp is None else dev(gp), eps_post=EPS_POST, gate=dgate,
              res_scale=rs, h_out=h, s_tok=s)
    if f8:
        q, _, _ = w8.w8a8_sandwich_rmsnorm_quant_fp8(dev_bf16(y), dev_bf16(res), dev(gs), EPS, **kw)
        cq = lambda: None  # noqa: E731
        q = q.view(torch.uint8)
    else:
        q, cq = i8_out((M, K))
        w8.w8a8_sandwich_rmsnorm_quant(dev_bf16(y), dev_bf16(res), dev(gs), EPS, q=q, **kw)
    torch.cuda.synchronize()
    ch(); cs(); cq()
    assert np.array_equal(host_bf16(h), ref_h)
    assert_rms_rows_match(host(q), host(s), ref_h, gs, EPS,
                          ref_fn=oracle.smooth_rmsnorm_quant_fp8 if f8 else
                          oracle.smooth_rmsnorm_quant)


@pytest.mark.parametrize("M,K", [(6, 512), (900, 2048)])
def test_forward_in_place_and_zero_rows(M, K):
    y, res, gs, gp = _inputs(M, K, True, 3)
    y[2] = 0
    res[2] = 0   # nothing in the row: h = 0, s = 0, every code 0
    y[4] = 0     # nothing from the block: h is the residual
    r = dev_bf16(res)
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(dev_bf16(y), r, dev(gs), 0.0, gamma_post=dev(gp),
                                             eps_post=EPS_POST, h_out=r)
    torch.cuda.synchronize()
    assert h.data_ptr() == r.data_ptr()
    ref = _h_reference(_f(y), _f(res), gp, None, 1.0)
    got = host_bf16(h)
    assert np.array_equal(np.delete(got, 2, 0), np.delete(ref, 2, 0))
    assert np.array_equal(_f(got[4]), _f(res[4]))
    assert not _f(got[2]).any()


def test_forward_zero_row_with_eps():
    y = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(y, y.clone(), torch.ones(64, device="cuda"), EPS,
                                             gamma_post=torch.ones(64, device="cuda"))
    assert not host(q).any() and not host(s).any() and not h.any()


@pytest.mark.parametrize("M,K", [(40, 4096), (500, 4096)])
def test_forward_without_extras_equals_the_residual_norm(M, K):
    """No post norm, no gate, scale 1: the residual form of w8a8_smooth_rmsnorm_quant."""
    y, res, gs, _ = _inputs(M, K, False, 11)
    q0, s0, h0 = w8.w8a8_smooth_rmsnorm_quant(dev_bf16(y), dev(gs), EPS, residual=dev_bf16(res))
    q1, s1, h1 = w8.w8a8_sandwich_rmsnorm_quant(dev_bf16(y), dev_bf16(res), dev(gs), EPS)
    assert torch.equal(h0.view(torch.int16), h1.view(torch.int16))
    assert torch.equal(q0, q1) and torch.equal(s0, s1)


def _check(name, got, ref, mag, roundings, stored_bf16):
    """|got - ref| <= roundings U magnitude, and half a bf16 step of the stored value."""
    err = np.abs(got.astype(np.float64) - ref)
    tol = roundings * U * mag
    if stored_bf16:
        tol = tol + HALF_BF16 * (np.abs(ref) + tol) + 2.0 ** -133
    bad = err > tol
    assert not bad.any(), (name, int(bad.sum()), float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("M,K", SHAPES + [(700, 4096), (150, 8192)])
@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_matches_formula(M, K, kind, post, with_dh):
    y, h, gs, gp = _inputs(M, K, post, seed=3 * M + K)
    gate, dgate = _gate(kind, M, K, M + K + 1)
    dz = synth.normal_bf16((M, K), M + 2, std=0.01)
    dh = synth.normal_bf16((M, K), M + 3, std=0.01) if with_dh else None
    dy, cdy = bf16_out((M, K))
    dr, cdr = bf16_out((M, K))
    got = w8.w8a8_sandwich_rmsnorm_backward(
        dev_bf16(dz), dev_bf16(y), dev_bf16(h), dev(gs), EPS,
        dh=None if dh is None else dev_bf16(dh), gamma_post=None if gp is None else dev(gp),
        eps_post=EPS_POST, gate=dgate, res_scale=0.75, dy=dy, dresidual=dr)
    torch.cuda.synchronize()
    cdy(); cdr()
    d = lambda a: None if a is None else np.asarray(a, dtype=np.float64)  # noqa: E731
    ref = backward(d(_f(dz)), d(_f(y)), d(_f(h)), d(gs), EPS, dh=None if dh is None else d(_f(dh)),
                   gamma_post=d(gp), eps_post=EPS_POST, gate=d(gate), res_scale=0.75)
    # roundings on the longest path to a value: a row sum adds 8 values in a thread, then over 32
    # lanes, 16 warps and 8 CTAs (8 + 5 + 8 + 5 < 32 of them), twice in a row for dy (the sums of
    # D use the first ones), with the factors around them: below 128; a sum over the tokens adds
    # at most one for each of a CTA's rows and each of at most 1024 / 8 + 8 parts
    n = 128
    _check("dy", _f(host_bf16(got[0])), *ref["dy"], n, True)
    _check("dresidual", _f(host_bf16(got[1])), *ref["dresidual"], n, True)
    _check("dgamma_pre", host(got[2]), *ref["dgamma_pre"], n + M + 136, False)
    if post:
        _check("dgamma_post", host(got[3]), *ref["dgamma_post"], n + M + 136, False)
    else:
        assert got[3] is None
    if kind == "none":
        assert got[4] is None
    elif kind == "full":
        _check("dgate", _f(host_bf16(got[4])), *ref["dgate"], n, True)
    else:
        _check("dgate", host(got[4]), *ref["dgate"], n + M + 136, False)


def test_backward_in_place_repeatable_and_replayed():
    """dresidual on dh, the same bits on every call, and a captured call replayed on new inputs."""
    M, K = 300, 4096
    mk = lambda seed: [dev_bf16(synth.normal_bf16((M, K), seed + i)) for i in range(4)]  # noqa: E731
    gs, gp = dev(synth.gamma(K, 1).astype(np.float32)), dev(synth.gamma(K, 2).astype(np.float32))
    gate = torch.rand(M, 1, device="cuda")

    def call(t, **kw):
        dz, dh, y, h = t
        return w8.w8a8_sandwich_rmsnorm_backward(dz, y, h, gs, EPS, dh=dh, gamma_post=gp,
                                                 gate=gate, **kw)

    a, b = mk(0), mk(50)
    first, other = call(a), call(b)
    again = call(a)
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    t = [x.clone() for x in a]
    placed = call(t, dresidual=t[1])
    assert placed[1].data_ptr() == t[1].data_ptr()
    for x, y in zip(first, placed):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    static = [x.clone() for x in a]
    with torch.cuda.stream(side):
        call(static)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(static)
    for x, y in zip(static, b):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(other, out):
        assert torch.equal(x, y)


def test_on_another_stream():
    M, K = 64, 4096
    y, res, gs, gp = _inputs(M, K, True, 21)
    args = (dev_bf16(y), dev_bf16(res), dev(gs), EPS)
    want = w8.w8a8_sandwich_rmsnorm_quant(*args, gamma_post=dev(gp))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = w8.w8a8_sandwich_rmsnorm_quant(*args, gamma_post=dev(gp), stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_argument_errors():
    K = 64
    y = torch.zeros(4, K, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(K, device="cuda")
    with pytest.raises(W8Error, match="INVALID_ARG"):
        w8.w8a8_sandwich_rmsnorm_quant(y, y.clone(), g, EPS, h_out=y)
    with pytest.raises(W8Error, match="INVALID_ARG"):
        w8.w8a8_sandwich_rmsnorm_quant(y, y.clone(), g, EPS, res_scale=float("nan"))
    with pytest.raises(ValueError, match="gate must be"):
        w8.w8a8_sandwich_rmsnorm_quant(y, y.clone(), g, EPS, gate=g)
    with pytest.raises(ValueError, match="shape"):
        w8.w8a8_sandwich_rmsnorm_quant(y, y[:2].clone(), g, EPS)
    with pytest.raises(W8Error, match="WORKSPACE"):
        w8.w8a8_sandwich_rmsnorm_backward(y, y.clone(), y.clone(), g, EPS,
                                          workspace=torch.empty(64, dtype=torch.uint8,
                                                                device="cuda"))


W8Error = w8.W8A8Error
