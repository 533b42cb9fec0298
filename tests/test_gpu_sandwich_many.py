"""The block-boundary norms where a CTA, a team of warps or a cluster takes row after row, and where
sums of squares leave binary32."""
import numpy as np
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
import oracle
from grad_reference import backward
from helpers import assert_rms_rows_match, dev, dev_bf16, host, host_bf16
from test_gpu_sandwich import EPS, EPS_POST, _check, _f, _gate, _h_reference, _inputs

pytestmark = pytest.mark.gpu


# few rows (one row a CTA) and enough of them for one, two and four warps a row
@pytest.mark.parametrize("M,K", [(100, 2048), (100, 4096), (100, 8192), (800, 2048), (400, 4096),
                                 (200, 8192)])
@pytest.mark.parametrize("post", [False, True])
def test_sums_of_squares_beyond_binary32(M, K, post):
    """Values of 2^62 to 2^63: their squares are finite in binary32, a sum of sixteen of them is
    not, and their mean is. The batch's size, which chooses the kernel, makes no difference, and
    the rows around them come out as always."""
    y, res, gs, gp = _inputs(M, K, post, 31)
    rng = np.random.default_rng(K)

    def huge():
        x = rng.uniform(1.0, 2.0, K) * rng.choice([-1.0, 1.0], K) * 2.0 ** 62
        return oracle.f32_to_bf16(x.astype(np.float32))

    for m in (1, M // 2, M - 1):
        y[m] = huge()        # in the first norm, or in h
        res[m - 1] = huge()  # in h
    ref_h = _h_reference(_f(y), _f(res), gp, None, 1.0)
    q, s, h = w8.w8a8_sandwich_rmsnorm_quant(dev_bf16(y), dev_bf16(res), dev(gs), EPS,
                                             gamma_post=None if gp is None else dev(gp),
                                             eps_post=EPS_POST)
    torch.cuda.synchronize()
    assert np.array_equal(host_bf16(h), ref_h)
    assert (host(s) > 0).all()
    assert_rms_rows_match(host(q), host(s), ref_h, gs, EPS)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -45, 2.0 ** -50])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind", ["none", "token"])
def test_backward_of_small_rows_without_eps(scale, post, kind):
    """eps = 0 and rows whose 1 / rms is finite where its cube is not (2^43 and more)."""
    M, K = 9, 1040
    y, h, gs, gp = _inputs(M, K, post, 41)
    y, h = (oracle.f32_to_bf16(_f(t) * np.float32(scale)).reshape(M, K) for t in (y, h))
    gate, dgate = _gate(kind, M, K, 42)
    dz = oracle.f32_to_bf16(np.random.default_rng(1).normal(size=(M, K)).astype(np.float32) * 0.01)
    dz = dz.reshape(M, K)
    got = w8.w8a8_sandwich_rmsnorm_backward(
        dev_bf16(dz), dev_bf16(y), dev_bf16(h), dev(gs), 0.0,
        gamma_post=None if gp is None else dev(gp), gate=dgate)
    d = lambda a: None if a is None else np.asarray(a, dtype=np.float64)  # noqa: E731
    ref = backward(d(_f(dz)), d(_f(y)), d(_f(h)), d(gs), 0.0, gamma_post=d(gp), gate=d(gate))
    n = 128  # roundings on the longest path, as for rows of any size
    _check("dy", _f(host_bf16(got[0])), *ref["dy"], n, True)
    _check("dresidual", _f(host_bf16(got[1])), *ref["dresidual"], n, True)
    _check("dgamma_pre", host(got[2]), *ref["dgamma_pre"], n + M + 136, False)
    if post:
        _check("dgamma_post", host(got[3]), *ref["dgamma_post"], n + M + 136, False)
    if kind == "token":
        _check("dgate", host(got[4]), *ref["dgate"], n + M + 136, False)


def _rows(M, K, seed, std=1.0):
    """bf16 [M, K] on the device, one channel in a hundred fifty times as wide."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda") * std
    wide = torch.rand(K, generator=g, device="cuda") < 0.01
    return (x * torch.where(wide, 50.0, 1.0)).bfloat16()


def _gate_on_device(kind, M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = {"none": None, "token": (M, 1), "channel": (1, K), "full": (M, K)}[kind]
    if shape is None:
        return None
    x = torch.randn(shape, generator=g, device="cuda")
    return x.bfloat16() if kind == "full" else x


def _gain(K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.1 * torch.randn(K, generator=g, device="cuda")


def _replayed(call, want, before=lambda: None):
    """Six calls of a graph, replayed three times, each with the first call's bits."""
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        outs = [call(i) for i in range(6)]
    for _ in range(3):
        before()
        g.replay()
        for o in outs:
            for a, b in zip(o, want):
                assert b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert w8.w8a8_last_device_status() == 0


KINDS = [("none", False, False), ("none", True, True), ("token", True, False),
         ("channel", False, True), ("channel", True, False), ("full", True, True),
         ("full", False, False)]


# one, two and four warps a row, with up to sixteen, eight and four rows of an SM at a time, three
# rows and more each; then one row a CTA with more rows than resident CTAs (narrow rows of few
# values in all; rows of more than 8192)
@pytest.mark.parametrize("M,K", [(100003, 16), (33001, 48), (8003, 208), (2501, 2064), (1301, 4112), (1301, 8192),
                                 (20011, 64), (5501, 272), (761, 2064), (601, 14336),
                                 (301, 32768)])
@pytest.mark.parametrize("kind,post,f8", KINDS)
def test_forward_row_after_row(M, K, kind, post, f8):
    y, res, gs = _rows(M, K, 51), _rows(M, K, 52), _gain(K, 53)
    gp = _gain(K, 54) if post else None
    gate = _gate_on_device(kind, M, K, 55)
    fn = w8.w8a8_sandwich_rmsnorm_quant_fp8 if f8 else w8.w8a8_sandwich_rmsnorm_quant

    def call(r, **kw):
        return fn(y, r, gs, EPS, gamma_post=gp, eps_post=EPS_POST, gate=gate, res_scale=0.75, **kw)

    q, s, h = call(res)
    # against the oracle on some of the rows, the first and the last among them
    some = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 96)])
    at = torch.from_numpy(some).cuda()
    hg = None
    if gate is not None:
        hg = gate if kind == "channel" else gate[at]
        hg = host(hg.float())
    ref_h = _h_reference(_f(host_bf16(y[at])), _f(host_bf16(res[at])),
                         None if gp is None else host(gp), hg, 0.75)
    assert np.array_equal(host_bf16(h[at]), ref_h)
    assert_rms_rows_match(host(q.view(torch.uint8)[at] if f8 else q[at]), host(s[at]), ref_h,
                          host(gs), EPS, ref_fn=oracle.smooth_rmsnorm_quant_fp8 if f8 else
                          oracle.smooth_rmsnorm_quant)
    # one call right after another, each in place on a residual of its own: all rows, bit for bit
    places = [res.clone() for _ in range(6)]
    _replayed(lambda i: call(places[i], h_out=places[i]), (q, s, h),
              lambda: [p.copy_(res) for p in places])


# clusters of two, three and four CTAs (the last one with fewer columns), and one CTA: three rows
# and more each
@pytest.mark.parametrize("M,K", [(250, 8208), (160, 16400), (120, 24592), (1500, 1040)])
@pytest.mark.parametrize("kind,post,with_dh", KINDS)
def test_backward_row_after_row(M, K, kind, post, with_dh):
    y, h, gs = _rows(M, K, 61), _rows(M, K, 62), _gain(K, 63)
    gp = _gain(K, 64) if post else None
    gate = _gate_on_device(kind, M, K, 65)
    dz = _rows(M, K, 66, 0.01)
    dh = _rows(M, K, 67, 0.01) if with_dh else None

    def call(_):
        return w8.w8a8_sandwich_rmsnorm_backward(dz, y, h, gs, EPS, dh=dh, gamma_post=gp,
                                                 eps_post=EPS_POST, gate=gate, res_scale=0.75)

    got = call(0)
    d = lambda t: None if t is None else host(t.double())  # noqa: E731
    ref = backward(d(dz), d(y), d(h), d(gs), EPS, dh=d(dh), gamma_post=d(gp), eps_post=EPS_POST,
                   gate=d(gate), res_scale=0.75)
    # a row sum adds 8 values in a thread, then over 32 lanes, up to 32 warps and 4 CTAs (8 + 5 + 5
    # + 4 additions), twice in a row for dy, with the factors around them: below 128; a sum over the
    # tokens adds at most one for each of a CTA's rows and each part of a lane: below M, and 136
    n, tokens = 128, 128 + M + 136
    _check("dy", d(got[0]), *ref["dy"], n, True)
    _check("dresidual", d(got[1]), *ref["dresidual"], n, True)
    _check("dgamma_pre", host(got[2]), *ref["dgamma_pre"], tokens, False)
    if post:
        _check("dgamma_post", host(got[3]), *ref["dgamma_post"], tokens, False)
    if kind != "none":
        _check("dgate", d(got[4]), *ref["dgate"], n if kind == "full" else tokens, kind == "full")
    _replayed(call, got)
