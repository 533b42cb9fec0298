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
