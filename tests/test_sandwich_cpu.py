"""The block-boundary norms without a GPU: the reference gradients against central differences,
and the host checks of w8a8_sandwich_rmsnorm_quant and its backward pass."""
import ctypes as C

import numpy as np
import pytest
import torch

import int8_w8a8_quantized_smoothed_b200 as w8
from int8_w8a8_quantized_smoothed_b200 import build as w8build
from grad_reference import backward, forward, silu_grads


@pytest.fixture(scope="module")
def L():
    w8build.build()
    return w8.lib()


@pytest.mark.parametrize("gate_shape", [None, (3, 1), (1, 16), (3, 16)])
@pytest.mark.parametrize("post", [False, True])
def test_reference_gradients_match_differences(gate_shape, post):
    rng = np.random.default_rng(7)
    M, K, step = 3, 16, 1e-6
    v = dict(y=rng.normal(size=(M, K)), residual=rng.normal(size=(M, K)),
             gamma_pre=rng.normal(size=K))
    if post:
        v["gamma_post"] = rng.normal(size=K)
    if gate_shape:
        v["gate"] = rng.normal(size=gate_shape)
    fixed = dict(eps=1e-2, eps_post=3e-2, res_scale=0.7)
    dz, dh = rng.normal(size=(M, K)), rng.normal(size=(M, K))

    def loss(**kw):
        h, z = forward(**kw, **fixed)
        return (h * dh).sum() + (z * dz).sum()

    h, _ = forward(**v, **fixed)
    args = {k: x for k, x in v.items() if k != "residual"}
    got = backward(dz=dz, h=h, dh=dh, **args, **fixed)
    for name, x in v.items():
        want = np.empty_like(x)
        for i in np.ndindex(*x.shape):
            up, down = x.copy(), x.copy()
            up[i] += step
            down[i] -= step
            want[i] = (loss(**{**v, name: up}) - loss(**{**v, name: down})) / (2 * step)
        # central differences: step^2 times a third derivative of order 100, and cancellation
        # 2^-53 |loss| / step
        assert np.allclose(got["d" + name][0], want, rtol=1e-6, atol=1e-7), name


def test_reference_silu_gradients_match_differences():
    g = np.linspace(-30.0, 30.0, 61)
    u, da, step = np.cos(g), np.sin(g) + 2.0, 1e-5

    def a(g, u):
        return g / (1.0 + np.exp(-g)) * u

    dg, du = silu_grads(da, g, u)
    assert np.allclose(dg, da * (a(g + step, u) - a(g - step, u)) / (2 * step), rtol=1e-7, atol=1e-7)
    assert np.allclose(du, da * (a(g, u + step) - a(g, u - step)) / (2 * step), rtol=1e-7, atol=1e-7)
    big = silu_grads(np.ones(2), np.array([-1e4, 1e4]), np.ones(2))
    assert np.array_equal(big[0], [0.0, 1.0]) and np.array_equal(big[1], [0.0, 1e4])


A = 0x10000  # a 16-byte aligned fake address; the host checks never dereference it


def _p(i, off=0):
    return None if i is None else C.c_void_p(A + i * 0x100000 + off)


def test_sandwich_quant_host_checks(L):
    def call(y=_p(0), res=_p(1), gp=_p(2), ep=1e-5, gate=None, kind=0, rs=1.0, gs=_p(3), eps=1e-5,
             M=4, K=64, h=_p(4), q=_p(5), s=_p(6), fn=L.w8a8_sandwich_rmsnorm_quant):
        return fn(y, res, gp, C.c_float(ep), gate, kind, C.c_float(rs), gs, C.c_float(eps), M, K,
                  h, q, s, None)

    for missing in ("y", "res", "gs", "h", "q", "s"):
        assert call(**{missing: None}) == -1, missing
    assert call(gate=_p(7)) == -1 and call(kind=1) == -1          # gate and kind disagree
    assert call(gate=_p(7), kind=4) == -1 and call(gate=_p(7), kind=-1) == -1
    assert call(eps=-1.0) == -1 and call(ep=-1.0) == -1 and call(eps=float("nan")) == -1
    assert call(rs=float("inf")) == -1 and call(rs=float("nan")) == -1
    assert call(M=0) == -1 and call(K=8) == -1
    assert call(K=24) == -3 and call(K=32784) == -3
    assert call(h=_p(0)) == -1 and call(q=_p(0)) == -1            # outputs on an input
    assert call(h=_p(7), gate=_p(7), kind=3) == -1
    for bad in ("y", "res", "gp", "gs", "h", "q"):
        assert call(**{bad: _p(8, 8)}) == -2, bad
    assert call(gate=_p(7, 8), kind=2) == -2 and call(gate=_p(7, 8), kind=3) == -2
    if not torch.cuda.is_available():
        assert call() == -7 and call(gp=None, ep=-1.0) == -7      # eps_post ignored without it
        assert call(h=_p(1)) == -7                                # in place on the residual
        assert call(gate=_p(7, 4), kind=1) == -7                  # per token: no alignment
        assert call(fn=L.w8a8_sandwich_rmsnorm_quant_fp8) == -7


def test_sandwich_backward_host_checks(L):
    size = L.w8a8_sandwich_rmsnorm_backward_workspace_size
    assert size(0, 64) == 0 and size(4, 24) == 0
    # at most one part per row: two arrays of K sums each
    assert size(4, 64) == 4 * 2 * 64 * 4 and size(1, 32768) == 2 * 32768 * 4

    def call(dz=_p(0), dh=_p(1), y=_p(2), h=_p(3), gp=_p(4), ep=1e-5, gate=None, kind=0, rs=1.0,
             gs=_p(5), eps=1e-5, M=4, K=64, dy=_p(6), dres=_p(7), dgp=_p(8), dgate=None,
             dgs=_p(9), ws=_p(10), n=1 << 20):
        return L.w8a8_sandwich_rmsnorm_backward(
            dz, dh, y, h, gp, C.c_float(ep), gate, kind, C.c_float(rs), gs, C.c_float(eps), M, K,
            dy, dres, dgp, dgate, dgs, ws, n, None)

    for missing in ("dz", "y", "h", "gs", "dy", "dres", "dgs"):
        assert call(**{missing: None}) == -1, missing
    assert call(gp=None) == -1 and call(dgp=None) == -1           # both or neither
    assert call(gate=_p(11), kind=2) == -1                        # a gate without its gradient
    assert call(dgate=_p(11)) == -1
    assert call(M=0) == -1 and call(K=24) == -3
    assert call(dy=_p(0)) == -1 and call(dy=_p(1)) == -1 and call(dres=_p(3)) == -1
    assert call(dy=_p(7)) == -1
    assert call(dz=_p(0, 8)) == -2 and call(dres=_p(7, 8)) == -2
    if not torch.cuda.is_available():
        assert call() == -7 and call(dres=_p(1)) == -7            # in place on dh
        assert call(dh=None) == -7


def test_binding_checks():
    y = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        w8.w8a8_sandwich_rmsnorm_quant(y, y, torch.ones(64), 1e-5)
    with pytest.raises(ValueError, match="CUDA"):
        w8.w8a8_sandwich_rmsnorm_backward(y, y, y, torch.ones(64), 1e-5)
    for gate in (torch.ones(64), torch.ones(4, 64), torch.ones(4, 1, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="gate must be"):
            w8._gate_arg(gate, 4, 64, 0)
