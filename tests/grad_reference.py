"""The block-boundary norms and the gradients of a W8A8 linear in binary64, written from their
formulas, with the magnitudes that bound a binary32 evaluation's error. U is the unit roundoff of
binary32; a value stored as bf16 is off by at most 2^-8 relative (half a step)."""
import numpy as np

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def rstd(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)


def forward(y, residual, gamma_pre, eps, gamma_post=None, eps_post=None, gate=None, res_scale=1.0):
    """(h, z) without any rounding."""
    n = y if gamma_post is None else y * rstd(y, eps if eps_post is None else eps_post) * gamma_post
    h = res_scale * residual + (n if gate is None else gate * n)
    return h, h * rstd(h, eps) * gamma_pre


def backward(dz, y, h, gamma_pre, eps, dh=None, gamma_post=None, eps_post=None, gate=None,
             res_scale=1.0):
    """name -> (gradient, magnitude): the magnitude is the same expression with every term's
    absolute value, so a binary32 evaluation is off by a small multiple of U times it."""
    K = y.shape[1]
    dh = np.zeros_like(dz) if dh is None else dh
    r2 = rstd(h, eps)
    w = dz * gamma_pre
    D = dh + r2 * w - h * r2 ** 3 * (w * h).sum(1, keepdims=True) / K
    Dm = np.abs(dh) + r2 * np.abs(w) + np.abs(h) * r2 ** 3 * np.abs(w * h).sum(1, keepdims=True) / K
    out = {"dresidual": (res_scale * D, abs(res_scale) * Dm),
           "dgamma_pre": ((dz * h * r2).sum(0), np.abs(dz * h * r2).sum(0))}
    g = 1.0 if gate is None else gate
    if gamma_post is not None:
        r1 = rstd(y, eps if eps_post is None else eps_post)
        n = y * r1 * gamma_post
        v, vm = g * gamma_post * D, np.abs(g * gamma_post) * Dm
        out["dy"] = (r1 * v - y * r1 ** 3 * (v * y).sum(1, keepdims=True) / K,
                     r1 * vm + np.abs(y) * r1 ** 3 * (vm * np.abs(y)).sum(1, keepdims=True) / K)
        out["dgamma_post"] = ((g * D * y * r1).sum(0), (np.abs(g * y * r1) * Dm).sum(0))
    else:
        n = y
        out["dy"] = (g * D, np.abs(g) * Dm)
    if gate is not None:
        full, fm = D * n, Dm * np.abs(n)
        if gate.shape[1] == 1:
            full, fm = full.sum(1, keepdims=True), fm.sum(1, keepdims=True)
        elif gate.shape[0] == 1:
            full, fm = full.sum(0, keepdims=True), fm.sum(0, keepdims=True)
        out["dgate"] = (full, fm)
    return out


def silu_grads(da, g, u):
    """(dg, du) of a = silu(g) u."""
    e = np.exp(-np.abs(g))
    sig = np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    rest = np.where(g >= 0, e / (1.0 + e), 1.0 / (1.0 + e))  # 1 - sig
    return da * u * sig * (1.0 + g * rest), da * g * sig
