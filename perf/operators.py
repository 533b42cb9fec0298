"""The operators around a quantized decoder block and the gradients of its W8A8 linears, as cases
to be measured: the norms after and before a block with its gate and residual scale (forward to
int8 or E4M3 codes, and backward), the input and weight gradients of a W8A8 linear, and the
backward pass of the gated feed-forward block (the down projection's input gradient with
SiLU(gate) * up differentiated in its epilogue).

`run` computes an operator in its plain form (elementary torch operations in binary32), or calls
the framework where `own` is true. Codes of 8 bits are returned as the values they stand for
(code times the row's scale), rounded to bf16.
"""
import math

import torch

own = False

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5


def _w8():
    import int8_w8a8_quantized_smoothed_b200 as w8
    return w8


# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a serving step between two blocks: latency
        dict(name="norm_token", op="norm", M=1, K=4096, code="int8", post=True, gate="none",
             res_scale=1.0),
        # a ragged batch, an odd row length, a learned gate per channel, FP8 codes
        dict(name="norm_ragged_fp8", op="norm", M=333, K=5136, code="fp8", post=True,
             gate="channel", res_scale=0.5),
        # a prefill batch whose block output passes an elementwise gate
        dict(name="norm_prefill", op="norm", M=8192, K=4096, code="int8", post=True, gate="full",
             res_scale=1.0),
        # one calibration batch of a block that is tuned, a gate per token
        dict(name="norm_back_512", op="norm_back", M=512, K=4096, post=True, gate="token",
             res_scale=1.0),
        # the largest rows and batch: the wider model's hidden size
        dict(name="norm_back_8192", op="norm_back", M=8192, K=8192, post=True, gate="channel",
             res_scale=0.5),
        # few tokens through the qkv projection: the weight's bytes count
        dict(name="dgrad_small", op="dgrad", M=16, N=6144, K=4096, code="int8"),
        # a tuning batch through the gate|up projection
        dict(name="dgrad_gate_up", op="dgrad", M=2048, N=28672, K=4096, code="int8"),
        # odd sizes on every side, FP8 codes
        dict(name="dgrad_ragged_fp8", op="dgrad", M=331, N=4104, K=4112, code="fp8"),
        # the gated block of the smaller model: down projection and SiLU backward
        dict(name="silu_back_512", op="silu_back", M=512, N=4096, K=14336, code="int8"),
        # the gated block of the wider model, FP8 codes: the largest product
        dict(name="silu_back_wide_fp8", op="silu_back", M=2048, N=8192, K=28672, code="fp8"),
        # the down projection's weight gradient
        dict(name="wgrad_down", op="wgrad", M=2048, N=4096, K=14336, code="int8"),
        # an odd number of tokens, odd sides, FP8 codes: short sums
        dict(name="wgrad_ragged_fp8", op="wgrad", M=777, N=1032, K=2064, code="fp8"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "dgrad", "silu_back", "wgrad"])
    code = rng.choice(["int8", "fp8"])
    if op in ("norm", "norm_back"):
        case = dict(op=op, M=_spread(rng, 1, 8192), K=_spread(rng, 256, 8192, 16),
                    post=rng.random() < 0.75,
                    gate=rng.choice(["none", "token", "channel", "full"]),
                    res_scale=rng.choice([1.0, 0.5, 1.25]))
        if op == "norm":
            case["code"] = code
        return case
    case = dict(op=op, M=_spread(rng, 1, 4096), N=_spread(rng, 512, 16384, 8),
                K=_spread(rng, 512, 16384, 16), code=code)
    most = 2048 * 8192 * 28672  # the largest listed product
    case["M"] = max(1, min(case["M"], most // (case["N"] * case["K"])))
    return case


# ----------------------------------------------------------------------------------- inputs


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _activation(g, M, K):
    """N(0, 1) with one channel in a hundred fifty times as wide, as activations have."""
    x = _normal(g, M, K)
    wide = torch.rand(K, generator=g, device="cuda") < 0.01
    return (x * torch.where(wide, 50.0, 1.0)).to(BF16)


def _codes(g, rows, cols, code):
    """Codes and row scales of a quantized N(0, 1) matrix (its scale a hundredth)."""
    x = _normal(g, rows, cols)
    top = 127.0 if code == "int8" else 448.0
    s = x.abs().amax(dim=1) / top
    x /= s[:, None]
    q = x.round().to(torch.int8) if code == "int8" else x.clamp(-448.0, 448.0).to(FP8)
    return q, s * 0.01


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    M, K, st = case["M"], case["K"], dict(case)
    if case["op"] in ("norm", "norm_back"):
        st["y"] = _activation(g, M, K)
        st["gamma_pre"] = 1.0 + 0.1 * _normal(g, K)
        st["gamma_post"] = 1.0 + 0.1 * _normal(g, K) if case["post"] else None
        gate = case["gate"]
        st["gate_value"] = {
            "none": lambda: None,
            "token": lambda: torch.sigmoid(_normal(g, M, 1)),
            "channel": lambda: 0.5 + 0.2 * _normal(g, 1, K),
            "full": lambda: torch.sigmoid(_normal(g, M, K)).to(BF16),
        }[gate]()
        if case["op"] == "norm":
            st["residual"] = _activation(g, M, K)
        else:
            st["h"] = _activation(g, M, K)
            st["dz"] = (1e-2 * _normal(g, M, K)).to(BF16)
            st["dh"] = (1e-2 * _normal(g, M, K)).to(BF16)
        return st
    N = case["N"]
    st["dy"] = (1e-2 * _normal(g, M, N)).to(BF16)
    if case["op"] == "wgrad":
        st["q"], st["s"] = _codes(g, M, K, case["code"])
    else:
        st["q"], st["s"] = _codes(g, N, K, case["code"])
    if case["op"] == "silu_back":
        st["gate_up"] = (2.0 * _normal(g, M, 2 * K)).to(BF16)
    return st


# ------------------------------------------------------------------------------------ passes


def _rstd(x, eps):
    """1 / rms of each row: the mean of squares in 64 bits (it decides codes next to a border)."""
    ms = (x.double().square().sum(dim=1, keepdim=True) / x.shape[1]).float()
    return 1.0 / torch.sqrt(ms + eps)


def _plain_norm(st):
    y, r = st["y"].float(), st["residual"].float()
    n = y * _rstd(y, EPS) * st["gamma_post"] if st["gamma_post"] is not None else y
    b = n if st["gate_value"] is None else st["gate_value"].float() * n
    h = (st["res_scale"] * r + b).to(BF16)
    hf = h.float()
    z = hf * _rstd(hf, EPS) * st["gamma_pre"]
    top = 127.0 if st["code"] == "int8" else 448.0
    s = z.abs().amax(dim=1) / top
    t = torch.where(s[:, None] > 0, z / s[:, None], torch.zeros_like(z))
    q = t.round().clamp(-127, 127) if st["code"] == "int8" else t.clamp(-448, 448).to(FP8).float()
    return (q * s[:, None]).to(BF16), s, h


def _plain_norm_back(st):
    y, h, dz, dh = (st[k].float() for k in ("y", "h", "dz", "dh"))
    K = y.shape[1]
    r2 = _rstd(h, EPS)
    w = dz * st["gamma_pre"]
    dht = dh + r2 * (w - h * (r2 * r2 * ((w * h).sum(dim=1, keepdim=True) / K)))
    dgamma_pre = (dz * h * r2).sum(dim=0)
    post, gate = st["gamma_post"], st["gate_value"]
    r1 = _rstd(y, EPS) if post is not None else None
    x1 = y * r1 if post is not None else y
    n = x1 * post if post is not None else y
    dn = dht if gate is None else dht * gate.float()
    dgate = None
    if st["gate"] == "token":
        dgate = (dht * n).sum(dim=1, keepdim=True)
    elif st["gate"] == "channel":
        dgate = (dht * n).sum(dim=0, keepdim=True)
    elif st["gate"] == "full":
        dgate = (dht * n).to(BF16)
    dgamma_post = None
    dy = dn
    if post is not None:
        dgamma_post = (dn * x1).sum(dim=0)
        v = dn * post
        dy = r1 * (v - x1 * ((v * x1).sum(dim=1, keepdim=True) / K))
    return (dy.to(BF16), (st["res_scale"] * dht).to(BF16), dgamma_pre, dgamma_post, dgate)


def _plain_products(st):
    x = st["q"].float() * st["s"][:, None]
    if st["op"] == "wgrad":
        return (st["dy"].float().t() @ x).to(BF16)
    d = st["dy"].float() @ x
    if st["op"] == "dgrad":
        return d.to(BF16)
    g, u = (t.float() for t in st["gate_up"].chunk(2, dim=1))
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg = d * u * sig * (1.0 + g * (1.0 - sig))
    return torch.cat([dg, d * g * sig], dim=1).to(BF16)


def _own(st):
    w8 = _w8()
    f8 = "_fp8" if st.get("code") == "fp8" else ""
    if st["op"] == "norm":
        call = getattr(w8, "w8a8_sandwich_rmsnorm_quant" + f8)
        q, s, h = call(st["y"], st["residual"], st["gamma_pre"], EPS, gamma_post=st["gamma_post"],
                       gate=st["gate_value"], res_scale=st["res_scale"])
        # the values the codes stand for: one product, rounded to bf16 as it is stored
        codes = q if not f8 else q.to(BF16)
        return torch.mul(codes, s[:, None], out=torch.empty_like(h)), s, h
    if st["op"] == "norm_back":
        return w8.w8a8_sandwich_rmsnorm_backward(
            st["dz"], st["y"], st["h"], st["gamma_pre"], EPS, dh=st["dh"],
            gamma_post=st["gamma_post"], gate=st["gate_value"], res_scale=st["res_scale"])
    if st["op"] == "dgrad":
        return getattr(w8, "w8a8_gemm_dgrad" + f8)(st["dy"], st["q"], st["s"])
    if st["op"] == "wgrad":
        return getattr(w8, "w8a8_gemm_wgrad" + f8)(st["dy"], st["q"], st["s"])
    return getattr(w8, "w8a8_gemm_dgrad_silu" + f8)(st["dy"], st["q"], st["s"], st["gate_up"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _plain_norm(state)
    if state["op"] == "norm_back":
        return _plain_norm_back(state)
    return _plain_products(state)


# -------------------------------------------------------------------------------------- work


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] in ("norm", "norm_back"):
        vectors = 4 * K * (1 + int(case["post"]) + int(case["gate"] == "channel"))
        rows = 4 * M * int(case["gate"] == "token")
        full = 2 * M * K * int(case["gate"] == "full")
        if case["op"] == "norm":  # y, residual in; h, codes, scales out
            return {"bytes": 7 * M * K + 4 * M + vectors + rows + full, "flops": 12 * M * K}
        # dz, dh, y, h in; dy, dresidual out; the gains and the gate in, their gradients out
        return {"bytes": 12 * M * K + 2 * (vectors + rows + full), "flops": 30 * M * K}
    N = case["N"]
    flops = 2 * M * N * K
    if case["op"] == "wgrad":
        return {"bytes": 2 * M * N + M * K + 4 * M + 2 * N * K, "flops": flops}
    moved = 2 * M * N + N * K + 4 * N
    if case["op"] == "dgrad":
        return {"bytes": moved + 2 * M * K, "flops": flops}
    return {"bytes": moved + 8 * M * K, "flops": flops + 12 * M * K}


# ----------------------------------------------------------------------- from the definition


def exact(case, seed):
    """What `run` returns, from the operators' definitions in 64 bits. The gradients follow from
    differentiating the definitions directly (the norm as a map x -> x / sqrt(mean x^2 + eps))."""
    st = prepare(case, seed)
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in st.items()}
    op = case["op"]
    if op == "wgrad":
        return torch.einsum("mn,mk->nk", f["dy"], f["q"] * f["s"].unsqueeze(1))
    if op in ("dgrad", "silu_back"):
        da = torch.einsum("mn,nk->mk", f["dy"] * f["s"], f["q"])
        if op == "dgrad":
            return da
        K = case["K"]
        g, u = f["gate_up"][:, :K], f["gate_up"][:, K:]
        e = torch.exp(-g.abs())  # the logistic function without overflow on either side
        sig = torch.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        slope = sig + g * sig * torch.where(g >= 0, e / (1.0 + e), 1.0 / (1.0 + e))
        out = torch.empty_like(f["gate_up"])
        out[:, :K] = da * u * slope
        out[:, K:] = da * g * sig
        return out
    y, K = f["y"], case["K"]
    gate = 1.0 if f["gate_value"] is None else f["gate_value"]

    def unit(x):
        return x / torch.sqrt(torch.mean(x * x, dim=1, keepdim=True) + EPS)

    def back(x, d):
        """d(unit(x)) applied to d: d / rms - x (x . d) / (K rms^3)."""
        rms = torch.sqrt(torch.mean(x * x, dim=1, keepdim=True) + EPS)
        return d / rms - x * (x * d).sum(dim=1, keepdim=True) / (K * rms ** 3)

    post = f["gamma_post"] if case["post"] else None
    n = unit(y) * post if case["post"] else y
    if op == "norm":
        h = (case["res_scale"] * f["residual"] + gate * n)
        hb = h.to(BF16).double()  # the norm reads the stored, rounded sum
        z = unit(hb) * f["gamma_pre"]
        if case["code"] == "int8":
            s = z.abs().amax(dim=1) / 127
            q = torch.round(z / s.clamp_min(1e-300)[:, None])
        else:
            s = z.abs().amax(dim=1) / 448
            q = (z / s.clamp_min(1e-300)[:, None]).clamp(-448, 448).float().to(FP8).double()
        return q * s[:, None], s, h
    dht = f["dh"] + back(f["h"], f["dz"] * f["gamma_pre"])
    dn = gate * dht
    dgate = {"none": lambda: None, "token": lambda: (dht * n).sum(1, keepdim=True),
             "channel": lambda: (dht * n).sum(0, keepdim=True), "full": lambda: dht * n}
    return (back(y, dn * post) if case["post"] else dn, case["res_scale"] * dht,
            (f["dz"] * unit(f["h"])).sum(0),
            (dn * unit(y)).sum(0) if case["post"] else None, dgate[case["gate"]]())
