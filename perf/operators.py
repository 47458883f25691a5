"""Measured cases of the 16-bit operators around the 4-bit layers: the dense
linear with its bias / activation / residual epilogue, the gated feed-forward
projection and the layer norm, each forward and backward.

`run` computes a case in its plain form (float32, elementary torch operations,
one rounding at the end) or, with `own` set, through the library's calls."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPI = {"none": 0, "gelu": 1, "silu": 2}
EPS = 1e-5
GELU_C = math.sqrt(2.0 / math.pi)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token through a small projection: the latency of a call
        dict(name="linear_token_bf16", op="linear", type="bf16", M=1, K=1024, N=1024, epi="gelu", bias=True,
             residual=True, keep=False),
        # a decode batch through the fused QKV projection: the weights' bytes
        dict(name="linear_decode_fp16", op="linear", type="fp16", M=23, K=3072, N=9216, epi="none", bias=True,
             residual=False, keep=False),
        # an odd batch at odd widths, kept for training, added to the residual stream
        dict(name="linear_ragged_fp16", op="linear", type="fp16", M=777, K=1160, N=2056, epi="silu", bias=True,
             residual=True, keep=True),
        # the QKV workload's shape with 16-bit weights: image and text tokens of one picture
        dict(name="linear_qkv_bf16", op="linear", type="bf16", M=4608, K=3072, N=9216, epi="none", bias=True,
             residual=False, keep=False),
        # the MLP's second projection in training: both products and the bias gradient
        dict(name="linear_bwd_fc2_bf16", op="linear_bwd", type="bf16", M=4608, K=12288, N=3072, epi="none", bias=True),
        # an odd micro-batch through an activation's derivative
        dict(name="linear_bwd_ragged_fp16", op="linear_bwd", type="fp16", M=1023, K=1160, N=2056, epi="gelu",
             bias=True),
        # one token through the gated feed-forward: twice the weights' bytes
        dict(name="gated_token_bf16", op="gated", type="bf16", M=1, K=3072, F=12288, act="silu", bias=False,
             keep=False),
        # the gated feed-forward of a training step, G and U kept
        dict(name="gated_train_bf16", op="gated", type="bf16", M=4608, K=3072, F=12288, act="silu", bias=True,
             keep=True),
        # its backward pass: four products, the gate's derivative, the bias gradients
        dict(name="gated_bwd_bf16", op="gated_bwd", type="bf16", M=4608, K=3072, F=12288, act="silu", bias=True),
        # a decode batch's norm, a latency case at an odd width
        dict(name="norm_decode_fp16", op="norm", type="fp16", M=33, C=1001, affine=True),
        # a long batch's norm
        dict(name="norm_train_bf16", op="norm", type="bf16", M=16384, C=3072, affine=True),
        # its backward pass with the weights' gradients
        dict(name="norm_bwd_bf16", op="norm_bwd", type="bf16", M=16384, C=3072, affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear_bwd", "gated", "gated_bwd", "norm", "norm_bwd"))
    if op.startswith("norm"):
        return dict(op=op, type=rng.choice(("bf16", "fp16", "fp32")), M=_log_int(rng, 1, 8192),
                    C=_log_int(rng, 64, 6000), affine=rng.random() < 0.8)
    # widths are multiples of 8; as many tokens as keep the case below the largest listed one
    K, N = 8 * _log_int(rng, 8, 1536), 8 * _log_int(rng, 8, 1536)
    most = max(1, min(8192, 150_000_000_000 // (K * N)))
    M = _log_int(rng, 1, most)
    case = dict(op=op, type=rng.choice(("bf16", "fp16")), M=M, K=K, bias=rng.random() < 0.7)
    act = rng.choice(("none", "gelu", "silu"))
    if op == "linear":
        return dict(case, N=N, epi=act, residual=rng.random() < 0.5, keep=act != "none" and rng.random() < 0.5)
    if op == "linear_bwd":
        return dict(case, N=N, epi=act)
    if op == "gated":
        return dict(case, F=N, act=act, keep=rng.random() < 0.5)
    return dict(case, F=N, act=act)


# ---------------------------------------------------------------- what a program holds before the call
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    op, M = case["op"], case["M"]
    s = {"op": op, "M": M, "case": case}
    if op.startswith("norm"):
        C = case["C"]
        # a residual stream: an offset and a scale of its own per row, a few large channels
        x = normal(M, C) * (0.5 + torch.rand(M, 1, generator=g, device="cuda")) + 0.3 * normal(M, 1) + 0.1
        wide = torch.randperm(C, generator=g, device="cuda")[:max(1, C // 200)]
        x[:, wide] *= 20.0
        s["X"] = x.to(t)
        s["gamma"] = (1.0 + normal(C, scale=0.1)).to(t) if case["affine"] else None
        s["beta"] = normal(C, scale=0.1).to(t) if case["affine"] else None
        if op == "norm":
            s.update(Y=empty(M, C), mean=empty(M, dtype=torch.float32), rstd=empty(M, dtype=torch.float32))
        else:
            xf = s["X"].float()
            mean = xf.mean(1)
            s["mean"] = mean
            s["rstd"] = 1.0 / torch.sqrt((xf - mean[:, None]).square().mean(1) + EPS)
            s["dY"] = normal(M, C, scale=0.1).to(t)
            s.update(dX=empty(M, C), dgamma=empty(C) if case["affine"] else None,
                     dbeta=empty(C) if case["affine"] else None)
        return s
    K = case["K"]
    N = case["F"] if op.startswith("gated") else case["N"]
    # the workloads' recipe: a few input channels are 20 times as large, and
    # 5 times in the weight
    wide = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 200)]

    def weight():
        w = normal(N, K, scale=0.02)
        w[:, wide] *= 5.0
        return w.to(t)

    x = normal(M, K)
    x[:, wide] *= 20.0
    s["X"] = x.to(t)
    if op.startswith("linear"):
        s["W"] = weight()
        s["b"] = normal(N, scale=0.1).to(t) if case["bias"] else None
        if op == "linear":
            s["R"] = normal(M, N, scale=2.0).to(t) if case["residual"] else None
            s.update(Y=empty(M, N), Z=empty(M, N) if case["keep"] else None)
        else:
            s["Z"] = normal(M, N, scale=2.0).to(t) if case["epi"] != "none" else None
            s["dY"] = normal(M, N, scale=0.05).to(t)
            s.update(dX=empty(M, K), dW=empty(N, K), db=empty(N) if case["bias"] else None)
        return s
    s["Wg"], s["Wu"] = weight(), weight()
    s["bg"] = normal(N, scale=0.1).to(t) if case["bias"] else None
    s["bu"] = normal(N, scale=0.1).to(t) if case["bias"] else None
    if op == "gated":
        s.update(H=empty(M, N), G=empty(M, N) if case["keep"] else None, U=empty(M, N) if case["keep"] else None)
    else:
        s["G"], s["U"] = normal(M, N, scale=2.0).to(t), normal(M, N, scale=2.0).to(t)
        s["dH"] = normal(M, N, scale=0.05).to(t)
        s.update(dX=empty(M, K), dWg=empty(N, K), dWu=empty(N, K), dbg=empty(N) if case["bias"] else None,
                 dbu=empty(N) if case["bias"] else None)
    return s


# ---------------------------------------------------------------- plain forms
def _act(z, kind):
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, kind):
    if kind == "gelu":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * 0.044715 * z * z)
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain_linear(s, c, t):
    z = s["X"].float() @ s["W"].float().T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, c["epi"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return [y.to(t)] + ([z.to(t)] if c["keep"] else [])


def _plain_linear_bwd(s, c, t):
    dz = s["dY"].float()
    if c["epi"] != "none":
        dz = dz * _act_slope(s["Z"].float(), c["epi"])
    out = [(dz @ s["W"].float()).to(t), (dz.T @ s["X"].float()).to(t)]
    return out + ([dz.sum(0).to(t)] if c["bias"] else [])


def _plain_gated(s, c, t):
    x = s["X"].float()
    a, u = x @ s["Wg"].float().T, x @ s["Wu"].float().T
    if s["bg"] is not None:
        a, u = a + s["bg"].float(), u + s["bu"].float()
    return [(_act(a, c["act"]) * u).to(t)] + ([a.to(t), u.to(t)] if c["keep"] else [])


def _plain_gated_bwd(s, c, t):
    dh, a, u, x = s["dH"].float(), s["G"].float(), s["U"].float(), s["X"].float()
    da, du = dh * u * _act_slope(a, c["act"]), dh * _act(a, c["act"])
    out = [(da @ s["Wg"].float() + du @ s["Wu"].float()).to(t), (da.T @ x).to(t), (du.T @ x).to(t)]
    return out + ([da.sum(0).to(t), du.sum(0).to(t)] if c["bias"] else [])


def _plain_norm(s, c, t):
    x = s["X"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None]
    if s["gamma"] is not None:
        y = y * s["gamma"].float() + s["beta"].float()
    return [y.to(t), mean, rstd]


def _plain_norm_bwd(s, c, t):
    dy, rstd = s["dY"].float(), s["rstd"][:, None]
    xh = (s["X"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float() if s["gamma"] is not None else dy
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["gamma"] is None:
        return [dx.to(t)]
    return [dx.to(t), (dy * xh).sum(0).to(t), dy.sum(0).to(t)]


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "gated": _plain_gated,
          "gated_bwd": _plain_gated_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


# ---------------------------------------------------------------- the library's calls
def _own(s, c):
    from rank_gemm_b200 import binding as B

    def workspace(nbytes):
        if "ws" not in s:   # kept from pass to pass, as a program keeps it
            s["ws"] = torch.empty(max(nbytes(), 16), dtype=torch.uint8, device="cuda")
        return s["ws"]

    op, M = s["op"], s["M"]
    if op == "linear":
        B.svdq_dense_linear(M, c["K"], c["N"], s["X"], s["W"], s["b"], EPI[c["epi"]], s["R"], s["Y"], s["Z"])
        return [s["Y"]] + ([s["Z"]] if c["keep"] else [])
    if op == "linear_bwd":
        K, N, epi = c["K"], c["N"], EPI[c["epi"]]
        ws = workspace(lambda: B.svdq_dense_linear_backward_workspace_bytes(M, K, N, epi))
        B.svdq_dense_linear_backward(M, K, N, s["dY"], s["X"], s["W"], s["Z"], epi, s["dX"], s["dW"], s["db"], ws)
        return [s["dX"], s["dW"]] + ([s["db"]] if c["bias"] else [])
    if op == "gated":
        B.svdq_gated_linear(M, c["K"], c["F"], s["X"], s["Wg"], s["Wu"], s["bg"], s["bu"], EPI[c["act"]], s["H"],
                            s["G"], s["U"])
        return [s["H"]] + ([s["G"], s["U"]] if c["keep"] else [])
    if op == "gated_bwd":
        K, F = c["K"], c["F"]
        ws = workspace(lambda: B.svdq_gated_linear_backward_workspace_bytes(M, K, F))
        B.svdq_gated_linear_backward(M, K, F, s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"], EPI[c["act"]],
                                     s["dX"], s["dWg"], s["dWu"], s["dbg"], s["dbu"], ws)
        return [s["dX"], s["dWg"], s["dWu"]] + ([s["dbg"], s["dbu"]] if c["bias"] else [])
    if op == "norm":
        B.svdq_layernorm(M, c["C"], s["X"], s["gamma"], s["beta"], EPS, s["Y"], s["mean"], s["rstd"])
        return [s["Y"], s["mean"], s["rstd"]]
    ws = workspace(lambda: B.svdq_layernorm_backward_workspace_bytes(M, c["C"]))
    B.svdq_layernorm_backward(M, c["C"], s["dY"], s["X"], s["gamma"], s["mean"], s["rstd"], s["dX"], s["dgamma"],
                              s["dbeta"], ws)
    return [s["dX"]] + ([s["dgamma"], s["dbeta"]] if c["affine"] else [])


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return _PLAIN[state["op"]](state, case, TYPES[case["type"]])


# ---------------------------------------------------------------- work
def work(case):
    size = 4 if case["type"] == "fp32" else 2
    op, M = case["op"], case["M"]
    if op.startswith("norm"):
        C, aff = case["C"], 1 if case["affine"] else 0
        if op == "norm":
            return {"bytes": size * (2 * M * C + 2 * C * aff) + 8 * M, "flops": 8 * M * C}
        return {"bytes": size * (3 * M * C + 3 * C * aff) + 8 * M, "flops": 14 * M * C}
    K, b = case["K"], 1 if case["bias"] else 0
    if op == "linear":
        N = case["N"]
        return {"bytes": size * (M * K + N * K + M * N * (1 + case["residual"] + case["keep"]) + N * b),
                "flops": 2 * M * K * N}
    if op == "linear_bwd":
        N = case["N"]
        return {"bytes": size * (M * N * (1 + (case["epi"] != "none")) + 2 * M * K + 2 * N * K + N * b),
                "flops": 4 * M * K * N}
    F = case["F"]
    if op == "gated":
        return {"bytes": size * (M * K + 2 * F * K + M * F * (1 + 2 * case["keep"]) + 2 * F * b), "flops": 4 * M * K * F}
    return {"bytes": size * (3 * M * F + 2 * M * K + 4 * F * K + 2 * F * b), "flops": 8 * M * K * F}


# ---------------------------------------------------------------- the definition in 64 bits
def _sigmoid64(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _act64(x, kind):
    """(act(x), act'(x)); the tanh-form GELU is x sigmoid(2u), u = sqrt(2/pi) (x + 0.044715 x^3)."""
    if kind == "none":
        return x, torch.ones_like(x)
    if kind == "silu":
        p, dp_arg = _sigmoid64(x), torch.ones_like(x)
    else:
        k = math.sqrt(8.0 / math.pi)
        p, dp_arg = _sigmoid64(k * (x + 0.044715 * x ** 3)), k * (1.0 + 0.134145 * x ** 2)
    return x * p, p + x * p * (1.0 - p) * dp_arg


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: x.double() for k, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    op = case["op"]
    if op == "norm":
        var, mean = torch.var_mean(v["X"], dim=1, correction=0)
        rstd = (var + EPS).rsqrt()
        y = torch.einsum("mc,m->mc", v["X"] - mean.unsqueeze(1), rstd)
        if case["affine"]:
            y = torch.addcmul(v["beta"].expand_as(y), y, v["gamma"].expand_as(y))
        return [y, mean, rstd]
    if op == "norm_bwd":
        C = case["C"]
        xh = torch.einsum("mc,m->mc", v["X"] - v["mean"].unsqueeze(1), v["rstd"])
        w = v["gamma"] if case["affine"] else torch.ones(C, dtype=torch.float64, device="cuda")
        a = torch.mv(v["dY"], w) / C                        # mean of dy gamma
        b = torch.mv(v["dY"] * xh, w) / C                   # mean of dy gamma xh
        dx = (v["dY"] * w - a.unsqueeze(1) - xh * b.unsqueeze(1)) * v["rstd"].unsqueeze(1)
        if not case["affine"]:
            return [dx]
        return [dx, torch.einsum("mc,mc->c", v["dY"], xh), torch.einsum("mc->c", v["dY"])]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", v["X"], v["W"]) + (v["b"] if case["bias"] else 0.0)
        y = _act64(z, case["epi"])[0] + (v["R"] if case["residual"] else 0.0)
        return [y] + ([z] if case["keep"] else [])
    if op == "linear_bwd":
        dz = v["dY"] if case["epi"] == "none" else v["dY"] * _act64(v["Z"], case["epi"])[1]
        out = [torch.einsum("mn,nk->mk", dz, v["W"]), torch.einsum("mn,mk->nk", dz, v["X"])]
        return out + ([torch.einsum("mn->n", dz)] if case["bias"] else [])
    if op == "gated":
        a = torch.einsum("mk,nk->mn", v["X"], v["Wg"]) + (v["bg"] if case["bias"] else 0.0)
        u = torch.einsum("mk,nk->mn", v["X"], v["Wu"]) + (v["bu"] if case["bias"] else 0.0)
        return [_act64(a, case["act"])[0] * u] + ([a, u] if case["keep"] else [])
    f, slope = _act64(v["G"], case["act"])
    da, du = v["dH"] * v["U"] * slope, v["dH"] * f
    out = [torch.einsum("mn,nk->mk", da, v["Wg"]) + torch.einsum("mn,nk->mk", du, v["Wu"]),
           torch.einsum("mn,mk->nk", da, v["X"]), torch.einsum("mn,mk->nk", du, v["X"])]
    return out + ([torch.einsum("mn->n", da), torch.einsum("mn->n", du)] if case["bias"] else [])
