"""Cases of the operators between a predictor's features and the rendered parameters.

    linear         y = act(x W^T + b) + r                    (rows in 16 bits, or in 8 bits with a scale a row)
    linear_bwd     dx, dW, db of it from dy                  (z = x W^T + b is formed again where the activation needs it)
    gated          h = act(x Wg^T) * (x Wu^T)                (16 or 8 bits)
    gated_bwd      dx, dWg, dWu of it from dh                (both products are formed again)
    rms_norm       s = x + r, y = s / sqrt(mean s^2 + eps) * w, optionally in 8 bits with a scale a row
    rms_norm_bwd   dx (which is dr too) and dw from dy and ds

Rows are Gaussians (frames x Gaussians a frame of the package's workloads) or feature tokens.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}
E4M3_MAX = 448.0          # largest finite value of the 8-bit type
MIN_SCALE = 2.0 ** -126   # scale of rows too small to have one
EPS = 1e-6


def listed():
    return [
        # The Gaussian head of 8 frames of 65536 Gaussians with 3 channels: features to 5 + 3 parameters on base positions.
        dict(name="linear head 512x512", op="linear", M=524288, K=256, N=8, dtype="bf16", out="fp32", act="none", bias=True, residual=True),
        # A feed-forward block's second product with the block's input added, 16 frames of 4096 Gaussians.
        dict(name="linear down rgb128", op="linear", M=65536, K=1024, N=256, dtype="bf16", out="bf16", act="none", bias=True, residual=True),
        # One small frame (64 Gaussians, 1 channel): latency counts.
        dict(name="linear head tiny", op="linear", M=64, K=128, N=6, dtype="fp16", out="fp32", act="none", bias=True, residual=True),
        # Training the head of 16 frames of 1024 Gaussians, 1 channel.
        dict(name="linear_bwd head mono64", op="linear_bwd", M=16384, K=512, N=6, dtype="bf16", out="fp32", act="none", bias=True, residual=False),
        # A hidden layer of odd sizes with its activation, trained in fp16.
        dict(name="linear_bwd ragged gelu", op="linear_bwd", M=10007, K=394, N=777, dtype="fp16", out="fp16", act="gelu", bias=True, residual=False),
        # The gated block of 16 frames of 4096 Gaussians.
        dict(name="gated rgb128", op="gated", M=65536, D=256, F=1024, dtype="bf16", act="silu"),
        # One token while serving.
        dict(name="gated one row", op="gated", M=1, D=512, F=2048, dtype="fp16", act="gelu_tanh"),
        # The same block in 8 bits, wider.
        dict(name="gated fp8 wide", op="gated", M=32768, D=512, F=2048, dtype="fp8", act="silu"),
        # Training the gated block of 16 frames of 1024 Gaussians.
        dict(name="gated_bwd mono64", op="gated_bwd", M=16384, D=256, F=1024, dtype="bf16", act="silu"),
        # The norm before the 8-bit block, with the residual stream's update.
        dict(name="rms_norm fp8 rgb128", op="rms_norm", M=65536, D=512, dtype="bf16", out="fp8", residual=True),
        # A norm of an odd width in fp32.
        dict(name="rms_norm ragged fp32", op="rms_norm", M=16384, D=333, dtype="fp32", out="fp32", residual=False),
        # Training the norm over 320 frames of 2048 / 8 tokens.
        dict(name="rms_norm_bwd field", op="rms_norm_bwd", M=81920, D=512, dtype="bf16", out="bf16", residual=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half of the time a multiple of 64, else any number."""
    n = _spread(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd", "rms_norm", "rms_norm_bwd"])
    kind = rng.choice(["bf16", "fp16"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op.startswith("linear"):
        head = rng.random() < 0.4
        c = dict(op=op, M=_spread(rng, 1, 131072), K=_width(rng, 16, 1024),
                 N=5 + rng.randint(1, 8) if head else _width(rng, 16, 1024),
                 dtype=kind, out="fp32" if head else kind, act="none" if head else rng.choice(["none", act]),
                 bias=head or rng.random() < 0.7, residual=op == "linear" and (head or rng.random() < 0.5))
        if op == "linear" and not head and rng.random() < 0.25:
            c.update(dtype="fp8", out="bf16")
    elif op.startswith("gated"):
        c = dict(op=op, M=_spread(rng, 1, 65536), D=_width(rng, 16, 1024), F=_width(rng, 32, 2048),
                 dtype="fp8" if op == "gated" and rng.random() < 0.3 else kind, act=act)
    else:
        kind = rng.choice(["bf16", "fp16", "fp32"])
        c = dict(op=op, M=_spread(rng, 1, 131072), D=_width(rng, 16, 8192), dtype=kind,
                 out="fp8" if op == "rms_norm" and rng.random() < 0.4 else kind, residual=rng.random() < 0.6)
    most = max(work(x)["flops"] for x in listed()), max(work(x)["bytes"] for x in listed())
    while work(c)["flops"] > most[0] or work(c)["bytes"] > most[1]:
        c["M"] = max(1, c["M"] * 3 // 4)
    return c


def work(case):
    c, M = case, case["M"]
    e = BYTES[c["dtype"]]
    if c["op"] == "linear":
        K, N, o = c["K"], c["N"], BYTES[c["out"]]
        scales = 4 * (M + N) if c["dtype"] == "fp8" else 0
        return {"flops": 2 * M * N * K, "bytes": e * (M * K + N * K) + o * M * N * (2 if c["residual"] else 1) + 4 * N * c["bias"] + scales}
    if c["op"] == "linear_bwd":
        K, N, o = c["K"], c["N"], BYTES[c["out"]]
        return {"flops": 2 * M * N * K * (2 if c["act"] == "none" else 3), "bytes": o * M * N + 2 * e * (M * K + N * K) + 8 * N * c["bias"]}
    if c["op"] == "gated":
        D, F = c["D"], c["F"]
        scales = 4 * (M + 2 * F) if c["dtype"] == "fp8" else 0
        return {"flops": 4 * M * D * F, "bytes": e * (M * D + 2 * D * F) + 2 * M * F + scales}
    if c["op"] == "gated_bwd":
        D, F = c["D"], c["F"]
        return {"flops": 12 * M * D * F, "bytes": e * (M * F + 2 * M * D + 4 * D * F)}
    D, n = c["D"], 2 if c["residual"] else 1
    if c["op"] == "rms_norm":
        return {"flops": 4 * M * D, "bytes": (e * (2 * n - 1) + BYTES[c["out"]]) * M * D + 4 * D + (4 * M if c["out"] == "fp8" else 0)}
    return {"flops": 8 * M * D, "bytes": e * (2 + n) * M * D + 8 * D}


def _weight(gen, dtype, n, k):
    """A layer's weight at its usual initial spread; in 8 bits with a scale for each row."""
    w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
    return _rows8(w) if dtype == "fp8" else (w.to(DTYPES[dtype]), None)


def _rows8(v):
    """Rows in 8 bits, as a checkpoint or the step before holds them: (values, scale of each row)."""
    scale = (v.abs().amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    M, dt = c["M"], c["dtype"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rows(width):
        v = normal(M, width)
        return _rows8(v) if dt == "fp8" else (v.to(DTYPES[dt]), None)

    def gradient(width, kind):
        # Gradients of a mean over pixels are small; fp16 training scales its loss up.
        return (normal(M, width) * (1.0 if kind == "fp16" else 0.01)).to(DTYPES[kind])

    s = dict(case=c)
    if c["op"].startswith("linear"):
        s["x"], s["x_scale"] = rows(c["K"])
        s["w"], s["w_scale"] = _weight(gen, dt, c["N"], c["K"])
        s["bias"] = 0.1 * normal(c["N"]) if c["bias"] else None
        s["residual"] = None
        if c["residual"]:
            r = normal(M, c["N"])
            if c["out"] == "fp32":  # base parameters: positions on the grid, scales, rotation, amplitudes
                r[:, :2] = 512 * torch.rand(M, 2, generator=gen, device="cuda")
            s["residual"] = r.to(DTYPES[c["out"]])
        if c["op"] == "linear_bwd":
            s["dy"] = gradient(c["N"], c["out"])
    elif c["op"].startswith("gated"):
        s["x"], s["x_scale"] = rows(c["D"])
        s["wg"], s["wg_scale"] = _weight(gen, dt, c["F"], c["D"])
        s["wu"], s["wu_scale"] = _weight(gen, dt, c["F"], c["D"])
        if c["op"] == "gated_bwd":
            s["dh"] = gradient(c["F"], dt)
    else:
        x = normal(M, c["D"])
        x[:, ::97] *= 8  # a residual stream has a few loud channels
        s["x"] = x.to(DTYPES[dt])
        s["w"] = (1 + 0.1 * normal(c["D"])).to(DTYPES[dt])
        s["residual"] = normal(M, c["D"]).to(DTYPES[dt]) if c["residual"] else None
        if c["op"] == "rms_norm_bwd":
            s["dy"] = gradient(c["D"], dt)
            s["ds"] = gradient(c["D"], dt) if c["residual"] else None
    return s


def _act(z, act):
    """An activation and its derivative by elementary operations, in z's type."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if act == "silu":
        t = 1 / (1 + torch.exp(-z))
        return z * t, t * (1 + z * (1 - t))
    if act == "gelu":
        p = 0.5 * torch.erfc(-z * 2 ** -0.5)
        return z * p, p + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    a, b = (2 / math.pi) ** 0.5, 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def _wide(v, scale, f):
    return v.to(f) if scale is None else v.to(f) * scale.to(f)[:, None]


def _compute(s, f):
    """The operators from elementary operations on type f: {output: tensor of type f}."""
    c = s["case"]
    if c["op"].startswith("linear"):
        x, w = _wide(s["x"], s["x_scale"], f), _wide(s["w"], s["w_scale"], f)
        if c["op"] == "linear" or c["act"] != "none":
            z = x @ w.t()
            if s["bias"] is not None:
                z = z + s["bias"].to(f)
        if c["op"] == "linear":
            y = _act(z, c["act"])[0]
            return {"y": y if s["residual"] is None else y + s["residual"].to(f)}
        dz = s["dy"].to(f)
        if c["act"] != "none":
            dz = dz * _act(z, c["act"])[1]
        out = {"dx": dz @ w, "dw": dz.t() @ x}
        if s["bias"] is not None:
            out["db"] = dz.sum(0)
        return out
    if c["op"].startswith("gated"):
        x = _wide(s["x"], s["x_scale"], f)
        wg, wu = _wide(s["wg"], s["wg_scale"], f), _wide(s["wu"], s["wu_scale"], f)
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, c["act"])
        if c["op"] == "gated":
            return {"h": a * u}
        dh = s["dh"].to(f)
        du, dg = dh * a, dh * u * da
        return {"dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x}
    x, w = s["x"].to(f), s["w"].to(f)
    v = x if s["residual"] is None else x + s["residual"].to(f)
    if c["op"] == "rms_norm":
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w
        out = {}
        if c["out"] == "fp8":
            out["scale"] = (y.abs().amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
            out["y"] = (y / out["scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        else:
            out["y"] = y
        if s["residual"] is not None:
            out["s"] = v
        return out
    # The norm's input here is the stored sum, whichever way it came about.
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n, p = x * r, s["dy"].to(f) * w
    dx = r * (p - n * (p * n).mean(1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].to(f)
    return {"dx": dx, "dw": (s["dy"].to(f) * n).sum(0)}


def _types(c):
    """The types in which a case's outputs come."""
    t, o = DTYPES.get(c["dtype"]), DTYPES[c.get("out", "bf16" if c["dtype"] == "fp8" else c["dtype"])]
    return {"y": o, "s": t, "scale": torch.float32, "dx": t, "dw": t, "db": torch.float32, "h": o, "dwg": t, "dwu": t}


def run(state):
    s, c = state, state["case"]
    if not own:
        types = _types(c)
        return {k: v.to(types[k]) for k, v in _compute(s, torch.float32).items()}

    import differentiable_gaussian_splatting_pdr_b200 as pdr

    if c["op"] == "linear":
        return {"y": pdr.linear_fwd(s["x"], s["w"], s["bias"], s["residual"], activation=c["act"], out_dtype=DTYPES[c["out"]],
                                    x_scale=s["x_scale"], weight_scale=s["w_scale"])}
    if c["op"] == "linear_bwd":
        dx, dw, db = pdr.linear_bwd(s["dy"], s["x"], s["w"], s["bias"], activation=c["act"])
        return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "gated":
        return {"h": pdr.gated_fwd(s["x"], s["wg"], s["wu"], activation=c["act"], x_scale=s["x_scale"],
                                   gate_scale=s["wg_scale"], up_scale=s["wu_scale"])}
    if c["op"] == "gated_bwd":
        dx, dwg, dwu = pdr.gated_bwd(s["dh"], s["x"], s["wg"], s["wu"], activation=c["act"])
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    if c["op"] == "rms_norm":
        y, v, scale = pdr.rms_norm_fwd(s["x"], s["w"], s["residual"], eps=EPS, out_dtype=DTYPES[c["out"]])
        out = {"y": y}
        if scale is not None:
            out["scale"] = scale
        if s["residual"] is not None:
            out["s"] = v
        return out
    dx, dw = pdr.rms_norm_bwd(s["dy"], s["x"], s["w"], s["ds"], eps=EPS)
    return {"dx": dx, "dw": dw}


def _exact_act(z, act):
    """(value, derivative) in 64 bits, from the definitions by torch's special functions."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "silu":
        t = torch.special.expit(z)
        return z * t, t + z * t * torch.special.expit(-z)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # tanh form of gelu: (1 + tanh v) / 2 is the logistic function of 2 v
    v = math.sqrt(2 / math.pi) * z * (1 + 0.044715 * z.square())
    t = torch.special.expit(2 * v)
    return z * t, t + 2 * z * t * torch.special.expit(-2 * v) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z.square())


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if c["op"].startswith("linear"):
        if s["x_scale"] is None:
            z = torch.einsum("mk,nk->mn", d["x"], d["w"])
        else:
            z = torch.einsum("mk,nk->mn", d["x"], d["w"]) * d["x_scale"].unsqueeze(1) * d["w_scale"].unsqueeze(0)
        if "bias" in d:
            z += d["bias"]
        value, slope = _exact_act(z, c["act"])
        if c["op"] == "linear":
            return {"y": value + d["residual"] if "residual" in d else value}
        dz = slope * d["dy"]
        out = {"dx": torch.einsum("mn,nk->mk", dz, d["w"]), "dw": torch.einsum("mn,mk->nk", dz, d["x"])}
        if "bias" in d:
            out["db"] = torch.einsum("mn->n", dz)
        return out
    if c["op"].startswith("gated"):
        g, u = torch.einsum("md,fd->mf", d["x"], d["wg"]), torch.einsum("md,fd->mf", d["x"], d["wu"])
        if s["x_scale"] is not None:
            g = g * d["x_scale"].unsqueeze(1) * d["wg_scale"]
            u = u * d["x_scale"].unsqueeze(1) * d["wu_scale"]
        value, slope = _exact_act(g, c["act"])
        if c["op"] == "gated":
            return {"h": value * u}
        dg, du = d["dh"] * slope * u, d["dh"] * value
        both, weights = torch.cat([dg, du], 1), torch.cat([d["wg"], d["wu"]], 0)
        grads = torch.einsum("mf,md->fd", both, d["x"])
        return {"dx": both @ weights, "dwg": grads[:c["F"]], "dwu": grads[c["F"]:]}
    if c["op"] == "rms_norm":
        v = d["x"] + d["residual"] if "residual" in d else d["x"]
        y = v / torch.sqrt(v.square().sum(1, keepdim=True) / c["D"] + EPS) * d["w"]
        out = {"y": y}
        if c["out"] == "fp8":
            largest = y.abs().max(1).values
            out = {"scale": torch.maximum(largest / E4M3_MAX, torch.full_like(largest, MIN_SCALE)), "y": None}
            out["y"] = y / out["scale"].unsqueeze(1)
        if "residual" in d:
            out["s"] = v
        return out
    # d/dx of <dy, w x / |x|_rms>, with |x|_rms^2 = mean x^2 + eps, written out
    m = torch.sqrt(d["x"].square().sum(1, keepdim=True) / c["D"] + EPS)
    p = d["dy"] * d["w"]
    dx = p / m - d["x"] * (p * d["x"]).sum(1, keepdim=True) / (c["D"] * m ** 3)
    return {"dx": dx + d["ds"] if "ds" in d else dx, "dw": (d["dy"] * d["x"] / m).sum(0)}
