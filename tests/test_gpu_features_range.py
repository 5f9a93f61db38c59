"""linear, gated and rms_norm at the ends of their values' range, and over several
tiles a pair of SMs: against the formulas in fp64 on the GPU, element by element.

Tolerances, derived before the first run; u(t) is half a step of type t, relative to
the value (fp32 2^-24, fp16 2^-11, bf16 2^-8, e4m3 2^-4).
  sums      n additions, each off by at most a whole fp32 step: (n + 4) 2^-23 sum |a||b|.
  acts      |slope|, |curvature| <= 1.13; the evaluation adds 2^-18 |value| + 1.5e-7 |z| to the
            value and 2^-18 (1 + |z|) to the slope (the tails have tests of their own).
  dz, dg, du are rounded to x's type: u(t) of their size.  fp16 has half a step of 2^-25 below
            its normal range; the power of two that is taken out before brings the largest value
            that can occur, B, to 2^14 at least, so that this is 2^-39 B.  B is
            max |dy| for dz, and max |dh| D max |x| max |w| for dg and du.
  outputs   rounded once: u(t) of the value (fp16: 2^-25 at least).
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from differentiable_gaussian_splatting_pdr_b200 import build as pdr_build  # noqa: E402
from differentiable_gaussian_splatting_pdr_b200 import features as F  # noqa: E402

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, F16: 2.0 ** -25, BF16: 2.0 ** -134}
STEP, EVAL = 2.0 ** -23, 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pdr_build.build()
    yield
    torch.cuda.synchronize()
    F.check_wait_error()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(gen, shape, dtype, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float64)).to(dtype)


def f64(t):
    return None if t is None else t.detach().double()


def close(got, want, tol, dtype, what=""):
    got = f64(got)
    assert got.shape == want.shape, what
    assert torch.isfinite(want).all()
    limit = tol * (1 + U[dtype]) + U[dtype] * want.abs() + TINY[dtype]
    bad = ~((got - want).abs() <= limit)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), float((got - want)[bad].abs().max()),
                           float(limit[bad].min()))


def act(z, kind):
    """(value, slope) in fp64; the tail of the normal distribution without cancellation."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp_min(0), (z > 0).double()
    if kind == "silu":
        t = torch.special.expit(z)
        return z * t, t * (1 + z * torch.special.expit(-z))
    if kind == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.special.expit(2 * c * (z + 0.044715 * z ** 3))
    return z * t, t + 2 * z * t * (1 - t) * c * (1 + 3 * 0.044715 * z * z)


def z_error(x, w, b):
    return (x.shape[-1] + 6) * STEP * (x.abs() @ w.abs().t() + (0 if b is None else b.abs()))


def value_error(z, dz, kind):
    return dz if kind == "none" else 1.13 * dz + EVAL * act(z, kind)[0].abs() + 1.5e-7 * z.abs()


def slope_error(z, dz, kind):
    if kind == "none":
        return torch.zeros_like(z)
    if kind == "relu":
        return (z.abs() <= dz).double()
    return 1.13 * dz + EVAL * (1 + z.abs())


# ---- rows of zeros and rows near the smallest numbers -----------------------------


@pytest.mark.parametrize("dtype,wt", [(F32, F32), (BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("D", [1, 8, 64, 333, 512, 4096, 12296])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rms_norm_to_8_bits_of_zero_rows(D, dtype, wt, with_residual):
    gen = generator(D)
    M = 21
    zero = [0, 7, 8, M - 1]
    x, w = rand(gen, (M, D), dtype, 2.0), 1 + 0.1 * rand(gen, (D,), wt).abs()
    x[zero] = 0
    r = None
    if with_residual:
        r = rand(gen, (M, D), dtype)
        x[8] = -r[8]  # a sum of zero
        r[[0, 7, M - 1]] = 0
    q, s, scale = F.rms_norm_fwd(x, w, r, out_dtype=E4M3)
    q = q.float()
    assert torch.isfinite(q).all() and torch.isfinite(scale).all()
    assert not q[zero].any() and (scale[zero] == 2.0 ** -126).all()
    rest = [m for m in range(M) if m not in zero]
    y = F.rms_norm_fwd(x, w, r)[0]
    # the 8-bit rows are those of the norm in the rows' own type
    assert ((q * scale[:, None] - y.float()).abs()[rest] <= (2.0 ** -4 + 2 * U[dtype] + 1e-5) * y[rest].float().abs()
            + 2.0 ** -9 * scale[rest, None]).all()
    q, _, scale = F.rms_norm_fwd(rand(gen, (M, D), dtype, 0.01), torch.zeros_like(w), r, out_dtype=E4M3)
    assert not q.float().any() and (scale == 2.0 ** -126).all()


@pytest.mark.parametrize("size", [1e-30, 1e-34, 1e-36, 1e-37, 1e-38])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 333])
def test_rms_norm_to_8_bits_of_tiny_rows(D, dtype, size):
    """1 / scale alone is near the largest number here; rstd is 1000."""
    gen = generator(D)
    x, w = rand(gen, (10, D), dtype, size), 1 + 0.1 * rand(gen, (D,), F32)
    q, _, scale = F.rms_norm_fwd(x, w, out_dtype=E4M3)
    X, W = f64(x), f64(w)
    want = X / (X.square().mean(-1, keepdim=True) + 1e-6).sqrt() * W
    ws = (want.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    # products of tiny numbers are off by half of the smallest one, 2^-150, times rstd
    assert ((f64(scale) - ws).abs() <= 32 * STEP * ws + 1000 * 2.0 ** -149).all()
    err = (f64(q.float()) * f64(scale)[:, None] - want).abs()
    assert (err <= (2.0 ** -4 + 1e-5) * want.abs() + 2.0 ** -10 * 1.001 * f64(scale)[:, None] + 1000 * 2.0 ** -149).all()


def test_adapter_in_8_bits_with_a_row_of_zeros():
    """A padded token: its parameters are those that the formulas give for zeros, the others stay."""
    gen = generator(3)
    B, N, D, Fw, P = 2, 40, 64, 96, 8
    w = F.AdapterWeights(1 + 0.1 * rand(gen, (D,), BF16), rand(gen, (Fw, D), BF16, D ** -0.5), rand(gen, (Fw, D), BF16, D ** -0.5),
                         rand(gen, (D, Fw), BF16, 0.3 * Fw ** -0.5), 1 + 0.1 * rand(gen, (D,), BF16),
                         rand(gen, (P, D), BF16, 0.2 * D ** -0.5), rand(gen, (P,), F32, 0.1)).quantized()
    f, base = rand(gen, (B, N, D), BF16), rand(gen, (B, N, P), F32)
    whole = F.adapter(f, w, base)
    f[:, 30:] = 0
    y = F.adapter(f, w, base)
    assert torch.equal(y[:, :30], whole[:, :30])
    assert torch.equal(y[:, 30:], (w.head_bias + base)[:, 30:])


@pytest.mark.parametrize("dtype,wt", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("M", [1, 5, 33, 601])
@pytest.mark.parametrize("D", [1, 8, 64, 333, 512, 777, 1024, 4170])
def test_rms_norm_gradients_without_eps(M, D, dtype, wt):
    """eps = 0: threads behind the last row have a norm of zero there and add nothing."""
    gen = generator(M + D)
    s, w, g = rand(gen, (M, D), dtype, 2.0), rand(gen, (D,), wt), rand(gen, (M, D), dtype)
    s = torch.where(s == 0, torch.ones_like(s), s)
    gs = rand(gen, (M, D), dtype) if M % 2 else None
    dx, dw = F.rms_norm_bwd(g, s, w, gs, eps=0.0)
    S, W, G = f64(s), f64(w), f64(g)
    m = S.square().mean(-1, keepdim=True).sqrt()
    p = G * W
    wx = p / m - S * (p * S).mean(-1, keepdim=True) / m ** 3 + (0 if gs is None else f64(gs))
    size = p.abs() / m + S.abs() * (p * S).abs().mean(-1, keepdim=True) / m ** 3
    close(dx, wx, (D + 40) * STEP * size + STEP * wx.abs(), dtype, "dx")
    close(dw, (G * S / m).sum(0), (D / 2 + M + 40) * STEP * ((G * S).abs() / m).sum(0), wt, "dw")
    y = F.rms_norm_fwd(s, w, eps=0.0)[0]
    close(y, S / m * W, (D / 2 + 16) * STEP * (S / m * W).abs(), dtype, "y")


# ---- small and large gradients ------------------------------------------------------


def check_linear_bwd(M, K, N, dtype, gdt, kind, gs=1.0, xs=1.0, ws=None, bias_dtype=F32, seed=0):
    gen = generator(seed + M + K + N)
    x, w, g = rand(gen, (M, K), dtype, xs), rand(gen, (N, K), dtype, K ** -0.5 if ws is None else ws), rand(gen, (M, N), gdt, gs)
    b = rand(gen, (N,), bias_dtype)
    X, W, B, G = f64(x), f64(w), f64(b), f64(g)
    dx, dw, db = F.linear_bwd(g, x, w, b, kind)
    z = X @ W.t() + B
    slope = act(z, kind)[1]
    dz = G * slope
    e = G.abs() * slope_error(z, z_error(X, W, B), kind) + 2 * STEP * dz.abs()
    er = e + U[dtype] * (dz.abs() + e) + (2.0 ** -39 * G.abs().max() if dtype == F16 else 0)
    if kind == "none" and gdt == dtype:
        er = torch.zeros_like(dz)
    a = dz.abs() + er
    close(dx, dz @ W, er @ W.abs() + (N + 4) * STEP * (a @ W.abs()), dtype, "dx")
    close(dw, dz.t() @ X, er.t() @ X.abs() + (M + 100) * STEP * (a.t() @ X.abs()), dtype, "dw")
    close(db, dz.sum(0), e.sum(0) + (M + 100) * STEP * (dz.abs() + e).sum(0), bias_dtype, "db")
    return dx, dw, db


@pytest.mark.parametrize("gdt,size", [(F32, 1e-6), (F32, 1e-8), (F32, 1e-12), (F32, 1e-25), (BF16, 1e-7), (F32, 1.0), (F32, 3e6), (BF16, 3e6)])
@pytest.mark.parametrize("M,K,N", [(150, 64, 8), (150, 72, 6), (200, 77, 45), (130, 64, 40)])
def test_linear_fp16_gradients_of_any_size(M, K, N, gdt, size):
    """Gradients of a mean over pixels are far below fp16's smallest normal number; they keep their bits
    on the way to dx and dW.  x and W are such that dx and dW lie in fp16's range where that is possible."""
    scale = max(2.0 ** -13, min(100.0, 1e-2 / size))
    dx, dw, db = check_linear_bwd(M, K, N, F16, gdt, "none", size, xs=scale, ws=scale)
    assert db.abs().max() > 0
    if 1e-8 <= size:
        assert dx.abs().max() > 0 and dw.abs().max() > 0


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gdt,size", [(F32, 1e-7), (BF16, 1e-7), (F16, 2e-6), (F32, 3e6), (F16, 1.2e4)])
@pytest.mark.parametrize("M,K,N", [(200, 64, 40), (150, 77, 45)])
def test_linear_fp16_gradients_of_any_size_with_an_activation(M, K, N, gdt, size, kind):
    xs = 30.0 if size < 1 else 2.0 ** -13
    check_linear_bwd(M, K, N, F16, gdt, kind, size, xs=xs, ws=K ** -0.5 / xs if size < 1 else 2.0 ** -13)


@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_linear_fp16_gradients_of_zeros_and_infinities(kind):
    gen = generator(9)
    x, w, b = rand(gen, (300, 64), F16), rand(gen, (40, 64), F16, 0.1), rand(gen, (40,), F32)
    dx, dw, db = F.linear_bwd(torch.zeros(300, 40, device="cuda"), x, w, b, kind)
    assert not dx.any() and not dw.any() and not db.any()
    g = rand(gen, (300, 40), F32, 1e-3)
    clean = g.clone()
    clean[[7, 150]] = 0
    g[7, 3], g[150, 39] = float("inf"), float("nan")
    hit = torch.zeros(300, dtype=torch.bool, device="cuda")
    hit[[7, 150]] = True
    got, want = F.linear_bwd(g, x, w, b, kind), F.linear_bwd(clean, x, w, b, kind)
    # (a factor that differs by a power of two moves roundings 2^-39 of the largest value below)
    assert ((got[0] - want[0])[~hit].abs().double() <= U[F16] * want[0][~hit].abs().double() + TINY[F16] * 2).all()
    assert not torch.isfinite(got[0][hit]).any()
    cols = torch.ones(40, dtype=torch.bool, device="cuda")
    cols[[3, 39]] = False
    assert torch.isfinite(got[1][cols]).all() and not torch.isfinite(got[1][~cols]).any()


@pytest.mark.parametrize("dtype,size", [(BF16, 1.0), (BF16, 1e-6), (F16, 1.0), (F16, 1e-6)])
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (1000, 64, 8), (1000, 72, 6), (500, 77, 13), (300, 64, 32), (200, 520, 1), (40000, 40, 29),
                                   (700, 9, 5), (2, 20000, 30), (130, 1001, 9)])
def test_linear_gradients_of_few_columns_round_once(M, K, N, dtype, size):
    """Up to 32 columns of fp32 gradients (the parameters'): dz in two parts of 16 bits leaves u(t)^2 of
    it (and in fp16 a part's last bits, 2^-39 of the largest), and dx and dW have one rounding, their own."""
    gen = generator(M + K + N)
    x, w, g = rand(gen, (M, K), dtype, 50.0), rand(gen, (N, K), dtype, 50.0), rand(gen, (M, N), F32, size)
    X, W, G = f64(x), f64(w), f64(g)
    dx, dw, _ = F.linear_bwd(g, x, w)
    er = U[dtype] ** 2 * G.abs() + (2.0 ** -39 * G.abs().max() if dtype == F16 else 0)
    a = G.abs() + er
    close(dx, G @ W, er @ W.abs() + (2 * N + 4) * STEP * (a @ W.abs()), dtype, "dx")
    close(dw, G.t() @ X, er.t() @ X.abs() + (2 * M + 100) * STEP * (a.t() @ X.abs()), dtype, "dw")
    assert torch.equal(F.linear_bwd(g, x, w, need=(True, False, False))[0], dx)
    assert torch.equal(F.linear_bwd(g, x, w, need=(False, True, False))[1], dw)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_gradients_of_few_columns_keep_infinities(dtype):
    gen = generator(11)
    x, w, g = rand(gen, (300, 64), dtype), rand(gen, (8, 64), dtype), rand(gen, (300, 8), F32)
    clean = F.linear_bwd(g, x, w)
    g[7, 3], g[150, 5] = float("inf"), float("nan")
    dx, dw, _ = F.linear_bwd(g, x, w)
    assert torch.equal(dx[7].float(), w[3].float().sign() * float("inf")) and torch.isnan(dx[150]).all()
    rows = torch.ones(300, dtype=torch.bool, device="cuda")
    rows[[7, 150]] = False
    assert ((dx - clean[0]).abs()[rows].double() <= U[dtype] * clean[0][rows].abs().double() + 2 * TINY[dtype]).all()
    assert torch.equal(dw[3].float(), x[7].float().sign() * float("inf")) and torch.isnan(dw[5]).all()


def check_gated_bwd(M, D, Fw, dtype, kind, gs=1.0, xs=1.0, wgs=None, wus=None, seed=0):
    gen = generator(seed + M + D + Fw)
    x = rand(gen, (M, D), dtype, xs)
    wg, wu = (rand(gen, (Fw, D), dtype, D ** -0.5 if s is None else s) for s in (wgs, wus))
    dh = rand(gen, (M, Fw), dtype, gs)
    X, G, Up, H = f64(x), f64(wg), f64(wu), f64(dh)
    g, u = X @ G.t(), X @ Up.t()
    a, s = act(g, kind)
    eg, eu = z_error(X, G, None), z_error(X, Up, None)
    ea, es = value_error(g, eg, kind), slope_error(g, eg, kind)
    dx, dg, du = F.gated_bwd(dh, x, wg, wu, kind)
    DG, DU = H * u * s, H * a
    eG = H.abs() * (es * (u.abs() + eu) + s.abs() * eu) + 3 * STEP * DG.abs()
    eU = H.abs() * ea + 2 * STEP * DU.abs()
    low = 2.0 ** -39 * H.abs().max() * D * X.abs().max() * max(G.abs().max(), Up.abs().max()) if dtype == F16 else 0
    eG, eU = eG + U[dtype] * (DG.abs() + eG) + low, eU + U[dtype] * (DU.abs() + eU) + low
    aG, aU = DG.abs() + eG, DU.abs() + eU
    close(dx, DG @ G + DU @ Up, eG @ G.abs() + eU @ Up.abs() + (2 * Fw + 4) * STEP * (aG @ G.abs() + aU @ Up.abs()), dtype, "dx")
    close(dg, DG.t() @ X, eG.t() @ X.abs() + (M + 100) * STEP * (aG.t() @ X.abs()), dtype, "dwg")
    close(du, DU.t() @ X, eU.t() @ X.abs() + (M + 100) * STEP * (aU.t() @ X.abs()), dtype, "dwu")
    return dx, dg, du


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("M,D,Fw", [(150, 64, 40), (120, 72, 32), (200, 77, 45)])
def test_gated_fp16_gradients_of_any_size(M, D, Fw, kind):
    # dh of 32 of fp16's smallest steps, whose products with slopes lie below them
    dx, dg, du = check_gated_bwd(M, D, Fw, F16, kind, 2e-6, xs=16.0, wgs=D ** -0.5 / 16, wus=D ** -0.5 / 16)
    assert dg.abs().max() > 0
    # dg beyond fp16's largest number on the way to a dx and dW inside its range
    check_gated_bwd(M, D, Fw, F16, kind, 1.2e4, xs=2.0 ** -7, wgs=1e-3, wus=100.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["none", "silu"])
def test_gated_gradients_of_zeros(dtype, kind):
    """Features, weights or gradients that are all zero: every gradient is zero, or what the others give."""
    gen = generator(10)
    x, wg, wu, dh = rand(gen, (150, 64), dtype), rand(gen, (40, 64), dtype, 0.1), rand(gen, (40, 64), dtype, 0.1), rand(gen, (150, 40), dtype, 1e3)
    z = torch.zeros_like
    for args in [(dh, z(x), wg, wu), (dh, x, z(wg), z(wu)), (z(dh), x, wg, wu)]:
        assert not any(t.any() for t in F.gated_bwd(*args, kind))
    dx, dg, du = F.gated_bwd(dh, x, z(wg), wu, kind)
    assert torch.isfinite(dg).all() and not du.any() and (not dx.any() if kind == "silu" else True) and dg.any()


# ---- tails of the activations -----------------------------------------------------


def tail(z, kind):
    """Relative error that an activation may have: the exponent's argument is rounded."""
    a = {"silu": z.abs(), "gelu": z * z / 2, "gelu_tanh": 1.6 * z.abs() * (1 + 0.0448 * z * z)}[kind]
    return (16 + 4 * a) * STEP


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_activations_relative_to_their_value(kind, dtype):
    """fp32 results of z from -12 to 6 (one input, weight 1: z is exact): small values keep their bits.
    Factors below 2^-126 become 0, which moves the value by at most |z| 2^-126."""
    z = torch.linspace(-12, 6, 4001, device="cuda").to(dtype)[:, None].contiguous()
    z = torch.cat([z, (z[:2000] * 2.0 ** -10).contiguous()])
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    Z = f64(z)
    want = act(Z, kind)[0]
    for got in (F.linear_fwd(z, one, activation=kind, out_dtype=F32),
                F.gated_fwd(torch.cat([z, torch.ones_like(z)], 1), torch.tensor([[1.0, 0.0]], device="cuda").to(dtype),
                            torch.tensor([[0.0, 1.0]], device="cuda").to(dtype), kind, out_dtype=F32)):
        err = (f64(got) - want).abs()
        assert (err <= tail(Z, kind) * want.abs() + (1 + Z.abs()) * 2.0 ** -126).all(), (kind, float((err / want.abs().clamp_min(1e-300)).max()))


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_slopes_relative_to_their_terms(kind):
    z = torch.linspace(-9, 6, 3001, device="cuda").to(BF16)[:, None].contiguous()
    one = torch.ones(1, 1, device="cuda", dtype=BF16)
    Z = f64(z)
    dx = F.linear_bwd(torch.ones(3001, 1, device="cuda", dtype=BF16), z, one, None, kind, need=(True, False, False))[0]
    value, slope = act(Z, kind)
    terms = (value / Z.where(Z != 0, torch.ones_like(Z))).abs() + (slope - value / Z.where(Z != 0, torch.ones_like(Z))).abs()
    assert ((f64(dx) - slope).abs() <= 2.01 * U[BF16] * slope.abs() + 2 * tail(Z, kind) * terms + STEP * terms).all()


# ---- several tiles a pair of SMs ---------------------------------------------------

# B kept in shared memory (short k), and streamed.
MANY = [(20000, 64, 700), (20000, 1000, 700), (40000, 72, 600)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,D,Fw", MANY)
def test_gated_gradients_over_many_tiles(M, D, Fw, dtype):
    check_gated_bwd(M, D, Fw, dtype, "silu")


@pytest.mark.parametrize("dtype,gdt,kind", [(BF16, BF16, "gelu"), (F16, F32, "silu"), (BF16, F32, "none")])
@pytest.mark.parametrize("M,K,N", MANY)
def test_linear_gradients_over_many_tiles(M, K, N, dtype, gdt, kind):
    check_linear_bwd(M, K, N, dtype, gdt, kind)


@pytest.mark.parametrize("M,K,N", [(20000, 384, 700), (20000, 2048, 700), (30000, 100, 333)])
def test_8_bits_over_many_tiles(M, K, N):
    gen = generator(M + K + N)
    x, xs = F.quantize_rows(rand(gen, (M, K), BF16))
    (wg, gs), (wu, us) = (F.quantize_rows(rand(gen, (N, K), F32, K ** -0.5)) for _ in range(2))
    b, r = rand(gen, (N,), F32), rand(gen, (M, N), F32)
    X, G, Up = (f64(q.float()) * f64(s)[:, None] for q, s in [(x, xs), (wg, gs), (wu, us)])
    g, u = X @ G.t(), X @ Up.t()
    eg, eu = z_error(X, G, None) + 4 * STEP * g.abs(), z_error(X, Up, None) + 4 * STEP * u.abs()
    z, ez = g + f64(b), z_error(X, G, f64(b)) + 4 * STEP * g.abs()
    y = F.linear_fwd(x, wg, b, r, "gelu", F32, xs, gs)
    want = act(z, "gelu")[0] + f64(r)
    close(y, want, value_error(z, ez, "gelu") + STEP * (want.abs() + f64(r).abs()), F32, "y")
    a = act(g, "silu")[0]
    h = F.gated_fwd(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us)
    close(h, a * u, value_error(g, eg, "silu") * (u.abs() + eu) + a.abs() * eu + STEP * (a * u).abs(), BF16, "h")


# ---- replayed, and with given workspaces --------------------------------------------


def backward_calls(gen):
    x, w, wu, b = rand(gen, (333, 77), F16), rand(gen, (45, 77), F16, 0.1), rand(gen, (45, 77), F16, 0.1), rand(gen, (45,), F32)
    g32, g6, g16 = rand(gen, (333, 45), F32), rand(gen, (333, 6), F32), rand(gen, (333, 45), F16)
    head = w[:6].contiguous()
    calls = [lambda: F.linear_bwd(g32, x, w, b), lambda: F.linear_bwd(g6, x, head, b[:6].contiguous()), lambda: F.linear_bwd(g16, x, w, b, "silu"),
             lambda: F.linear_bwd(g32, x, w, b, "gelu"), lambda: F.gated_bwd(g16, x, w, wu)]
    return (g32, g6, g16), calls


def test_captured_gradients_fit_their_factor_to_each_replay():
    """The power of two comes from the gradients of the replay, not of the capture; two graphs share a pool."""
    grads, calls = backward_calls(generator(12))
    clean = [g.clone() for g in grads]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
            outs.append([t for c in calls for t in c()])
        graphs.append(graph)
    for size in (1.0, 2.0 ** -12, 2.0 ** 8):
        for g, c in zip(grads, clean):
            g.copy_(c * size)
        want = [t for c in calls for t in c()]
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            for a, e in zip(out, want):
                assert torch.equal(a, e)


def test_workspaces_full_of_nan_change_nothing():
    from differentiable_gaussian_splatting_pdr_b200 import _lib
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    gen = generator(13)
    ws = torch.empty(64 << 20, device="cuda", dtype=torch.uint8)
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    code = {F32: 0, F16: 1, BF16: 2}
    for M, K, N, dt, gdt, act_ in [(333, 77, 6, F16, F32, 0), (129, 64, 29, BF16, F32, 0), (70, 9, 1, F16, F32, 0), (200, 72, 40, F16, F16, 3),
                                   (200, 72, 45, F16, F32, 0), (100, 64, 33, F16, BF16, 2)]:
        x, w, b, g = rand(gen, (M, K), dt), rand(gen, (N, K), dt), rand(gen, (N,), F32), rand(gen, (M, N), gdt)
        want = F.linear_bwd(g, x, w, b, acts[act_])
        got = [torch.full_like(t, 7) for t in want]
        ws.fill_(255)
        assert lib.pdr_linear_bwd(g.data_ptr(), code[gdt], x.data_ptr(), w.data_ptr(), code[dt], b.data_ptr(), 0, act_, M, N, K,
                                  *(t.data_ptr() for t in got), ws.data_ptr(), ws.numel(), stream) == 0
        for a, e in zip(got, want):
            assert torch.equal(a, e)
        if gdt == dt:
            wu = rand(gen, (N, K), dt)
            want = F.gated_bwd(g, x, w, wu)
            got = [torch.full_like(t, 7) for t in want]
            ws.fill_(255)
            assert lib.pdr_gated_bwd(g.data_ptr(), x.data_ptr(), w.data_ptr(), wu.data_ptr(), code[dt], 2, M, K, N,
                                     *(t.data_ptr() for t in got), ws.data_ptr(), ws.numel(), stream) == 0
            for a, e in zip(got, want):
                assert torch.equal(a, e)
