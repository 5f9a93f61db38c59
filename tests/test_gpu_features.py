"""linear, gated, rms_norm and quantize_rows on the GPU against the fp64 oracle
(oracle/features.py), element by element.

Tolerances, derived before the first run.  u(t) is half a step of type t (fp32
2^-24, fp16 2^-11, bf16 2^-8, e4m3 2^-4), relative to the value; fp16 has an
absolute half step of 2^-25 below its normal range.
  sums      operands are exact in fp32 products; n additions, each off by at
            most a whole fp32 step (the tensor cores may truncate):
            |error| <= (n + 4) 2^-23 sum |a||b|.
  acts      |slope| <= 1.13, |curvature| <= 1.13 for all of them, so an error d of z
            becomes at most 1.13 d of the value and of the slope.  The evaluation adds at most
            2^-18 |value| + 1.5e-7 |z| (the exponential is good to 2 + 1.2 |x| steps,
            |x| <= 20 here; the normal distribution to 7.5e-8) to the value,
            2^-18 (1 + |z|) to the slope.  relu's slope may be either where |z| <= d.
  dz, dg, du rounded to x's type: u(t) of their size, carried through the products.
  outputs   rounded once: u(t) of the value.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from oracle import features as O  # noqa: E402
from differentiable_gaussian_splatting_pdr_b200 import build as pdr_build  # noqa: E402
from differentiable_gaussian_splatting_pdr_b200 import features as F  # noqa: E402

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 0.0, F16: 2.0 ** -25, BF16: 0.0}
STEP = 2.0 ** -23
EVAL = 2.0 ** -18
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pdr_build.build()
    yield
    torch.cuda.synchronize()
    F.check_wait_error()


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, tol, dtype, what=""):
    """Every element within tol + the rounding of its own type."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    limit = tol * (1 + U[dtype]) + U[dtype] * np.abs(want) + TINY[dtype]
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.abs(got - want)[bad].max()), float(limit[bad].min()))


def z_error(x, w, b):
    """Error bound of x W^T + b."""
    n = x.shape[-1]
    return (n + 6) * STEP * (np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b)))


def value_error(z, dz, kind):
    if kind == "none":
        return dz
    return 1.13 * dz + EVAL * np.abs(O.act(z, kind)[0]) + 1.5e-7 * np.abs(z)


def slope_error(z, dz, kind):
    if kind == "none":
        return np.zeros_like(z)
    if kind == "relu":
        return (np.abs(z) <= dz).astype(np.float64)
    return 1.13 * dz + EVAL * (1 + np.abs(z))


# rows x inputs x outputs: one of each; single tiles, edges of tiles, ragged, several tiles a block
SHAPES = [(1, 1, 1), (1, 64, 256), (3, 7, 5), (64, 128, 6), (127, 72, 31), (128, 64, 32), (129, 200, 33),
          (300, 264, 136), (513, 511, 257), (1000, 96, 1000), (20011, 40, 130)]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_shapes(M, K, N, dtype, out):
    rng = np.random.default_rng(M + K + N)
    x, w, b, r = rand(rng, (M, K), dtype), rand(rng, (N, K), dtype, K ** -0.5), rand(rng, (N,), F32), rand(rng, (M, N), out)
    y = F.linear_fwd(x, w, b, r, out_dtype=out)
    X, W, B, R = f64(x), f64(w), f64(b), f64(r)
    want = O.linear(X, W, B, R)
    close(y, want, z_error(X, W, B) + STEP * (np.abs(want) + np.abs(R)), out, "y")
    plain = F.linear_fwd(x, w, out_dtype=out)
    close(plain, O.linear(X, W), z_error(X, W, None), out, "no bias, no residual")


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("bias_dtype", [F32, BF16])
def test_linear_activations(kind, bias_dtype):
    rng = np.random.default_rng(5)
    x, w, b, r = rand(rng, (150, 96), BF16, 3.0), rand(rng, (140, 96), BF16, 0.1), rand(rng, (140,), bias_dtype), rand(rng, (150, 140), F32)
    X, W, B, R = f64(x), f64(w), f64(b), f64(r)
    z, d = X @ W.T + B, z_error(X, W, B)
    assert np.abs(z).max() < 20
    y = F.linear_fwd(x, w, b, r, activation=kind, out_dtype=F32)
    want = O.linear(X, W, B, R, kind)
    close(y, want, value_error(z, d, kind) + STEP * (np.abs(want) + np.abs(R)), F32, "y")


@pytest.mark.parametrize("M,K,N", [(1, 16, 1), (50, 77, 100), (129, 128, 40), (1000, 512, 333)])
@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_linear_in_8_bits(M, K, N, kind):
    rng = np.random.default_rng(M + K)
    x, xs = F.quantize_rows(rand(rng, (M, K), BF16))
    w, ws = F.quantize_rows(rand(rng, (N, K), F32, K ** -0.5))
    b = rand(rng, (N,), F32)
    X, W = f64(x.float()) * f64(xs)[:, None], f64(w.float()) * f64(ws)[:, None]
    z, d = X @ W.T + f64(b), z_error(X, W, f64(b)) + 4 * STEP * np.abs(X @ W.T)
    y = F.linear_fwd(x, w, b, activation=kind, x_scale=xs, weight_scale=ws, out_dtype=F32)
    close(y, O.act(z, kind)[0], value_error(z, d, kind), F32, "y")
    assert F.linear_fwd(x, w, b, x_scale=xs, weight_scale=ws).dtype == BF16


def check_linear_bwd(M, K, N, dtype, gdt, kind, bias_dtype=F32, seed=0):
    rng = np.random.default_rng(seed + M + K + N)
    x, w, g = rand(rng, (M, K), dtype), rand(rng, (N, K), dtype, K ** -0.5), rand(rng, (M, N), gdt)
    b = None if bias_dtype is None else rand(rng, (N,), bias_dtype)
    X, W, B, G = f64(x), f64(w), f64(b), f64(g)
    dx, dw, db = F.linear_bwd(g, x, w, b, kind)
    z = X @ W.T + (0 if B is None else B)
    slope = O.act(z, kind)[1]
    dz = G * slope
    e = np.abs(G) * slope_error(z, z_error(X, W, B), kind) + 2 * STEP * np.abs(dz)  # before rounding
    er = e + U[dtype] * (np.abs(dz) + e) + TINY[dtype]
    if kind == "none" and gdt == dtype:
        er = np.zeros_like(dz)
    wx, ww, wb = O.linear_bwd(G, X, W, B, kind)
    a = np.abs(dz) + er
    close(dx, wx, er @ np.abs(W) + (N + 4) * STEP * (a @ np.abs(W)), dtype, "dx")
    close(dw, ww, er.T @ np.abs(X) + (M + 100) * STEP * (a.T @ np.abs(X)), dtype, "dw")
    if b is not None:
        close(db, wb, e.sum(0) + (M + 100) * STEP * (np.abs(dz) + e).sum(0), bias_dtype, "db")
    else:
        assert db is None


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (5, 9, 3), (64, 128, 6), (130, 66, 40), (300, 264, 136), (777, 130, 257), (4099, 72, 13)])
@pytest.mark.parametrize("dtype,gdt,kind", [(BF16, F32, "none"), (F16, F16, "none"), (BF16, BF16, "gelu"), (F16, F32, "silu")])
def test_linear_gradients(M, K, N, dtype, gdt, kind):
    check_linear_bwd(M, K, N, dtype, gdt, kind)


@pytest.mark.parametrize("kind", ACTS)
def test_linear_gradients_of_each_activation(kind):
    check_linear_bwd(200, 64, 72, BF16, BF16, kind, bias_dtype=BF16)
    check_linear_bwd(200, 64, 72, F16, BF16, kind, bias_dtype=None)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M,D,Fw", [(1, 1, 1), (1, 512, 300), (37, 72, 31), (128, 64, 32), (129, 200, 130), (700, 129, 257)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated(M, D, Fw, dtype, kind):
    rng = np.random.default_rng(M + D + Fw)
    x, wg, wu = rand(rng, (M, D), dtype), rand(rng, (Fw, D), dtype, D ** -0.5), rand(rng, (Fw, D), dtype, D ** -0.5)
    X, G, Up = f64(x), f64(wg), f64(wu)
    g, u = X @ G.T, X @ Up.T
    a, s = O.act(g, kind)
    eg, eu = z_error(X, G, None), z_error(X, Up, None)
    ea, es = value_error(g, eg, kind), slope_error(g, eg, kind)
    h = F.gated_fwd(x, wg, wu, kind)
    want = O.gated(X, G, Up, kind)
    close(h, want, ea * (np.abs(u) + eu) + np.abs(a) * eu + STEP * np.abs(want), dtype, "h")

    dh = rand(rng, (M, Fw), dtype)
    H = f64(dh)
    dx, dg, du = F.gated_bwd(dh, x, wg, wu, kind)
    DG, DU = H * u * s, H * a
    eG = np.abs(H) * (es * (np.abs(u) + eu) + np.abs(s) * eu) + 3 * STEP * np.abs(DG)
    eU = np.abs(H) * ea + 2 * STEP * np.abs(DU)
    eG, eU = eG + U[dtype] * (np.abs(DG) + eG) + TINY[dtype], eU + U[dtype] * (np.abs(DU) + eU) + TINY[dtype]
    wx, wwg, wwu = O.gated_bwd(H, X, G, Up, kind)
    aG, aU = np.abs(DG) + eG, np.abs(DU) + eU
    close(dx, wx, eG @ np.abs(G) + eU @ np.abs(Up) + (2 * Fw + 4) * STEP * (aG @ np.abs(G) + aU @ np.abs(Up)), dtype, "dx")
    close(dg, wwg, eG.T @ np.abs(X) + (M + 100) * STEP * (aG.T @ np.abs(X)), dtype, "dwg")
    close(du, wwu, eU.T @ np.abs(X) + (M + 100) * STEP * (aU.T @ np.abs(X)), dtype, "dwu")


@pytest.mark.parametrize("M,D,Fw", [(1, 16, 1), (60, 77, 100), (1000, 256, 333)])
def test_gated_in_8_bits(M, D, Fw):
    rng = np.random.default_rng(M + D)
    (x, xs), (wg, gs), (wu, us) = (F.quantize_rows(rand(rng, s, F32, c)) for s, c in
                                   [((M, D), 1.0), ((Fw, D), D ** -0.5), ((Fw, D), D ** -0.5)])
    X, G, Up = (f64(q.float()) * f64(s)[:, None] for q, s in [(x, xs), (wg, gs), (wu, us)])
    g, u = X @ G.T, X @ Up.T
    eg, eu = z_error(X, G, None) + 4 * STEP * np.abs(g), z_error(X, Up, None) + 4 * STEP * np.abs(u)
    a = O.act(g, "silu")[0]
    h = F.gated_fwd(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us, out_dtype=F32)
    close(h, a * u, value_error(g, eg, "silu") * (np.abs(u) + eu) + np.abs(a) * eu + STEP * np.abs(a * u), F32, "h")


NORM_SHAPES = [(1, 1), (1, 4096), (7, 3), (33, 16), (100, 64), (65, 333), (50, 512), (20, 1000), (9, 2056), (5, 8192), (3, 16384), (3000, 48)]


@pytest.mark.parametrize("dtype,wt", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("M,D", NORM_SHAPES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_rms_norm(M, D, dtype, wt, with_residual):
    rng = np.random.default_rng(M + D)
    x, w = rand(rng, (M, D), dtype, 2.0), rand(rng, (D,), wt)
    r = rand(rng, (M, D), dtype) if with_residual else None
    X, W, R = f64(x), f64(w), f64(r)
    y, s, scale = F.rms_norm_fwd(x, w, r)
    assert scale is None
    wy, wsum = O.rms_norm(X, W, R)
    # the row's sum of squares, its root and two products: within (D + 16) / 2 steps, relative
    rel = (D / 2 + 16) * STEP
    absx = np.abs(X) + (0 if R is None else np.abs(R))
    m = np.abs(wy) / np.maximum(np.abs(wsum), 1e-300)
    close(y, wy, rel * np.abs(wy) + U[F32] * absx * np.nan_to_num(m), dtype, "y")
    if with_residual:
        close(s, wsum, U[F32] * np.abs(wsum), dtype, "s")
    else:
        assert s is x

    q, s8, scale = F.rms_norm_fwd(x, w, r, out_dtype=E4M3)
    assert scale.shape == (M,) and (not with_residual or torch.equal(s8, s))
    assert np.allclose(f64(scale), O.row_scales(wy), rtol=rel + 8 * STEP, atol=0)
    err = np.abs(f64(q.float()) * f64(scale)[:, None] - wy)
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its normal range
    assert (err <= (2.0 ** -4 + 2 * rel + 1e-6) * np.abs(wy) + 2.0 ** -10 * f64(scale)[:, None] * 1.001
            + U[F32] * absx * np.nan_to_num(m)).all()


@pytest.mark.parametrize("dtype,wt", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("M,D", NORM_SHAPES)
@pytest.mark.parametrize("with_sum", [False, True])
def test_rms_norm_gradients(M, D, dtype, wt, with_sum):
    rng = np.random.default_rng(M + D + 1)
    s, w, g = rand(rng, (M, D), dtype, 2.0), rand(rng, (D,), wt), rand(rng, (M, D), dtype)
    gs = rand(rng, (M, D), dtype) if with_sum else None
    S, W, G, GS = f64(s), f64(w), f64(g), f64(gs)
    dx, dw = F.rms_norm_bwd(g, s, w, gs)
    wx, ww = O.rms_norm_bwd(G, S, W, GS)
    m = np.sqrt((S * S).mean(-1, keepdims=True) + 1e-6)
    rel = (D + 40) * STEP
    p = np.abs(G * W)
    size = p / m + np.abs(S) * (p * np.abs(S)).mean(-1, keepdims=True) / m ** 3
    close(dx, wx, rel * size + STEP * np.abs(wx), dtype, "dx")
    close(dw, ww, ((D / 2 + M + 40) * STEP) * (np.abs(G * S) / m).sum(0), wt, "dw")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_rows(dtype):
    rng = np.random.default_rng(8)
    x = rand(rng, (40, 200), dtype, 5.0)
    x[3] = 0
    x[4, 1:] = 0
    q, scale = F.quantize_rows(x)
    X = f64(x)
    assert np.allclose(f64(scale), O.row_scales(X), rtol=4 * STEP, atol=0)
    back = f64(q.float()) * f64(scale)[:, None]
    assert (np.abs(back - X) <= (2.0 ** -4 + 1e-6) * np.abs(X) + 2.0 ** -10 * 1.001 * f64(scale)[:, None]).all()
    assert (back[3] == 0).all() and f64(scale)[3] == 2.0 ** -126
    assert abs(back[4, 0] - X[4, 0]) <= 8 * STEP * abs(X[4, 0])  # the largest value is 448 scales


def test_no_rows():
    w, b, n = torch.randn(6, 32, device="cuda", dtype=BF16), torch.randn(6, device="cuda"), torch.randn(32, device="cuda", dtype=BF16)
    x = torch.empty(0, 32, device="cuda", dtype=BF16)
    assert F.linear_fwd(x, w, b).shape == (0, 6) and F.gated_fwd(x, w, w).shape == (0, 6)
    dx, dw, db = F.linear_bwd(x.new_empty(0, 6), x, w, b, "gelu")
    assert dx.shape == (0, 32) and not dw.any() and not db.any()
    dx, dg, du = F.gated_bwd(x.new_empty(0, 6), x, w, w)
    assert dx.shape == (0, 32) and not dg.any() and not du.any()
    assert F.rms_norm_fwd(x, n)[0].shape == (0, 32)
    dx, dw = F.rms_norm_bwd(x, x, n)
    assert not dw.any()
    assert F.quantize_rows(x)[0].shape == (0, 32)


def test_leading_dimensions_and_given_output():
    rng = np.random.default_rng(9)
    x, w, wu = rand(rng, (2, 3, 50, 64), BF16), rand(rng, (40, 64), BF16), rand(rng, (40, 64), BF16)
    y = F.linear_fwd(x, w)
    assert y.shape == (2, 3, 50, 40)
    assert torch.equal(y.view(-1, 40), F.linear_fwd(x.view(-1, 64), w))
    out = torch.empty(2, 3, 50, 40, device="cuda", dtype=BF16)
    assert F.linear_fwd(x, w, out=out) is out and torch.equal(out, y)
    assert F.gated_fwd(x, w, wu, out=out) is out and torch.equal(out, F.gated_fwd(x, w, wu))
    n, _, sc = F.rms_norm_fwd(x, w[0].contiguous(), out_dtype=E4M3)
    assert n.shape == x.shape and sc.shape == (2, 3, 50)


@pytest.mark.parametrize("N", [40, 41, 8])
def test_rows_behind_the_last_stay_as_they_were(N):
    """Outputs live in larger buffers; what lies behind them is not touched."""
    rng = np.random.default_rng(10)
    M, K = 131, 64
    x, w, wu = rand(rng, (M, K), F16), rand(rng, (N, K), F16), rand(rng, (N, K), F16)
    for call, dt in [(lambda o: F.linear_fwd(x, w, out=o), F16), (lambda o: F.gated_fwd(x, w, wu, out=o), F16),
                     (lambda o: F.linear_fwd(x, w, out=o, out_dtype=F32), F32)]:
        buf = torch.full((M * N + 4096,), 7.0, device="cuda", dtype=dt)
        call(buf[:M * N].view(M, N))
        assert (buf[M * N:] == 7).all()


@pytest.mark.parametrize("shift", [1, 3, 8])
def test_tensors_at_odd_addresses(shift):
    """Slices of a buffer that start anywhere give the bits of aligned ones."""
    rng = np.random.default_rng(11)
    M, K, N = 70, 64, 48

    def moved(t):
        buf = torch.empty(t.numel() + 16, device="cuda", dtype=t.dtype)
        v = buf[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    x, w, wu, g, b, r = (rand(rng, s, BF16) for s in [(M, K), (N, K), (N, K), (M, N), (N,), (M, N)])
    want = F.linear_fwd(x, w, b, r, "gelu")
    out = moved(torch.zeros_like(want))
    assert torch.equal(F.linear_fwd(moved(x), moved(w), moved(b), moved(r), "gelu", out=out), want)
    for a, e in zip(F.linear_bwd(moved(g), moved(x), moved(w), moved(b), "gelu"), F.linear_bwd(g, x, w, b, "gelu")):
        assert torch.equal(a, e)
    assert torch.equal(F.gated_fwd(moved(x), moved(w), moved(wu)), F.gated_fwd(x, w, wu))
    for a, e in zip(F.gated_bwd(moved(g), moved(x), moved(w), moved(wu)), F.gated_bwd(g, x, w, wu)):
        assert torch.equal(a, e)
    n, n2 = x[0].contiguous(), rand(rng, (M, K), BF16)
    for dt in (BF16, E4M3):
        got, want = F.rms_norm_fwd(moved(x), moved(n), moved(n2), out_dtype=dt), F.rms_norm_fwd(x, n, n2, out_dtype=dt)
        assert torch.equal(got[1], want[1])
        # the order of a row's sum differs with the alignment: the last bit may
        assert (got[0].float() - want[0].float()).abs().max() <= (2.0 ** -7 if dt == BF16 else 2.0 ** -3) * want[0].float().abs().max()


def test_non_finite_values_stay_in_their_rows():
    rng = np.random.default_rng(12)
    x, w, wu = rand(rng, (200, 72), BF16), rand(rng, (50, 72), BF16), rand(rng, (50, 72), BF16)
    x[7, 3], x[130, 0], x[199, 71] = float("nan"), float("inf"), float("-inf")
    hit = torch.zeros(200, dtype=torch.bool, device="cuda")
    hit[[7, 130, 199]] = True
    clean = torch.where(hit[:, None], torch.zeros_like(x), x)
    for kind in ACTS:
        for f in (lambda v: F.linear_fwd(v, w, activation=kind), lambda v: F.gated_fwd(v, w, wu, kind)):
            y, ref = f(x), f(clean)
            assert torch.equal(y[~hit], ref[~hit])
            assert torch.isnan(y[7]).all()
    y, _, scale = F.rms_norm_fwd(x, w[0].contiguous(), out_dtype=E4M3)
    assert not torch.isfinite(scale[hit]).any() and torch.isfinite(scale[~hit]).all()
    q, scale = F.quantize_rows(x)
    assert torch.isnan(scale[7]) and torch.isinf(scale[130]) and torch.isfinite(scale[~hit]).all()


def test_non_finite_weights_stay_in_their_columns():
    rng = np.random.default_rng(34)
    x, w, wu = rand(rng, (300, 72), F16), rand(rng, (70, 72), F16), rand(rng, (70, 72), F16)
    bad = w.clone()
    bad[5, 3], bad[64, 0] = float("nan"), float("inf")
    hit = torch.zeros(70, dtype=torch.bool, device="cuda")
    hit[[5, 64]] = True
    for kind in ACTS:
        for a, b in [(F.linear_fwd(x, bad, activation=kind), F.linear_fwd(x, w, activation=kind)),
                     (F.gated_fwd(x, bad, wu, kind), F.gated_fwd(x, w, wu, kind)),
                     (F.gated_fwd(x, wu, bad, kind), F.gated_fwd(x, wu, w, kind))]:
            assert torch.equal(a[:, ~hit], b[:, ~hit]) and torch.isnan(a[:, 5]).all()


def test_vectors_are_single_rows():
    rng = np.random.default_rng(35)
    x, w, wu, b, n = (rand(rng, s, BF16) for s in [(40,), (24, 40), (24, 40), (24,), (40,)])
    assert torch.equal(F.linear_fwd(x, w, b), F.linear_fwd(x[None], w, b)[0])
    assert torch.equal(F.gated_fwd(x, w, wu), F.gated_fwd(x[None], w, wu)[0])
    assert torch.equal(F.rms_norm_fwd(x, n, x)[0], F.rms_norm_fwd(x[None], n, x[None])[0][0])
    q, sc = F.quantize_rows(x)
    assert q.shape == (40,) and sc.shape == ()
    for a, e in zip(F.linear_bwd(b, x, w, b, "silu"), F.linear_bwd(b[None], x[None], w, b, "silu")):
        assert torch.equal(a, e.view(a.shape))


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(13)
    x, w, wu, b, g = (rand(rng, s, BF16) for s in [(5000, 136), (96, 136), (96, 136), (96,), (5000, 96)])
    n = rand(rng, (136,), F32)
    calls = [lambda: (F.linear_fwd(x, w, b, activation="gelu"),), lambda: F.linear_bwd(g, x, w, b, "gelu"),
             lambda: F.linear_bwd(g, x, w, b), lambda: (F.gated_fwd(x, w, wu),), lambda: F.gated_bwd(g, x, w, wu),
             lambda: F.rms_norm_fwd(x, n, x)[:2], lambda: F.rms_norm_bwd(x, x, n, x)]
    for call in calls:
        first = call()
        for _ in range(3):
            for a, e in zip(call(), first):
                assert torch.equal(a, e)


def test_partial_gradients_equal_the_whole():
    rng = np.random.default_rng(14)
    x, w, wu, b, g = (rand(rng, s, F16) for s in [(333, 77), (90, 77), (90, 77), (90,), (333, 90)])
    for kind in ("none", "silu"):
        full = F.linear_bwd(g, x, w, b, kind)
        for i in range(3):
            need = tuple(j == i for j in range(3))
            part = F.linear_bwd(g, x, w, b, kind, need)
            assert all((p is None) == (j != i) for j, p in enumerate(part)) and torch.equal(part[i], full[i])
        assert F.linear_bwd(g, x, w, b, kind, (False, False, False)) == (None, None, None)
    full = F.gated_bwd(g, x, w, wu)
    assert torch.equal(F.gated_bwd(g, x, w, wu, need=(True, False))[0], full[0])
    part = F.gated_bwd(g, x, w, wu, need=(False, True))
    assert part[0] is None and torch.equal(part[1], full[1]) and torch.equal(part[2], full[2])
    n = x[0].contiguous()
    dx, dw = F.rms_norm_bwd(x, x, n)
    assert torch.equal(F.rms_norm_bwd(x, x, n, need=(True, False))[0], dx)
    assert torch.equal(F.rms_norm_bwd(x, x, n, need=(False, True))[1], dw)


def test_long_outputs_past_32_bit_offsets():
    """More than 2^31 output elements: the last rows are right."""
    M, K, N = (1 << 22) + 300, 32, 520
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, device="cuda", dtype=BF16, generator=gen)
    w = torch.randn(N, K, device="cuda", dtype=BF16, generator=gen)
    assert M * N > 2 ** 31
    tail = slice(M - 400, M)
    y = F.linear_fwd(x, w)
    assert torch.equal(y[tail], F.linear_fwd(x[tail].contiguous(), w))
    assert torch.equal(F.gated_fwd(x, w, w)[tail], F.gated_fwd(x[tail].contiguous(), w, w))
    n = torch.ones(N, device="cuda", dtype=BF16)
    assert torch.equal(F.rms_norm_fwd(y, n)[0][tail], F.rms_norm_fwd(y[tail].contiguous(), n)[0])
    dx = F.linear_bwd(y, x, w, need=(True, False, False))[0]
    assert torch.equal(dx[tail], F.linear_bwd(y[tail].contiguous(), x[tail].contiguous(), w, need=(True, False, False))[0])


def test_streams_and_concurrent_calls():
    rng = np.random.default_rng(15)
    xs = [rand(rng, (3000 + i, 128), BF16) for i in range(4)]
    w, wu = rand(rng, (256, 128), BF16), rand(rng, (256, 128), BF16)
    g = [rand(rng, (3000 + i, 256), BF16) for i in range(4)]
    want = [(F.linear_fwd(x, w, activation="gelu"), *F.gated_bwd(d, x, w, wu)) for x, d in zip(xs, g)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x, d in zip(streams, xs, g):
        with torch.cuda.stream(s):
            got.append((F.linear_fwd(x, w, activation="gelu"), *F.gated_bwd(d, x, w, wu)))
    torch.cuda.synchronize()
    for a, e in zip(got, want):
        for p, q in zip(a, e):
            assert torch.equal(p, q)


def test_captured_and_replayed():
    rng = np.random.default_rng(16)
    x, g = rand(rng, (700, 100), BF16), rand(rng, (700, 90), BF16)
    w, wu, b, n = rand(rng, (90, 100), BF16), rand(rng, (90, 100), BF16), rand(rng, (90,), F32), rand(rng, (100,), F32)

    def step():
        y, s, sc = F.rms_norm_fwd(x, n, x)
        return (y, s, F.gated_fwd(y, w, wu), F.linear_fwd(y, w, b, activation="silu"), *F.gated_bwd(g, y, w, wu),
                *F.linear_bwd(g, y, w, b, "silu"), *F.rms_norm_bwd(y, s, n))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):  # two graphs of one memory pool
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
            outs.append(step())
        graphs.append(graph)
    for seed in range(2):
        x.copy_(rand(np.random.default_rng(seed), (700, 100), BF16))
        want = step()
        for graph, out in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            for a, e in zip(out, want):
                assert torch.equal(a, e)


def test_refusals():
    x, w = torch.randn(4, 64, device="cuda", dtype=BF16), torch.randn(8, 64, device="cuda", dtype=BF16)
    b = torch.randn(8, device="cuda")
    q, sc = F.quantize_rows(x)
    wq, wsc = F.quantize_rows(w)
    bad = [lambda: F.linear_fwd(x.float(), w.float()), lambda: F.linear_fwd(x, w.half()), lambda: F.linear_fwd(x, w[:, :32].contiguous()),
           lambda: F.linear_fwd(x, w.t()), lambda: F.linear_fwd(x[:, ::2], w), lambda: F.linear_fwd(x, w, b[:4]),
           lambda: F.linear_fwd(x, w, residual=x), lambda: F.linear_fwd(x, w, residual=x[:, :8].float().contiguous()),
           lambda: F.linear_fwd(x, w, residual=x[:1, :8].contiguous()), lambda: F.linear_fwd(x, w, out_dtype=torch.float64),
           lambda: F.linear_fwd(x, w, out=torch.empty(4, 7, device="cuda", dtype=BF16)), lambda: F.linear_fwd(x, w, x_scale=sc),
           lambda: F.linear_fwd(q, wq), lambda: F.linear_fwd(q, wq, x_scale=sc[:2], weight_scale=wsc),
           lambda: F.linear_fwd(q, wq, x_scale=sc, weight_scale=wsc[:2]), lambda: F.linear_fwd(q, w, x_scale=sc),
           lambda: F.linear_bwd(x, x, w), lambda: F.linear_bwd(x[:, :8].contiguous(), q, wq), lambda: F.linear_fwd(x, w.cpu()),
           lambda: F.gated_fwd(x, w, w[:4].contiguous()), lambda: F.gated_fwd(x, w, w.half()), lambda: F.gated_fwd(q, wq, wq, x_scale=sc),
           lambda: F.gated_bwd(x[:, :8].float().contiguous(), x, w, w), lambda: F.rms_norm_fwd(x, b), lambda: F.rms_norm_fwd(x, w[0].half()),
           lambda: F.rms_norm_fwd(x, w[0], x.float()), lambda: F.rms_norm_fwd(x, w[0], out_dtype=F32),
           lambda: F.rms_norm_bwd(x.float(), x, w[0]), lambda: F.rms_norm_bwd(x[:2], x, w[0]), lambda: F.quantize_rows(q),
           lambda: F.rms_norm_fwd(x, w[0], x[:2])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    from differentiable_gaussian_splatting_pdr_b200._lib import PdrError
    wide = torch.zeros(1, 16385, device="cuda")
    with pytest.raises(PdrError, match="TOO_LARGE"):
        F.rms_norm_fwd(wide, wide[0])
    with pytest.raises(PdrError, match="INVALID"):
        F.rms_norm_fwd(wide[:, :64].contiguous(), wide[0, :64], eps=-1.0)


def _weights(rng, D, Fw, P, dtype):
    w = F.AdapterWeights(norm_in=1 + 0.1 * rand(rng, (D,), dtype), gate=rand(rng, (Fw, D), dtype, D ** -0.5),
                         up=rand(rng, (Fw, D), dtype, D ** -0.5), down=rand(rng, (D, Fw), dtype, 0.3 * Fw ** -0.5),
                         norm_out=1 + 0.1 * rand(rng, (D,), dtype), head=rand(rng, (P, D), dtype, 0.2 * D ** -0.5),
                         head_bias=rand(rng, (P,), F32, 0.1))
    return w


def _adapter64(f, w, base, update=None):
    """The adapter in fp64 torch operations, differentiable."""
    def norm(v, g):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * g
    s = f if update is None else f + update
    n = norm(s, w["norm_in"])
    h = torch.nn.functional.silu(n @ w["gate"].t()) * (n @ w["up"].t())
    t = h @ w["down"].t() + s
    return norm(t, w["norm_out"]) @ w["head"].t() + w["head_bias"] + base


NAMES = ["norm_in", "gate", "up", "down", "norm_out", "head", "head_bias"]


@pytest.mark.parametrize("dtype,D,Fw,update", [(BF16, 64, 128, False), (F16, 72, 100, True), (BF16, 50, 66, True)])
def test_adapter_gradients(dtype, D, Fw, update):
    """norm -> gated -> linear + residual -> norm -> head, trained: against fp64 autograd of the same formulas.

    Each of at most 12 roundings to x's type on the way to a gradient is off by at most
    u(t) of a value, at random and hence less in the norm; 12 u(t) bounds the relative error."""
    rng = np.random.default_rng(20)
    B, N, P = 2, 70, 8
    w = _weights(rng, D, Fw, P, dtype)
    f, base, g = rand(rng, (B, N, D), dtype), rand(rng, (B, N, P), F32), rand(rng, (B, N, P), F32)
    up = rand(rng, (B, N, D), dtype, 0.5) if update else None
    leaves = [f, base] + ([up] if update else []) + [getattr(w, n) for n in NAMES]
    for t in leaves:
        t.requires_grad_(True)
    y = F.adapter(f, w, base, up)
    assert y.dtype == F32 and y.shape == (B, N, P)
    grads = torch.autograd.grad(y, leaves, g)
    leaves64 = [t.detach().double().requires_grad_(True) for t in leaves]
    k = 3 if update else 2
    y64 = _adapter64(leaves64[0], dict(zip(NAMES, leaves64[k:])), leaves64[1], leaves64[2] if update else None)
    grads64 = torch.autograd.grad(y64, leaves64, g.double())
    assert (y.double() - y64).norm() <= 12 * U[dtype] * y64.norm()
    for a, e, t in zip(grads, grads64, leaves):
        assert a.dtype == t.dtype and a.shape == t.shape
        assert (a.double() - e).norm() <= 12 * U[dtype] * e.norm()


def test_adapter_feeds_the_renderer_and_its_loss():
    """Features to image to loss and back: every weight gets the gradient that the parts' chain gives."""
    from differentiable_gaussian_splatting_pdr_b200 import l1_ssim, render, render_bwd, l1_ssim_loss, render_fwd
    rng = np.random.default_rng(21)
    B, N, C, H, W, D = 2, 256, 3, 48, 40, 64
    w = _weights(rng, D, 96, 5 + C, BF16)
    f = rand(rng, (B, N, D), BF16)
    base = torch.zeros(B, N, 5 + C)
    base[..., 0] = torch.from_numpy(rng.uniform(0, W, (B, N)))
    base[..., 1] = torch.from_numpy(rng.uniform(0, H, (B, N)))
    base = base.cuda()
    target = torch.rand(B, C, H, W, device="cuda")
    for n in NAMES:
        getattr(w, n).requires_grad_(True)
    params = F.adapter(f, w, base)
    image = render(params, H, W, 7)
    loss = l1_ssim(image, target)
    loss.backward()
    want = oracle.render_fwd(params.detach().cpu().numpy(), H, W, 7)
    assert np.abs(image.detach().cpu().numpy() - want).max() <= 1e-5 * np.abs(want).max()
    # the chain by hand, from the single calls
    with torch.no_grad():
        img, ws = render_fwd(params.detach(), H, W, 7)
        _, gi = l1_ssim_loss(img, target)
        gp = render_bwd(params.detach(), gi, H, W, 7, ws)
        n1, _, _ = F.rms_norm_fwd(f, w.norm_in)
        h = F.gated_fwd(n1, w.gate, w.up)
        t = F.linear_fwd(h, w.down, residual=f)
        n2, _, _ = F.rms_norm_fwd(t, w.norm_out)
        dn2, dhead, dbias = F.linear_bwd(gp, n2, w.head, w.head_bias)
        dt, dnorm = F.rms_norm_bwd(dn2, t, w.norm_out)
        dh, ddown, _ = F.linear_bwd(dt, h, w.down)
        dn1, dgate, dup = F.gated_bwd(dh, n1, w.gate, w.up)
        _, dnorm_in = F.rms_norm_bwd(dn1, f, w.norm_in)
    for name, g in zip(NAMES, [dnorm_in, dgate, dup, ddown, dnorm, dhead, dbias]):
        assert torch.equal(getattr(w, name).grad, g), name
        assert torch.isfinite(g).all() and g.abs().max() > 0


def test_adapter_in_8_bits():
    """The 8-bit block against the 16-bit one on the weights and features that its 8-bit rows stand for."""
    rng = np.random.default_rng(22)
    B, N, D, P = 2, 100, 64, 8
    w = _weights(rng, D, 96, P, BF16)
    f, up, base = rand(rng, (B, N, D), BF16), rand(rng, (B, N, D), BF16), rand(rng, (B, N, P), F32)
    w8 = w.quantized()
    assert w8.gate.dtype == E4M3 and w8.gate_scale.shape == (96,)
    y8 = F.adapter(f, w8, base, up)
    q, s, sc = F.rms_norm_fwd(f, w.norm_in, up, out_dtype=E4M3)
    X = q.double() * sc.double()[..., None]
    g, u = (X @ (a.double() * b.double()[:, None]).t() for a, b in [(w8.gate, w8.gate_scale), (w8.up, w8.up_scale)])
    t = (torch.nn.functional.silu(g) * u) @ w.down.double().t() + f.double() + up.double()
    n = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.norm_out.double()
    want = n @ w.head.double().t() + w.head_bias.double() + base.double()
    # roundings to bf16 on the way: s, h, t, n
    assert (y8.double() - want).norm() <= 5 * U[BF16] * want.norm()
    y16 = F.adapter(f, w, base, up)
    assert (y8 - y16).norm() <= 2.0 ** -3 * y16.norm()
    assert not y8.requires_grad


def test_gradients_against_differences():
    """linear and gated gradients against central differences of the fp32 output, fp16 operands.

    x moves by +-h along a direction that fp16 holds exactly; the quotient's error is h^2 of the
    third derivative plus the output's fp32 rounding over h."""
    rng = np.random.default_rng(23)
    M, K, N = 8, 16, 24
    x = torch.round(rand(rng, (M, K), F32) * 64).div(64).half()
    w, wu = rand(rng, (N, K), F16, 0.3), rand(rng, (N, K), F16, 0.3)
    d = torch.sign(rand(rng, (M, K), F32)).half()
    h = 2.0 ** -5
    for kind in ["none", "silu", "gelu", "gelu_tanh"]:
        for fwd, bwd in [(lambda v: F.linear_fwd(v, w, activation=kind, out_dtype=F32), lambda g: F.linear_bwd(g, x, w, None, kind)[0]),
                         (lambda v: F.gated_fwd(v, w, wu, kind, out_dtype=F32), lambda g: F.gated_bwd(g.half(), x, w, wu, kind)[0])]:
            g = torch.round(rand(rng, (M, N), F32) * 8).div(8)
            num = ((fwd(x + h * d) - fwd(x - h * d)).double() * g.double()).sum() / (2 * h)
            got = (bwd(g).double() * d.double()).sum()
            scale = (bwd(g).double().abs()).sum()
            # third derivative along d: |d.w|^3 of some units, h^2 / 6 of it; fp16 gradients: u of each term
            assert abs(float(num - got)) <= (4 * U[F16] + 16 * h * h) * float(scale)


def test_backward_with_unused_outputs_and_frozen_weights():
    x = torch.randn(30, 64, device="cuda", dtype=BF16, requires_grad=True)
    r = torch.randn(30, 64, device="cuda", dtype=BF16, requires_grad=True)
    n = torch.ones(64, device="cuda", dtype=BF16, requires_grad=True)
    y, s = F.rms_norm(x, n, r)
    gx, gr, gn = torch.autograd.grad(s.float().sum(), [x, r, n], allow_unused=True)
    assert (gx == 1).all() and (gr == 1).all() and not gn.any()
    y, s = F.rms_norm(x, n, r)
    gx, gr = torch.autograd.grad(y.float().square().sum(), [x, r])
    assert torch.equal(gx, gr)
    w = torch.randn(16, 64, device="cuda", dtype=BF16)
    y = F.linear(x.t().contiguous().t(), w, residual=None, activation="relu")  # a strided view
    (gx,) = torch.autograd.grad(y, [x], torch.ones_like(y).t().contiguous().t())
    assert torch.equal(gx, F.linear_bwd(torch.ones_like(y), x.detach(), w, None, "relu")[0])
    h = F.gated(x, w, w)
    (gx,) = torch.autograd.grad(h.float().sum(), [x])
    assert gx.shape == x.shape


@pytest.mark.parametrize("M,K,N", [(3, 8, 65536), (2, 65536, 5), (130, 1000, 4100), (100001, 24, 9), (70000, 33, 14)])
def test_extreme_sizes(M, K, N):
    """The widest operands, long sums of few columns, many rows: forward and all gradients."""
    rng = np.random.default_rng(M + K)
    x, w, b, r = rand(rng, (M, K), BF16), rand(rng, (N, K), BF16, K ** -0.5), rand(rng, (N,), F32), rand(rng, (M, N), F32)
    X, W, B, R = f64(x), f64(w), f64(b), f64(r)
    want = O.linear(X, W, B, R)
    close(F.linear_fwd(x, w, b, r, out_dtype=F32), want, z_error(X, W, B) + STEP * (np.abs(want) + np.abs(R)), F32, "y")
    check_linear_bwd(M, K, N, BF16, F32, "none")


def test_norm_rows_behind_the_last_stay_as_they_were():
    """Rows of every residue of 16 bytes: what lies behind the outputs is not touched."""
    from differentiable_gaussian_splatting_pdr_b200 import _lib
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(30)
    for D in list(range(1, 18)) + [77, 100, 333, 4099, 8191]:
        for M in (1, 5, 33, 100):
            for dt, code in ((F32, 0), (BF16, 2)):
                x, g, w = rand(rng, (M, D), dt), rand(rng, (M, D), dt), rand(rng, (D,), dt)
                n = M * D
                bufs = {k: torch.full((n + 512,), 7.0, device="cuda", dtype=dt) for k in ("s", "y", "dx")}
                q, sc = torch.full((n + 512,), 7, device="cuda", dtype=torch.uint8), torch.full((M + 64,), 7.0, device="cuda")
                dw = torch.full((D + 64,), 7.0, device="cuda", dtype=dt)
                ws = torch.empty(lib.pdr_rms_norm_bwd_workspace_bytes(M, D), device="cuda", dtype=torch.uint8)
                a = {k: v.data_ptr() for k, v in bufs.items()}
                assert lib.pdr_rms_norm_fwd(x.data_ptr(), x.data_ptr(), code, w.data_ptr(), code, 1e-6, M, D, a["s"], a["y"], code, None, stream) == 0
                assert lib.pdr_quantize_rows(x.data_ptr(), code, M, D, q.data_ptr(), sc.data_ptr(), stream) == 0
                assert lib.pdr_rms_norm_bwd(g.data_ptr(), x.data_ptr(), code, w.data_ptr(), code, None, 1e-6, M, D, a["dx"], dw.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
                for t in bufs.values():
                    assert (t[n:] == 7).all() and torch.isfinite(t[:n]).all()
                assert (q[n:] == 7).all() and (sc[M:] == 7).all() and (dw[D:] == 7).all()
                assert torch.equal(bufs["s"][:n].view(M, D), x + x)


def test_calls_from_several_threads():
    import threading
    rng = np.random.default_rng(31)
    x, w, wu, g = rand(rng, (900, 72), BF16), rand(rng, (64, 72), BF16), rand(rng, (64, 72), BF16), rand(rng, (900, 64), BF16)
    want = (F.linear_fwd(x, w, activation="silu"), F.gated_fwd(x, w, wu), *F.gated_bwd(g, x, w, wu))
    torch.cuda.synchronize()
    got, errors = [None] * 6, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    out = (F.linear_fwd(x, w, activation="silu"), F.gated_fwd(x, w, wu), *F.gated_bwd(g, x, w, wu))
                torch.cuda.current_stream().synchronize()
                got[i] = out
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for out in got:
        for a, e in zip(out, want):
            assert torch.equal(a, e)


def test_adapter_captured_with_its_renderer():
    """A training step (forward, loss, gradients) captured and replayed on new features gives the eager step's bits."""
    from differentiable_gaussian_splatting_pdr_b200 import l1_ssim, render
    rng = np.random.default_rng(32)
    B, N, C, H, W, D = 1, 128, 1, 32, 32, 64
    w = _weights(rng, D, 96, 5 + C, BF16)
    f = rand(rng, (B, N, D), BF16)
    base = torch.rand(B, N, 5 + C, device="cuda") * 30
    base[..., 2:5] = 0.3
    target = torch.rand(B, C, H, W, device="cuda")
    leaves = [getattr(w, n).requires_grad_(True) for n in NAMES]

    def step():
        loss = l1_ssim(render(F.adapter(f, w, base), H, W, 7), target)
        return (loss.detach(), *torch.autograd.grad(loss, leaves))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2):
        f.copy_(rand(np.random.default_rng(100 + seed), (B, N, D), BF16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, want):
            assert torch.equal(a, e)


def test_given_workspaces_hold_nothing_between_calls():
    """One workspace full of NaN bytes serves calls of any size: nothing is read from it that the call did not write."""
    from differentiable_gaussian_splatting_pdr_b200 import _lib
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng(33)
    ws = torch.full((64 << 20,), 255, device="cuda", dtype=torch.uint8)
    for M, K, N, act in [(300, 77, 45, 3), (64, 130, 260, 2), (1000, 40, 6, 0), (129, 64, 41, 1)]:
        x, w, b, g = rand(rng, (M, K), BF16), rand(rng, (N, K), BF16), rand(rng, (N,), F32), rand(rng, (M, N), BF16)
        kind = ACTS[act]
        want_y, want = F.linear_fwd(x, w, b, g, kind), F.linear_bwd(g, x, w, b, kind)
        y = torch.empty(M, N, device="cuda", dtype=BF16)
        d = [torch.empty_like(t) for t in (x, w, b)]
        for _ in range(2):
            ws.fill_(255)
            assert lib.pdr_linear_fwd(x.data_ptr(), w.data_ptr(), 2, None, None, b.data_ptr(), 0, g.data_ptr(), act, M, N, K,
                                      y.data_ptr(), 2, ws.data_ptr(), ws.numel(), stream) == 0
            assert torch.equal(y, want_y)
            ws.fill_(255)
            assert lib.pdr_linear_bwd(g.data_ptr(), 2, x.data_ptr(), w.data_ptr(), 2, b.data_ptr(), 0, act, M, N, K,
                                      *(t.data_ptr() for t in d), ws.data_ptr(), ws.numel(), stream) == 0
            for a, e in zip(d, want):
                assert torch.equal(a, e)
        wu = rand(rng, (N, K), BF16)
        want = F.gated_bwd(g, x, w, wu)
        d = [torch.empty_like(t) for t in (x, w, wu)]
        ws.fill_(255)
        assert lib.pdr_gated_bwd(g.data_ptr(), x.data_ptr(), w.data_ptr(), wu.data_ptr(), 2, 2, M, K, N,
                                 *(t.data_ptr() for t in d), ws.data_ptr(), ws.numel(), stream) == 0
        for a, e in zip(d, want):
            assert torch.equal(a, e)


# Rows shared by one to 32 warps, and more rows than the machine has blocks for.
WIDE_SHAPES = [(2500, 1032), (2500, 1152), (2401, 1409), (1300, 2304), (700, 4170), (500, 6464), (333, 8191), (300, 12296),
               (160, 12289), (300, 16377)]


@pytest.mark.parametrize("M,D", WIDE_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rms_norm_of_wide_rows(M, D, dtype):
    test_rms_norm(M, D, dtype, dtype, M % 2 == 0)
    test_rms_norm_gradients(M, D, dtype, dtype, M % 2 == 1)


@pytest.mark.parametrize("D", [16381, 16384])
def test_rms_norm_of_the_widest_fp32_rows(D):
    test_rms_norm(160, D, F32, F32, True)
    test_rms_norm_gradients(160, D, F32, F32, True)


@pytest.mark.parametrize("M,N", [(40000, 600), (12000, 1800), (40000, 130), (9000, 4000), (70000, 256)])
def test_linear_of_many_rows_of_tiles(M, N):
    """Columns of tiles that divide the machine evenly, or leave pairs over."""
    rng = np.random.default_rng(N)
    x, w, b = rand(rng, (M, 72), BF16), rand(rng, (N, 72), BF16, 0.2), rand(rng, (N,), F32)
    X, W, B = f64(x), f64(w), f64(b)
    want = O.linear(X, W, B)
    close(F.linear_fwd(x, w, b, out_dtype=F32), want, z_error(X, W, B) + STEP * np.abs(want), F32, "y")


@pytest.mark.parametrize("M,N", [(20000, 700), (9000, 2056)])
def test_gated_of_many_rows_of_tiles(M, N):
    rng = np.random.default_rng(N)
    x, g, u = rand(rng, (M, 64), BF16), rand(rng, (N, 64), BF16, 0.2), rand(rng, (N, 64), BF16, 0.2)
    X, G, Up = f64(x), f64(g), f64(u)
    eg, eu = z_error(X, G, None) + 4 * STEP * np.abs(X @ G.T), z_error(X, Up, None) + 4 * STEP * np.abs(X @ Up.T)
    a, z = O.act(X @ G.T, "silu")[0], X @ Up.T
    h = F.gated_fwd(x, g, u, out_dtype=F32)
    close(h, a * z, value_error(X @ G.T, eg, "silu") * (np.abs(z) + eu) + np.abs(a) * eu + STEP * np.abs(a * z), F32, "h")


@pytest.mark.parametrize("N", [1, 6, 8, 45, 256, 300, 777, 2050])
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
def test_bias_sums_of_any_width(N, grad_dtype):
    check_linear_bwd(5003, 40, N, BF16, grad_dtype, "none")
