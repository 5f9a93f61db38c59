"""linear, gated, rms_norm and quantize_rows on the host: sizes, refusals of the
C entry points and of the Python calls, before anything is launched."""
import pytest
import torch

from differentiable_gaussian_splatting_pdr_b200 import _lib, build as pdr_build
from differentiable_gaussian_splatting_pdr_b200 import features as F

INVALID, SMALL, LARGE = 1, 2, 6
F32, F16, BF16, E4M3 = 0, 1, 2, 3
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers only without a GPU")
P = 0x100000  # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    pdr_build.build()
    return _lib.load()


def test_workspace_sizes(lib):
    assert lib.pdr_linear_workspace_bytes(100, 8, 64, BF16, F32, 1) == 0   # rows of 128 and 32 bytes: in place
    assert lib.pdr_linear_workspace_bytes(100, 6, 64, BF16, F32, 1) == 0   # narrow results: in place
    n = lib.pdr_linear_workspace_bytes(100, 40, 64, BF16, BF16, 1)         # 80 bytes: the residual padded to 96
    assert n >= 100 * 48 * 2 and lib.pdr_linear_workspace_bytes(100, 40, 64, BF16, BF16, 0) == 0
    assert lib.pdr_linear_workspace_bytes(100, 41, 64, BF16, BF16, 1) > n  # and the result to 96
    n = lib.pdr_linear_workspace_bytes(100, 8, 63, BF16, F32, 1)           # padded copies of x and weight
    assert n >= (100 + 8) * 64 * 2 and n % 256 == 0
    assert lib.pdr_linear_workspace_bytes(100, 8, 24, E4M3, BF16, 0) > 0   # 24 bytes
    assert lib.pdr_linear_bwd_workspace_bytes(0, 8, 64, BF16, F32, 0) >= 0
    a = lib.pdr_linear_bwd_workspace_bytes(1000, 64, 64, BF16, BF16, 0)
    assert lib.pdr_linear_bwd_workspace_bytes(1000, 64, 64, BF16, F32, 0) >= a + 1000 * 64 * 2
    assert lib.pdr_linear_bwd_workspace_bytes(1000, 64, 64, BF16, BF16, 3) > a
    assert lib.pdr_gated_workspace_bytes(100, 64, 40, F16, F16) == 0
    assert lib.pdr_gated_workspace_bytes(100, 64, 41, F16, F16) >= 100 * 48 * 2
    assert lib.pdr_gated_bwd_workspace_bytes(100, 64, 40, F16) >= 2 * 100 * 40 * 2
    assert lib.pdr_rms_norm_bwd_workspace_bytes(100, 64) >= 64 * 4


@pytest.mark.parametrize("args", [(-1, 8, 64, BF16), (1, 0, 64, BF16), (1, 8, 0, BF16), (1, 8, 64, F32),
                                  (1, 8, 64, 9), (1, 65537, 64, BF16), (1, 8, 65537, BF16)])
def test_workspace_sizes_of_bad_arguments(lib, args):
    assert lib.pdr_linear_workspace_bytes(4, 8, 64, BF16, E4M3, 0) == 0
    assert lib.pdr_gated_workspace_bytes(4, 64, 8, BF16, E4M3) == 0
    assert lib.pdr_linear_workspace_bytes(*args, F32, 1) == 0
    assert lib.pdr_linear_bwd_workspace_bytes(*args, F32, 0) == 0
    M, N, K, t = args
    assert lib.pdr_gated_workspace_bytes(M, K, N, t, BF16) == 0
    assert lib.pdr_gated_bwd_workspace_bytes(M, K, N, t) == 0


@no_gpu
def test_linear_fwd_refusals(lib):
    ok = dict(x=P, w=P, dtype=BF16, xs=None, ws=None, bias=P, bt=F32, res=P, act=0, M=4, N=8, K=64, y=P, yt=F32,
              wsp=None, wsn=0)

    def call(**kw):
        a = {**ok, **kw}
        return lib.pdr_linear_fwd(a["x"], a["w"], a["dtype"], a["xs"], a["ws"], a["bias"], a["bt"], a["res"],
                                  a["act"], a["M"], a["N"], a["K"], a["y"], a["yt"], a["wsp"], a["wsn"], None)

    for bad in [dict(M=-1), dict(N=0), dict(K=0), dict(dtype=F32), dict(dtype=7), dict(yt=E4M3), dict(act=5),
                dict(act=-1), dict(x=None), dict(w=None), dict(y=None), dict(xs=P), dict(ws=P),
                dict(dtype=E4M3), dict(dtype=E4M3, xs=P), dict(dtype=E4M3, ws=P), dict(bt=E4M3), dict(bt=9),
                dict(x=P + 8), dict(w=P + 2), dict(y=P + 8), dict(res=P + 16), dict(bias=P + 2),
                dict(K=63), dict(K=63, wsp=P + 16, wsn=1 << 30)]:
        assert call(**bad) == INVALID, bad
    assert call(K=63, wsp=P, wsn=100) == SMALL
    assert call(K=65537) == LARGE and call(N=65537) == LARGE and call(M=(1 << 30) + 1) == LARGE


@no_gpu
def test_linear_bwd_refusals(lib):
    ok = dict(g=P, gt=BF16, x=P, w=P, dtype=BF16, bias=P, bt=F32, act=1, M=4, N=8, K=64, dx=P, dw=P, db=P,
              wsp=P, wsn=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return lib.pdr_linear_bwd(a["g"], a["gt"], a["x"], a["w"], a["dtype"], a["bias"], a["bt"], a["act"],
                                  a["M"], a["N"], a["K"], a["dx"], a["dw"], a["db"], a["wsp"], a["wsn"], None)

    for bad in [dict(M=-1), dict(N=0), dict(K=0), dict(dtype=F32), dict(dtype=E4M3), dict(gt=E4M3), dict(act=9),
                dict(g=None), dict(x=None), dict(w=None), dict(bt=E4M3), dict(g=P + 16), dict(x=P + 4),
                dict(w=P + 4), dict(dx=P + 8), dict(dw=P + 8), dict(db=P + 1), dict(wsp=None), dict(wsp=P + 8)]:
        assert call(**bad) == INVALID, bad
    assert call(wsn=8) == SMALL
    assert call(K=65537) == LARGE


@no_gpu
def test_gated_refusals(lib):
    def fwd(x=P, g=P, u=P, t=F16, xs=None, gs=None, us=None, act=2, M=4, D=64, Fw=8, h=P, ht=F16, w=None, n=0):
        return lib.pdr_gated_fwd(x, g, u, t, xs, gs, us, act, M, D, Fw, h, ht, w, n, None)

    for bad in [dict(M=-1), dict(D=0), dict(Fw=0), dict(t=F32), dict(ht=E4M3), dict(act=7), dict(x=None),
                dict(g=None), dict(u=None), dict(h=None), dict(xs=P), dict(gs=P), dict(t=E4M3, xs=P, gs=P),
                dict(x=P + 2), dict(g=P + 2), dict(u=P + 2), dict(h=P + 8), dict(D=63)]:
        assert fwd(**bad) == INVALID, bad
    assert fwd(D=63, w=P, n=1) == SMALL
    assert fwd(D=70000) == LARGE

    def bwd(g=P, x=P, wg=P, wu=P, t=F16, act=2, M=4, D=64, Fw=8, dx=P, dg=P, du=P, w=P, n=1 << 30):
        return lib.pdr_gated_bwd(g, x, wg, wu, t, act, M, D, Fw, dx, dg, du, w, n, None)

    for bad in [dict(M=-1), dict(t=E4M3), dict(t=F32), dict(g=None), dict(x=None), dict(wg=None), dict(wu=None),
                dict(dg=None), dict(du=None), dict(w=None), dict(w=P + 32), dict(x=P + 2), dict(g=P + 16)]:
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=16) == SMALL


@no_gpu
def test_norm_refusals(lib):
    def fwd(x=P, r=P, t=BF16, w=P, wt=BF16, eps=1e-6, M=4, D=64, s=P, y=P, yt=BF16, sc=None):
        return lib.pdr_rms_norm_fwd(x, r, t, w, wt, eps, M, D, s, y, yt, sc, None)

    for bad in [dict(M=-1), dict(D=0), dict(t=E4M3), dict(wt=F16), dict(yt=F32), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(y=None), dict(sc=P), dict(yt=E4M3),
                dict(r=None), dict(x=P + 1), dict(r=P + 1), dict(s=P + 1), dict(y=P + 1), dict(w=P + 1),
                dict(yt=E4M3, sc=P + 2)]:
        assert fwd(**bad) == INVALID, bad
    assert fwd(D=16385) == LARGE

    def bwd(g=P, s=P, t=BF16, w=P, wt=BF16, gs=P, eps=1e-6, M=4, D=64, dx=P, dw=P, ws=P, n=1 << 20):
        return lib.pdr_rms_norm_bwd(g, s, t, w, wt, gs, eps, M, D, dx, dw, ws, n, None)

    for bad in [dict(M=-1), dict(D=0), dict(t=E4M3), dict(wt=F16), dict(g=None), dict(s=None), dict(w=None),
                dict(ws=None), dict(ws=P + 8), dict(dx=P + 1), dict(gs=P + 1), dict(eps=-1.0)]:
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=4) == SMALL
    q = lib.pdr_quantize_rows
    assert q(None, BF16, 4, 64, P, P, None) == INVALID and q(P, E4M3, 4, 64, P, P, None) == INVALID
    assert q(P, BF16, 4, 64, P, None, None) == INVALID and q(P, BF16, 4, 0, P, P, None) == INVALID
    assert q(P, BF16, 4, 16385, P, P, None) == LARGE


@no_gpu
def test_no_rows_need_no_arrays_and_launch_nothing(lib):
    assert lib.pdr_linear_fwd(None, P, BF16, None, None, None, 0, None, 0, 0, 8, 64, None, F32, None, 0, None) == 0
    assert lib.pdr_gated_fwd(None, P, P, E4M3, None, P, P, 2, 0, 64, 8, None, BF16, None, 0, None) == 0
    assert lib.pdr_rms_norm_fwd(None, None, F32, P, F32, 1e-6, 0, 64, None, None, F32, None, None) == 0
    assert lib.pdr_quantize_rows(None, F32, 0, 64, None, None, None) == 0


def test_python_calls_refuse_host_tensors_and_unknown_activations():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.linear_fwd(x, w)
    with pytest.raises(ValueError, match="activation"):
        F.linear_fwd(x, w, activation="swish")
    with pytest.raises(ValueError, match="activation"):
        F.gated_fwd(x, w, w, activation=None)
    for call in (lambda: F.linear_bwd(x, x, w), lambda: F.gated_fwd(x, w, w), lambda: F.gated_bwd(x, x, w, w),
                 lambda: F.rms_norm_fwd(x, w[0]), lambda: F.rms_norm_bwd(x, x, w[0]), lambda: F.quantize_rows(x),
                 lambda: F.rms_norm(x, w[0]), lambda: F.linear(x, w), lambda: F.gated(x, w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_package_exports():
    import differentiable_gaussian_splatting_pdr_b200 as pkg
    for name in ["linear", "linear_fwd", "linear_bwd", "gated", "gated_fwd", "gated_bwd", "rms_norm",
                 "rms_norm_fwd", "rms_norm_bwd", "quantize_rows", "adapter", "AdapterWeights", "check_wait_error"]:
        assert getattr(pkg, name) is getattr(F, name)


@no_gpu
def test_norm_refuses_the_widest_rows_that_start_inside_a_vector(lib):
    """1024 threads hold 16384 elements, of which a row that is no multiple of 16
    bytes cannot use the last ones."""
    def fwd(D, t, yt, sc):
        return lib.pdr_rms_norm_fwd(P, None, t, P, t, 1e-6, 4, D, None, P, yt, sc, None)

    for t, first in ((BF16, 16378), (F32, 16382)):
        for D in range(first, 16384):
            if D % (4 if t == F32 else 8) == 0:
                continue
            assert fwd(D, t, t, None) == LARGE and lib.pdr_quantize_rows(P, t, 4, D, P, P, None) == LARGE
            assert lib.pdr_rms_norm_bwd(P, P, t, P, t, None, 1e-6, 4, D, P, P, P, 1 << 40, None) == LARGE
