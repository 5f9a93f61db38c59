"""Bounded waits of the products' kernels that run out: the launch ends, the host learns of it, nothing
around the results is touched, and the next launch gives the usual bits.

The limit is set so low that a wait whose barrier is about to be reached gives up; every wait of
these launches would return."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from differentiable_gaussian_splatting_pdr_b200 import _lib, build as pdr_build  # noqa: E402
from differentiable_gaussian_splatting_pdr_b200 import features as F  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TIMEOUT = _lib.STATUS_CODES["PDR_ERR_DEVICE_TIMEOUT"]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pdr_build.build()
    lib = _lib.load()
    yield lib
    lib.pdr_set_wait_limit(-1)
    torch.cuda.synchronize()
    F.check_wait_error()


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(dtype)


def gave_up():
    """Whether a launch since the last call gave up a wait; reported once."""
    try:
        F.check_wait_error()
    except _lib.PdrError as e:
        assert e.status == TIMEOUT
        F.check_wait_error()
        return True
    return False


# B kept in shared memory (with an odd number of k blocks, two a stage), B streamed, few and many
# tiles a pair, one launch with two products, narrow results, 8 bits.
def calls(rng):
    x, w, wu = rand(rng, (40000, 320), BF16), rand(rng, (256, 320), BF16, 0.1), rand(rng, (256, 320), BF16, 0.1)
    long, wide = rand(rng, (3000, 4096), F16), rand(rng, (520, 4096), F16, 0.02)
    head, g = rand(rng, (6, 320), BF16), rand(rng, (40000, 256), BF16)
    q, qs = F.quantize_rows(x)
    qw, qws = F.quantize_rows(w)
    return {
        "stationary": lambda: (F.linear_fwd(x, w, activation="silu"),),
        "streamed": lambda: (F.linear_fwd(long, wide),),
        "one tile": lambda: (F.linear_fwd(long[:100], wide[:64]),),
        "narrow": lambda: (F.linear_fwd(x, head, out_dtype=F32),),
        "8 bits": lambda: (F.linear_fwd(q, qw, x_scale=qs, weight_scale=qws),),
        "gated": lambda: (F.gated_fwd(x, w, wu),),
        "two products": lambda: F.linear_bwd(g, x, w)[:2],
        "gated backward": lambda: F.gated_bwd(g, x, w, wu),
    }


NAMES = ["stationary", "streamed", "one tile", "narrow", "8 bits", "gated", "two products", "gated backward"]


@pytest.mark.parametrize("name", NAMES)
def test_a_wait_that_gives_up_ends_the_launch_and_is_reported(lib, name):
    call = calls(np.random.default_rng(1))[name]
    want = call()
    assert not gave_up()
    lib.pdr_set_wait_limit(0)
    try:
        call()
        torch.cuda.synchronize()
        assert gave_up()
    finally:
        lib.pdr_set_wait_limit(-1)
    for a, e in zip(call(), want):
        assert torch.equal(a, e)
    assert not gave_up()


@pytest.mark.parametrize("name", NAMES)
def test_waits_that_give_up_at_any_place(lib, name):
    """Limits from one try on: a launch reports that it gave up, or its results are right."""
    call = calls(np.random.default_rng(2))[name]
    want = call()
    assert not gave_up()
    up = 0
    try:
        for tries in [1, 1, 2, 2, 3, 4, 5, 6, 8, 12, 20]:
            lib.pdr_set_wait_limit(tries)
            got = call()
            torch.cuda.synchronize()
            if gave_up():
                up += 1
            else:
                for a, e in zip(got, want):
                    assert torch.equal(a, e)
    finally:
        lib.pdr_set_wait_limit(-1)
    for a, e in zip(call(), want):
        assert torch.equal(a, e)
    print(name, up)


def test_arrays_around_the_results_stay_as_they_were(lib):
    rng = np.random.default_rng(3)
    M, K, N = 5000, 320, 200
    x, w = rand(rng, (M, K), BF16), rand(rng, (N, K), BF16)
    want = F.linear_fwd(x, w)
    buf = torch.full((M * N + 2 * 4096,), 7.0, device="cuda", dtype=BF16)
    out = buf[4096:4096 + M * N].view(M, N)
    xs, ws = x.clone(), w.clone()
    for tries in (0, 1, 2):
        lib.pdr_set_wait_limit(tries)
        F.linear_fwd(x, w, out=out)
        torch.cuda.synchronize()
        gave_up()
    lib.pdr_set_wait_limit(-1)
    assert (buf[:4096] == 7).all() and (buf[4096 + M * N:] == 7).all()
    assert torch.equal(x, xs) and torch.equal(w, ws)
    assert torch.equal(F.linear_fwd(x, w, out=out), want)


def test_the_next_calls_refuse_until_the_error_was_reported(lib):
    """Without check_wait_error too a wrong result does not stay unnoticed: the next product raises."""
    rng = np.random.default_rng(4)
    x, w, g = rand(rng, (300, 64), BF16), rand(rng, (64, 64), BF16), rand(rng, (300, 64), BF16)
    want = F.linear_fwd(x, w)
    lib.pdr_set_wait_limit(0)
    F.linear_fwd(x, w)
    lib.pdr_set_wait_limit(-1)
    torch.cuda.synchronize()
    y = torch.full_like(want, 7.0)
    for call in (lambda: F.linear_fwd(x, w, out=y), lambda: F.linear_bwd(g, x, w), lambda: F.gated_fwd(x, w, w, out=y),
                 lambda: F.gated_bwd(g, x, w, w), lambda: F.linear(x, w), lambda: F.gated(x, w, w)):
        with pytest.raises(_lib.PdrError) as e:
            call()
        assert e.value.status == TIMEOUT
    torch.cuda.synchronize()
    assert (y == 7).all()  # nothing was launched
    n = F.rms_norm_fwd(x, w[0].contiguous())[0]  # has no waits
    assert torch.isfinite(n).all()
    assert gave_up()
    assert torch.equal(F.linear_fwd(x, w), want)


def test_the_first_product_of_a_process_may_be_captured():
    """The error word is made by the first launch, also inside a capture."""
    import os
    import subprocess
    import sys
    code = ("import torch; from differentiable_gaussian_splatting_pdr_b200 import features as F\n"
            "x = torch.randn(100, 64, device='cuda', dtype=torch.bfloat16); w = x[:48].clone()\n"
            "torch.cuda.synchronize(); g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n    y = F.linear_fwd(x, w)\n"
            "g.replay(); torch.cuda.synchronize()\n"
            "assert torch.equal(y, F.linear_fwd(x, w)); F.check_wait_error(); print('fine')\n")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0 and "fine" in out.stdout, out.stderr[-2000:]
