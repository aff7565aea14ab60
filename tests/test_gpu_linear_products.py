"""How the linear layer's products are formed: the caller's choice, and the rule
of AUTO. Tolerances as derived in test_gpu_linear.py; exact products are off by
the fp32 sums alone: a chain has up to K / 32 + 8 + 4 additions, each of four
more products that the instruction adds."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import BF, U, activations, check_mx8, rand, weights

pytestmark = pytest.mark.gpu


def equal(x, y):
    return torch.equal(x.out, y.out) and (x.scales is None or torch.equal(x.scales, y.scales))


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,gated,exact", [(1, 64, False, True), (32, 1024, False, True), (33, 1024, False, False),
                                             (1, 9216, True, True), (4, 9216, True, False), (9, 4096, False, False),
                                             (300, 1024, False, False)])
def test_auto(m, n, gated, exact, fmt):
    """MXFP8 outputs of up to 32768 values are those of EXACT, larger ones those
    of SCALED; bf16 outputs are SCALED's."""
    a, _ = activations(m, 4096, 200)
    b, _ = weights(2 * n if gated else n, 4096, fmt, 201)
    call = {p: A.adahop_linear_mx(a, b, gated=gated, act="SILU", out_dtype="MXFP8", products=p)
            for p in ("AUTO", "SCALED", "EXACT")}
    assert equal(call["AUTO"], call["EXACT" if exact else "SCALED"])
    if m * n > 30000:
        assert not equal(call["SCALED"], call["EXACT"])
    bf = {p: A.adahop_linear_mx(a, b, gated=gated, act="SILU", products=p) for p in ("AUTO", "SCALED")}
    assert equal(bf["AUTO"], bf["SCALED"])


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(1, 33, 96), (7, 70, 1056), (17, 1000, 544), (64, 640, 2080), (40, 8224, 160),
                                   (3, 9000, 320), (150, 1056, 320)])
def test_exact(m, n, K, fmt):
    """bf16 outputs of any width, MXFP8 ones above AUTO's limit; plain and gated.
    A bf16 output's rounding is taken away by a residual that cancels it."""
    a, va = activations(m, K, 210)
    b, vb = weights(n, K, fmt, 211)
    want, tol = va @ vb.t(), (K / 4 + 16) * U * (va.abs() @ vb.abs().t())
    first = A.adahop_linear_mx(a, b, products="EXACT").out
    assert bool(((first.cpu().double() - want).abs() <= tol + BF * (want.abs() + tol)).all())
    rest = A.adahop_linear_mx(a, b, residual=-first, products="EXACT").out.cpu().double()
    left = want - first.cpu().double()
    assert bool(((rest - left).abs() <= tol + U * left.abs() + BF * (left.abs() + 2 * tol)).all())
    if n % 32 == 0:
        got = A.adahop_linear_mx(a, b, out_dtype="MXFP8", products="EXACT")
        check_mx8(got.out, got.scales, want, tol)
    bias = rand(2 * n, seed=213)
    g, vg = weights(2 * n, K, fmt, 212)
    got = A.adahop_linear_mx(a, g, bias=bias.to("cuda:0"), act="RELU", gated=True, save_z=True, products="EXACT")
    z = va @ vg.t() + bias.double()
    mag = (K / 4 + 16) * U * (va.abs() @ vg.abs().t()) + U * z.abs()
    assert bool(((got.z.cpu().double() - z).abs() <= mag + BF * (z.abs() + mag)).all())
    f, up = z[:, :n].clamp(min=0), z[:, n:]
    bound = mag[:, :n] * up.abs() + (f + mag[:, :n]) * mag[:, n:] + U * (f * up).abs()
    assert bool(((got.out.cpu().double() - f * up).abs() <= bound + BF * ((f * up).abs() + bound)).all())


def test_names():
    a, _ = activations(4, 64, 220)
    b, _ = weights(32, 64, "MXFP8", 221)
    with pytest.raises(KeyError):
        A.adahop_linear_mx(a, b, products="FAST")
