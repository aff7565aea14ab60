"""How the linear layer's products are formed: the caller's choice, and the rule
of AUTO. Tolerances as derived in test_gpu_linear.py; exact products are off by
the fp32 sums alone: a chain has up to K / 32 + 8 + 4 additions, each of four
more products that the instruction adds."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import BF, U, activations, check_mx8, decode, decode4, linear_ref, rand, weights

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


# ---- scales near the ends of E8M0 ---------------------------------------------
def far_operands(m, n, K, fmt, seed):
    """Codes and scales whose values lie near both ends of what the formats hold,
    in blocks where the other operand's lie near the other end; ordinary blocks
    and blocks of zeros (byte 0) between them."""
    g = torch.Generator().manual_seed(seed)

    def codes(rows):
        c = torch.randint(0, 0x7F, (rows, K), dtype=torch.uint8, generator=g)
        return c | torch.randint(0, 2, (rows, K), dtype=torch.uint8, generator=g) << 7

    kind = torch.arange(K // 32) % 3

    def scales(rows, first, second):
        """Bytes of `first`, `second` and 120 .. 132 in turn, block by block."""
        s = torch.randint(0, 13, (rows, K // 32), generator=g)
        return torch.where(kind == 0, first(s), torch.where(kind == 1, second(s), 120 + s)).to(torch.uint8)

    top = 252 if fmt == "MXFP4" else 254
    ac, asc = codes(m), scales(m, lambda s: s, lambda s: 254 - s)
    bsc = scales(n, lambda s: top - s, lambda s: s)
    ac[0, :32], asc[0, 0] = 0, 0
    ac[m - 1, 64:96], asc[m - 1, 2] = 0, 0
    bc = codes(n) if fmt == "MXFP8" else torch.randint(0, 256, (n, K // 2), dtype=torch.uint8, generator=g)
    bc[1, :32 if fmt == "MXFP8" else 16], bsc[1, 0] = 0, 0
    return tuple(t.to("cuda:0") for t in (ac, asc)), tuple(t.to("cuda:0") for t in (bc, bsc))


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(1, 64, 96), (5, 64, 1056), (20, 128, 544), (3, 9216, 288)])
def test_far_scales(m, n, K, fmt):
    """Products of values that fp32, or bf16, cannot hold are finite, and exact
    with EXACT."""
    a, b = far_operands(m, n, K, fmt, 230 + m)
    va, vb = decode(*a), (decode if fmt == "MXFP8" else decode4)(*b)
    want, tol = va @ vb.t(), (K / 4 + 16) * U * (va.abs() @ vb.abs().t())
    got = A.adahop_linear_mx(a, b, out_dtype="MXFP8", products="EXACT")
    check_mx8(got.out, got.scales, want, tol)
    gated = A.adahop_linear_mx(a, b, act="RELU", gated=True, out_dtype="MXFP8", products="EXACT")
    h = n // 2
    f, up = want[:, :h].clamp(min=0), want[:, h:]
    bound = tol[:, :h] * up.abs() + (f + tol[:, :h]) * tol[:, h:] + U * (f * up).abs()
    check_mx8(gated.out, gated.scales, f * up, bound)
    out = A.adahop_linear_mx(a, b, products="EXACT").out.cpu().double()
    assert bool(((out - want).abs() <= tol + BF * (want.abs() + tol)).all())


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
def test_far_scales_non_finite(fmt):
    """Among far scales, a NaN byte or code reaches its own row or column and no other."""
    a, b = far_operands(6, 64, 288, fmt, 240)
    a[1][2, 4] = 255
    a[0][4, 33] = 0x7F
    b[1][7, 3] = 255
    out = A.adahop_linear_mx(a, b, products="EXACT").out.cpu()
    want = torch.zeros(6, 64, dtype=torch.bool)
    want[2] = want[4] = True
    want[:, 7] = True
    assert torch.equal(out.isnan(), want) and not bool(out[~want].isinf().any())


@pytest.mark.parametrize("m,n", [(5, 64), (40, 320), (1200, 1600)])
@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
def test_far_scales_of_scaled_products(m, n, fmt):
    a, b = far_operands(m, n, 288, fmt, 250)
    at = torch.tensor(sorted({0, 1, m // 2, m - 1}))
    va, vb = decode(a[0].cpu()[at], a[1].cpu()[at]), (decode if fmt == "MXFP8" else decode4)(*b)
    z, dz, out, dout = linear_ref(va, vb, None, "NONE", False, None)
    got = A.adahop_linear_mx(a, b, products="SCALED").out.cpu()[at].double()
    assert bool(((got - out).abs() <= dout + BF * (out.abs() + dout)).all())


# ---- how far scaled products are off ------------------------------------------
@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(8, 256, 4096), (300, 512, 4096), (300, 512, 1056), (2100, 5410, 512)])
def test_accuracy_of_scaled_products(m, n, K, fmt):
    """Documented: within about 5e-5 of the result, root mean square, with 1 % of
    A's columns 30 times the rest; twice that is the bound. A residual that
    cancels the result leaves 2^-8 of it at most for the output's rounding, which
    is then off by 2^-16 of the result at most (and the fp32 sum by less)."""
    x = rand(m, K, seed=260)
    g = torch.Generator().manual_seed(261)
    x[:, torch.randint(0, K, (K // 100,), generator=g)] *= 30
    a = A.adahop_mx8_quant(x.to("cuda:0"))
    b, vb = weights(n, K, fmt, 262)
    at = torch.arange(0, m, max(1, m // 300))
    want = decode(a[0].cpu()[at], a[1].cpu()[at]) @ vb.t()
    first = A.adahop_linear_mx(a, b, products="SCALED").out
    rest = A.adahop_linear_mx(a, b, residual=-first, products="SCALED").out
    off = (rest.cpu()[at].double() + first.cpu()[at].double()) - want
    assert float(off.norm()) <= (1e-4 + 2.0 ** -16) * float(want.norm())
    exact = A.adahop_linear_mx(a, b, products="EXACT").out
    rest = A.adahop_linear_mx(a, b, residual=-exact, products="EXACT").out
    off = (rest.cpu()[at].double() + exact.cpu()[at].double()) - want
    assert float(off.norm()) <= (1e-6 + 2.0 ** -16) * float(want.norm())
