"""The linear layer's tile kernels at sizes that take each of their shapes:
whole and ragged tiles, several tiles a workgroup, one stage of K to many,
odd numbers of stages, K that ends inside a stage. Rows that lie on and next
to the tiles' borders are compared with the definition in 64 bits; tolerances
as derived in test_gpu_linear.py."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import (BF, DEV, DT, activations, check_mx8, decode, decode4, linear_ref, rand, strided,
                             weights)

pytestmark = pytest.mark.gpu


def some_rows(m):
    at = {0, 1, m - 1, m // 2}
    for edge in (16, 31, 32, 63, 64, 127, 128, 255, 256, 511, 512, m // 256 * 256):
        at |= {edge - 1, edge}
    return torch.tensor(sorted(r for r in at if 0 <= r < m))


def check(m, n, K, fmt, act="NONE", gated=False, bias=None, residual=False, mx8=False, save_z=False,
          strides=False, seed=100):
    N = 2 * n if gated else n
    a, va = activations(m, K, seed)
    b, vb = weights(N, K, fmt, seed + 1)
    bv = None if bias is None else rand(N, seed=seed + 2).to(DT[bias])
    res = rand(m, n, seed=seed + 3, std=4.0, dtype=torch.bfloat16) if residual else None
    if strides:
        a = (strided(a[0].cpu(), 32), strided(a[1].cpu(), 5, 3))
        b = (strided(b[0].cpu(), 16), strided(b[1].cpu(), 3, 1))
    got = A.adahop_linear_mx(a, b, bias=None if bv is None else bv.to(DEV), act=act, gated=gated,
                             residual=None if res is None else res.to(DEV),
                             out_dtype="MXFP8" if mx8 else torch.bfloat16, save_z=save_z)
    at = some_rows(m)
    z, dz, out, dout = linear_ref(va[at], vb, bv, act, gated, None if res is None else res[at])
    if save_z:
        err = (got.z.cpu()[at].double() - z).abs()
        assert bool((err <= dz + BF * (z.abs() + dz)).all())
    if mx8:
        check_mx8(got.out.cpu()[at], got.scales.cpu()[at], out, dout)
    else:
        err = (got.out.cpu()[at].double() - out).abs()
        assert bool((err <= dout + BF * (out.abs() + dout)).all())


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,K", [
    (33, 32, 32), (40, 70, 128), (63, 129, 256), (64, 256, 384), (129, 500, 1184),     # 64 rows
    (700, 2100, 160), (1000, 1700, 640), (1536, 1536, 544),                            # 128 rows
    (2100, 5410, 288), (4096, 4096, 128), (4200, 4200, 96), (2049, 6200, 1024),        # 256 rows
])
def test_tiles(m, n, K, fmt, gated):
    check(m, n, K, fmt, act="SILU" if gated else "NONE", gated=gated, save_z=m < 1000, residual=n % 4 == 0)


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(50, 96, 288), (1100, 1824, 416), (2300, 5600, 224), (4300, 4160, 512)])
def test_tiles_mx8_out(m, n, K, fmt):
    check(m, n, K, fmt, act="GELU", bias="f32", mx8=True)
    check(m, n // 64 * 32, K, fmt, act="SILU", gated=True, bias="bf16", mx8=True)


@pytest.mark.parametrize("act", list(A.ACT))
@pytest.mark.parametrize("m,n,K", [(2200, 5200, 128), (1100, 1800, 96)])
def test_tiles_epilogues(m, n, K, act):
    check(m, n, K, "MXFP4", act=act, bias="f32", residual=True, save_z=True)
    check(m, n // 2, K, "MXFP8", act=act, gated=True, bias="bf16", residual=True, save_z=True)


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(90, 210, 192), (1100, 1800, 256), (2200, 5200, 384)])
def test_tiles_strides(m, n, K, fmt):
    """Operands inside larger buffers whose other bytes are NaN."""
    check(m, n, K, fmt, strides=True, residual=True)


@pytest.mark.parametrize("m,n", [(100, 320), (1200, 1600), (2400, 5200)])
def test_tiles_non_finite(m, n):
    """A NaN or an infinity reaches its own row and no other; the codes that
    follow a row in memory are another row's, some of them NaN."""
    K = 160
    x = rand(m, K, seed=110)
    bad_rows = [3, m // 2, m - 1]
    x[bad_rows[0], 5], x[bad_rows[1], K - 1], x[bad_rows[2], 0] = float("nan"), float("inf"), float("-inf")
    a = A.adahop_mx8_quant(x.to(DEV))
    b, _ = weights(n, K, "MXFP8", 111)
    bad = A.adahop_linear_mx(a, b).out.isnan().cpu()
    want = torch.zeros(m, dtype=torch.bool)
    want[bad_rows] = True
    assert torch.equal(bad.all(1), want) and torch.equal(bad.any(1), want)


def test_tiles_deterministic():
    for m, n, K in ((100, 512, 8192), (1024, 2048, 1024), (2048, 8192, 512)):
        a, _ = activations(m, K, 112)
        b, _ = weights(n, K, "MXFP4", 113)
        first = A.adahop_linear_mx(a, b).out
        for _ in range(3):
            assert torch.equal(A.adahop_linear_mx(a, b).out, first)


# ---- operands of 2 GB and more, more rows than a grid's second dimension -------
def codes(rows, K, seed, fmt="MXFP8"):
    """Codes and scales of small magnitudes, made on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if fmt == "MXFP8":
        c = torch.randint(0x20, 0x40, (rows, K), dtype=torch.uint8, device=DEV, generator=g)
        c |= torch.randint(0, 2, (rows, K), dtype=torch.uint8, device=DEV, generator=g) << 7
    else:
        c = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    return c, torch.randint(124, 130, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)


def values(m, fmt="MXFP8"):
    return (decode if fmt == "MXFP8" else decode4)(*m)


def at_rows(m, rows):
    return m[0][rows.to(DEV)], m[1][rows.to(DEV)]


def check_at(a, b, fmt, act="NONE", gated=False):
    """The output at some rows and columns, the last and those around every
    2^31 bytes among them."""
    m, K = a[0].shape
    N = b[0].shape[0]
    n = N // 2 if gated else N
    got = A.adahop_linear_mx(a, b, act=act, gated=gated).out

    def some(rows, ld):
        at = {0, 1, rows // 2, rows - 1}
        for k in range(1, rows * ld // 2 ** 31 + 1):
            at |= {k * 2 ** 31 // ld + d for d in (-2, -1, 0, 1)}
        return torch.tensor(sorted(r for r in at if 0 <= r < rows))

    r, c = some(m, K), some(n, b[0].shape[1])
    cols = torch.cat((c, n + c)) if gated else c
    z, dz, out, dout = linear_ref(values(at_rows(a, r)), values(at_rows(b, cols), fmt), None, act, gated, None)
    err = (got[r.to(DEV)][:, c.to(DEV)].cpu().double() - out).abs()
    assert bool((err <= dout + BF * (out.abs() + dout)).all())


def test_far_rows_of_a():
    check_at(codes(131500, 16384, 120), codes(64, 16384, 121), "MXFP8")


def test_far_rows_of_b():
    check_at(codes(70, 16384, 122), codes(132000, 16384, 123), "MXFP8")


def test_far_rows_of_gated_b():
    check_at(codes(40, 16384, 124), codes(264000, 16384, 125), "MXFP8", act="SILU", gated=True)


def test_rows_far_apart():
    """40 rows 60 MB apart (one token of each of 40 long sequences)."""
    base, sc = codes(40, 60 << 20, 126)
    a = (base[:, :512], sc[:, :16])
    check_at(a, codes(96, 512, 127, "MXFP4"), "MXFP4")


def test_many_rows():
    check_at(codes((1 << 21) + 65, 32, 128), codes(32, 32, 129, "MXFP4"), "MXFP4")


def test_norm_many_rows():
    """More rows than one launch takes."""
    rows, cols = (1 << 22) + 70, 32
    g = torch.Generator(device=DEV).manual_seed(130)
    x, r = (torch.randn(rows, cols, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    gain = torch.ones(cols, device=DEV)
    got = A.adahop_rmsnorm(x, gain, r, bf16=True, save_rstd=True)
    for at in (slice(0, 70), slice((1 << 22) - 70, rows)):
        part = A.adahop_rmsnorm(x[at], gain, r[at], bf16=True, save_rstd=True)
        for a, b in zip(got, part):
            assert torch.equal(a[at], b)


# ---- MXFP8 outputs of few values ------------------------------------------------
@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(1, 32, 32), (1, 64, 4096), (5, 96, 1056), (16, 160, 544), (17, 64, 2080), (33, 96, 8192),
                                   (100, 320, 320)])
def test_mx8_out_of_exact_products(m, n, K, fmt):
    """Off by the fp32 sums alone: a product of two formats' values is exact,
    a chain has up to K / 32 + 8 + 4 additions in fp32, each of four more
    products that the instruction adds."""
    a, va = activations(m, K, 140)
    b, vb = weights(n, K, fmt, 141)
    got = A.adahop_linear_mx(a, b, out_dtype="MXFP8")
    want = va @ vb.t()
    check_mx8(got.out, got.scales, want, (K / 4 + 16) * 2.0 ** -24 * (va.abs() @ vb.abs().t()))
    ga, _ = weights(2 * n, K, fmt, 142)
    gated = A.adahop_linear_mx(a, ga, act="RELU", gated=True, out_dtype="MXFP8")
    _, vg = ga, (decode if fmt == "MXFP8" else decode4)(*ga)
    z, mag = va @ vg.t(), (K / 4 + 16) * 2.0 ** -24 * (va.abs() @ vg.abs().t())
    f, up = z[:, :n].clamp(min=0), z[:, n:]
    bound = mag[:, :n] * up.abs() + (f + mag[:, :n]) * mag[:, n:] + 2.0 ** -24 * (f * up).abs()
    check_mx8(gated.out, gated.scales, f * up, bound)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("m", [3, 40])
def test_scale_byte_255(m, mx8):
    """A block whose scale is the NaN byte is NaN whatever its codes."""
    (ac, asc), _ = activations(m, 256, 143)
    (bc, bsc), _ = weights(64, 256, "MXFP4", 144)
    asc[1, 3] = 255
    got = A.adahop_linear_mx((ac, asc), (bc, bsc), out_dtype="MXFP8" if mx8 else torch.bfloat16)
    out = A.adahop_mx8_dequant(got.out, got.scales) if mx8 else got.out
    want = torch.zeros(m, dtype=torch.bool)
    want[1] = True
    assert torch.equal(out.isnan().all(1).cpu(), want) and torch.equal(out.isnan().any(1).cpu(), want)
    bsc[5, 2] = 255
    asc[1, 3] = 120
    got = A.adahop_linear_mx((ac, asc), (bc, bsc), out_dtype="MXFP8" if mx8 else torch.bfloat16)
    out = A.adahop_mx8_dequant(got.out, got.scales) if mx8 else got.out
    cols = out.isnan().all(0).cpu()
    assert bool(cols[5]) and int(cols.sum()) == (32 if mx8 else 1)
