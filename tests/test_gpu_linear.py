"""Norm, MXFP8, linear layer and their gradients against their definitions in
64 bits, at the sizes where they can go wrong.

Tolerances count roundings. u = 2^-24 is an fp32 rounding; a sum of n terms is
off by at most (its longest chain of additions) u times the sum of their
magnitudes, a rounding to bf16 by 2^-8 and to E4M3 by 2^-4 of the value (2^-10
of the block's scale below E4M3's normal range). The scaled matrix cores drop,
within a group of 8 products of one instruction, each product's part under 2^-13
of the largest's power of two (measured on the device with single products):
at most 16 * 2^-13 of the largest for two groups."""
import math

import numpy as np
import pytest
import torch

import mxfp4_precision_gemms_amd as A

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(1000 * seed + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def strided(t, pad, offset=0):
    """t on the device, in rows `pad` elements longer, starting `offset` elements
    into the buffer; what surrounds it is NaN (or 0x7F for codes)."""
    r, c = t.shape
    fill = 0x7F if t.dtype == torch.uint8 else float("nan")
    buf = torch.full((offset + r * (c + pad) + 16,), fill, dtype=t.dtype, device=DEV)
    v = buf[offset:offset + r * (c + pad)].view(r, c + pad)[:, :c]
    v.copy_(t)
    return v


# ---- MXFP8 ------------------------------------------------------------------
def decode(codes, scales):
    """fp64 values of MXFP8 codes and scales (CPU)."""
    i = codes.cpu().int()
    e, f = (i >> 3) & 15, (i & 7).double()
    v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
    v = torch.where((i & 127) == 127, torch.full_like(v, float("nan")), v)
    v = torch.where(i > 127, -v, v)
    s = scales.cpu().double()
    p = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return v * p.repeat_interleave(32, 1)


def decode4(codes, scales):
    c = codes.cpu()
    i = torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1).int()
    e, f = (i >> 1) & 3, (i & 1).double()
    v = torch.where(e > 0, (2 + f) * torch.exp2(e.double() - 2), f * 0.5)
    return torch.where(i > 7, -v, v) * torch.exp2(scales.cpu().double() - 127).repeat_interleave(32, 1)


def check_mx8(codes, scales, want, rel):
    """MXFP8 of values known to be within `rel` (an array or a number, absolute
    errors `rel * |want|` or an array of absolute bounds) of want."""
    d = torch.as_tensor(rel).double() * (want.abs() if not torch.is_tensor(rel) else 1.0)
    got = decode(codes, scales)
    s = scales.cpu().double() - 127
    lo = (want.abs() - d).clamp(min=0).view(*scales.shape, 32).amax(2)
    hi = (want.abs() + d).view(*scales.shape, 32).amax(2)
    # the least power of two with amax <= 448 * 2^e, for some amax in [lo, hi]
    assert bool((lo <= 448 * torch.exp2(s)).all())
    assert bool(((hi > 224 * torch.exp2(s)) | (scales.cpu() == 0)).all())
    step = torch.exp2(s - 10).repeat_interleave(32, 1)
    bound = torch.maximum((want.abs() + d) * 2.0 ** -4, step) + d
    err = (got - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,off", [(1, 32, 0, 0), (3, 64, 0, 0), (7, 96, 5, 3),
                                               (130, 2080, 32, 1), (33, 8192, 0, 0)])
def test_quant_dequant(rows, cols, pad, off, dtype):
    x = rand(rows, cols, seed=1, std=3.0).to(DT[dtype])
    x[rows // 2, :32] = 0
    x[0, 1] = 448.0                      # a block whose largest value is a border
    x[rows - 1, cols - 32:] *= 2.0 ** -120
    codes, scales = A.adahop_mx8_quant(strided(x, pad, off))
    check_mx8(codes, scales, x.double(), 0.0)
    assert int(scales[rows // 2, 0]) == (0 if rows > 1 else int(scales[rows // 2, 0]))
    want = decode(codes, scales)
    assert torch.equal(A.adahop_mx8_dequant(codes, scales, torch.float32).cpu().double(), want)
    out = strided(torch.zeros(rows, cols, dtype=torch.bfloat16), pad, off)
    got = A.adahop_mx8_dequant(strided(codes.cpu(), pad, off), strided(scales.cpu(), 3, 1), out=out)
    assert torch.equal(got.cpu().double(), want)


def test_quant_every_border():
    """Blocks whose largest value sits at, just above and just below 1.75 * 2^k,
    and every rounding tie of E4M3."""
    e = torch.arange(-118, 120).double()
    top = 1.75 * torch.exp2(e)
    x = torch.zeros(3 * len(e), 32)
    x[0::3, 0] = top.float()
    x[1::3, 5] = -torch.nextafter(top.float(), torch.tensor(float("inf")))
    x[2::3, 31] = torch.nextafter(top.float(), torch.tensor(0.0))
    codes, scales = A.adahop_mx8_quant(x.to(DEV))
    s = scales.cpu().int().view(-1, 3) - 127
    k = (e - 8).int()
    assert torch.equal(s[:, 0], k) and torch.equal(s[:, 1], k + 1) and torch.equal(s[:, 2], k)
    # ties: odd multiples of half a step in every binade, exact in fp32
    v = torch.tensor([(8 + f + 0.5) * 2.0 ** (q - 3) for q in range(-6, 8) for f in range(8)]
                     + [(f + 0.5) * 2.0 ** -9 for f in range(8)])
    v = v[v <= 448]
    y = torch.zeros(len(v), 32)
    y[:, 0] = 448.0
    y[:, 1] = v
    y[:, 2] = -v
    c = A.adahop_mx8_quant(y.to(DEV))[0].cpu()
    want = v.double()
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    got = decode(c, torch.full((len(v), 1), 127, dtype=torch.uint8))
    assert torch.equal(got[:, 1], torch.round(want / step) * step)
    assert torch.equal(got[:, 2], -got[:, 1])


def test_non_finite_blocks():
    x = torch.ones(4, 96)
    x[0, 3] = float("inf")
    x[1, 40] = float("nan")
    x[2, 95] = float("-inf")
    x[3, 64:] = torch.finfo(torch.float32).max
    codes, scales = A.adahop_mx8_quant(x.to(DEV))
    v = A.adahop_mx8_dequant(codes, scales, torch.float32).cpu()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(v.view(4, 3, 32).isnan().all(2), bad)
    assert torch.equal(v.view(4, 3, 32).isnan().any(2), bad)
    # fp32's largest value rounds to 2^128: a finite MXFP8 value that fp32 cannot hold
    assert bool((decode(codes, scales)[3, 64:] == 2.0 ** 128).all())
    assert torch.equal(scales.cpu() == 255, bad)


# ---- RMS norm ---------------------------------------------------------------
# Longest chain of additions of a row's sum: 32 in a thread, 6 over a wave, 16
# over waves; half of it reaches rstd, with the mean's, eps', root's and
# division's roundings.
RSTD = (54 / 2 + 4) * U
NORM_Y = RSTD + 3 * U


NORM_SIZES = [(1, 32), (5, 64), (3, 480), (9, 544), (4, 1024), (5, 1056), (7, 2048), (2, 2080), (3, 4096),
              (2, 4128), (2, 8192), (2, 8224), (1, 16384), (2, 16416), (1, 32768)]


def norm_ref(h, gain, eps):
    rstd = (h.double().square().mean(1) + eps) ** -0.5
    return h.double() * rstd[:, None] * gain.double(), rstd


@pytest.mark.parametrize("xt,rt", [("bf16", None), ("f32", None), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_rmsnorm(rows, cols, xt, rt):
    x = rand(rows, cols, seed=2).to(DT[xt])
    gain = (1 + rand(cols, seed=3, std=0.2)).to(DT["f32" if cols % 64 else "bf16"])
    r = None if rt is None else rand(rows, cols, seed=4, std=4.0).to(DT[rt])
    got = A.adahop_rmsnorm(x.to(DEV), gain.to(DEV), None if r is None else r.to(DEV), eps=1e-5, mx8=True,
                           bf16=True, save_rstd=True)
    h = x if r is None else (x.float() + r.float()).to(DT[rt])
    if r is None:
        assert got.h is None
    else:
        assert torch.equal(got.h.cpu(), h)
    y, rstd = norm_ref(h, gain, 1e-5)
    assert bool(((got.rstd.cpu().double() - rstd).abs() <= RSTD * rstd).all())
    assert bool(((got.y.cpu().double() - y).abs() <= (BF + NORM_Y) * y.abs()).all())
    check_mx8(got.codes, got.scales, y, NORM_Y)


@pytest.mark.parametrize("rows,cols", [(3, 1), (5, 7), (4, 513), (3, 2049), (2, 4101), (1, 32767)])
def test_rmsnorm_odd_columns(rows, cols):
    """Odd widths, rows that start anywhere, the stream updated in place."""
    x = strided(rand(rows, cols, seed=5, dtype=torch.bfloat16), 3, 1)
    r = rand(rows, cols, seed=6)
    gain = rand(cols, seed=7, dtype=torch.bfloat16)
    h = (x.float().cpu() + r)
    stream = strided(r, 1, 3)
    got = A.adahop_rmsnorm(x, gain.to(DEV), stream, mx8=False, bf16=True, h=stream)
    assert got.h.data_ptr() == stream.data_ptr() and torch.equal(stream.cpu(), h)
    y, _ = norm_ref(h, gain, 1e-5)
    assert bool(((got.y.cpu().double() - y).abs() <= (BF + NORM_Y) * y.abs()).all())
    assert got.codes is None and got.rstd is None


def test_rmsnorm_extremes():
    """A row of zeros gives zeros, a NaN its whole row, an infinity NaN and
    zeros, eps = 0 a row of zeros NaN; other rows are untouched."""
    x = torch.ones(5, 64)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    gain = torch.ones(64)
    got = A.adahop_rmsnorm(x.to(DEV), gain.to(DEV), mx8=True, bf16=True)
    y = got.y.cpu().float()
    v = A.adahop_mx8_dequant(got.codes, got.scales, torch.float32).cpu()
    assert bool((y[1] == 0).all()) and bool((v[1] == 0).all())
    assert bool(y[2].isnan().all()) and bool(v[2].isnan().all())
    assert bool(y[3, 9].isnan()) and bool((y[3, 10:] == 0).all()) and bool(v[3, :32].isnan().all())
    assert bool((y[0] == 1).all()) and bool((v[4] == 1).all())
    z = A.adahop_rmsnorm(x.to(DEV), gain.to(DEV), eps=0.0, mx8=False, bf16=True).y.cpu()
    assert bool(z[1].isnan().all()) and bool((z[0] == 1).all())
    empty = A.adahop_rmsnorm(torch.empty(0, 64, device=DEV), gain.to(DEV), save_rstd=True)
    assert empty.codes.shape == (0, 64) and empty.rstd.shape == (0,)


def norm_back_ref(dy, h, gain, rstd, dh):
    g, hh, s = dy.double() * gain.double(), h.double(), rstd.double()[:, None]
    n = hh * s
    c = (g * n).mean(1, keepdim=True)
    dx = s * (g - n * c)
    # magnitudes that the roundings act on
    mag = s * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, mag, (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)


@pytest.mark.parametrize("yt,ht,with_dh", [("bf16", "bf16", True), ("bf16", "f32", False),
                                           ("f32", "bf16", False), ("f32", "f32", True)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (9, 512), (70, 520), (5, 1024), (6, 2041),
                                       (3, 2056), (4, 4096), (3, 8192), (2, 8200), (2, 16385), (1, 32768),
                                       (4500, 48), (1300, 2104)])
def test_rmsnorm_backward(rows, cols, yt, ht, with_dh):
    h = rand(rows, cols, seed=8, std=3.0).to(DT[ht])
    dy = rand(rows, cols, seed=9).to(DT[yt])
    gain = (1 + rand(cols, seed=10, std=0.2)).to(DT[yt])
    dh = rand(rows, cols, seed=11).to(DT[ht]) if with_dh else None
    rstd = ((h.double().square().mean(1) + 1e-5) ** -0.5).float()
    dx, dgain = A.adahop_rmsnorm_backward(strided(dy, 1, 1), strided(h, 3), gain.to(DEV), rstd.to(DEV),
                                          None if dh is None else strided(dh, 2, 1))
    want, mag, wgain, mgain = norm_back_ref(dy, h, gain, rstd, dh)
    out = BF if ht == "bf16" else U
    tol = out * want.abs() + (1 + out) * (54 + 10) * U * mag
    assert bool(((dx.cpu().double() - want).abs() <= tol).all())
    # a column's chain: a thread's rows, 4 waves, the parts a wave adds, 16 waves
    chain = -(-rows // 1024) + 4 + 64 + 16 + 3
    assert bool(((dgain.cpu().double() - wgain).abs() <= chain * U * mgain + 1e-300).all())
    again = A.adahop_rmsnorm_backward(strided(dy, 1, 1), strided(h, 3), gain.to(DEV), rstd.to(DEV),
                                      None if dh is None else strided(dh, 2, 1), gain_grad=False)
    assert again[1] is None and torch.equal(again[0], dx)


def test_rmsnorm_backward_differences():
    """The gradient of sum(w * y) by central differences of the definition in
    64 bits, and by the operators."""
    rows, cols, eps = 3, 40, 1e-5
    h, gain, w = rand(rows, cols, seed=12), 1 + rand(cols, seed=13, std=0.3), rand(rows, cols, seed=14)

    def loss(hh, gg):
        return float((norm_ref(hh, gg, eps)[0] * w.double()).sum())

    rstd = A.adahop_rmsnorm(h.to(DEV), gain.to(DEV), eps=eps, mx8=False, bf16=True, save_rstd=True).rstd
    dx, dgain = A.adahop_rmsnorm_backward(w.to(DEV), h.to(DEV), gain.to(DEV), rstd)
    for i, j in ((0, 0), (1, 17), (2, 39)):
        d = torch.zeros(rows, cols, dtype=torch.float64)
        d[i, j] = 1e-5
        num = (loss(h.double() + d, gain) - loss(h.double() - d, gain)) / 2e-5
        assert abs(num - float(dx[i, j])) <= 1e-5 * (1 + abs(num))
        e = torch.zeros(cols, dtype=torch.float64)
        e[j] = 1e-5
        num = (loss(h, gain.double() + e) - loss(h, gain.double() - e)) / 2e-5
        assert abs(num - float(dgain[j])) <= 1e-5 * (1 + abs(num))


def test_rmsnorm_backward_no_rows():
    e = torch.empty(0, 96, device=DEV)
    dx, dgain = A.adahop_rmsnorm_backward(e, e, torch.ones(96, device=DEV), torch.empty(0, device=DEV))
    assert dx.shape == (0, 96) and bool((dgain == 0).all())


# ---- linear layer -----------------------------------------------------------
def weights(N, K, fmt, seed):
    w = rand(N, K, seed=seed, std=0.5)
    if fmt == "MXFP8":
        c, s = A.adahop_mx8_quant(w.to(DEV))
        return (c, s), decode(c, s)
    c, s, _ = A.adahop_iht_quant(w.to(torch.bfloat16).to(DEV), "COLS", hadamard_block=0)
    return (c, s), decode4(c, s)


def activations(m, K, seed):
    x = rand(m, K, seed=seed)
    x[:, K // 3] *= 30
    c, s = A.adahop_mx8_quant(x.to(DEV))
    return (c, s), decode(c, s)


def act_ref(z, act):
    """(f, f') in 64 bits."""
    if act == "NONE":
        return z, torch.ones_like(z)
    if act == "RELU":
        return z.clamp(min=0), (z > 0).double()
    if act == "SILU":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "GELU":
        c = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    p = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * p, p + z * p * (1 - p) * k * (1 + 3 * 0.044715 * z * z)


def linear_ref(va, vb, bias, act, gated, residual):
    """(z, bound of z's error, out, bound of out's error before its rounding)."""
    m, K = va.shape
    z = va @ vb.t()
    # per 16 products the matrix cores drop at most 16 * 2^-13 of the largest;
    # the fp32 sums over K / 64 steps and 8 parts, at most
    # (K / 64 + 16) roundings of sums below sum |a b|
    mag = va.abs() @ vb.abs().t()
    top = torch.zeros_like(z)
    for k in range(0, K, 16):
        pa, pb = va[:, k:k + 16], vb[:, k:k + 16]
        top += (pa[:, None, :] * pb[None]).abs().amax(2)
    dz = 16 * 2.0 ** -13 * top + (K / 64 + 16) * U * mag
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * z.abs()
    n = z.shape[1] // 2 if gated else z.shape[1]
    f, slope = act_ref(z[:, :n], act)
    # activations bend by |f''| <= 1.2 (relu: slopes 0 or 1, so dz itself
    # bounds the change); their own evaluation: 16 roundings of max(|f|, |z| / 16)
    df = dz[:, :n] * torch.clamp(slope.abs() + 1.2 * dz[:, :n], max=1.2)
    if act == "RELU":
        df = dz[:, :n]
    if act != "NONE":
        df = df + 16 * U * (f.abs() + z[:, :n].abs() / 16)
    out, dout = f, df
    if gated:
        up, dup = z[:, n:], dz[:, n:]
        out, dout = f * up, df * up.abs() + f.abs() * dup + df * dup + U * (f * up).abs()
    if residual is not None:
        out = out + residual.double()
        dout = dout + U * out.abs()
    return z, dz, out, dout


def run_linear(m, n, K, fmt, act="NONE", gated=False, bias=None, residual=False, mx8=False, save_z=False,
               strides=False, seed=20):
    N = 2 * n if gated else n
    a, va = activations(m, K, seed)
    b, vb = weights(N, K, fmt, seed + 1)
    bv = None if bias is None else rand(N, seed=seed + 2).to(DT[bias])
    res = rand(m, n, seed=seed + 3, std=4.0, dtype=torch.bfloat16) if residual else None
    rd = None if res is None else strided(res, 3, 1) if strides else res.to(DEV)
    if strides:
        a = (strided(a[0].cpu(), 16), strided(a[1].cpu(), 5, 3))
        b = (strided(b[0].cpu(), 48), strided(b[1].cpu(), 3, 1))
    got = A.adahop_linear_mx(a, b, bias=None if bv is None else bv.to(DEV), act=act, gated=gated,
                             residual=rd, out_dtype="MXFP8" if mx8 else torch.bfloat16, save_z=save_z)
    z, dz, out, dout = linear_ref(va, vb, bv, act, gated, res)
    if save_z:
        err = (got.z.cpu().double() - z).abs()
        assert bool((err <= dz + BF * (z.abs() + dz)).all()), float((err / (dz + BF * z.abs())).max())
    else:
        assert got.z is None
    if mx8:
        check_mx8(got.out, got.scales, out, dout)
    else:
        err = (got.out.cpu().double() - out).abs()
        tol = dout + BF * (out.abs() + dout)
        assert bool((err <= tol).all()), float((err / tol).max())
        # root mean square: the rounding, and a ten-thousandth for the products
        assert float(err.norm()) <= (BF / math.sqrt(3) + 1e-4) * float(out.norm()) + 1e-3 * float(z.norm())
    return got


SIZES = [(1, 32, 32), (1, 64, 96), (2, 1, 64), (3, 33, 128), (15, 48, 160), (16, 64, 512), (17, 100, 544),
         (31, 31, 992), (33, 160, 1024), (47, 96, 2080), (64, 128, 512), (65, 130, 480), (100, 257, 1056),
         (130, 300, 256), (257, 258, 288), (200, 520, 4096 + 32)]


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", SIZES)
def test_linear_sizes(m, n, K, fmt):
    run_linear(m, n, K, fmt)
    run_linear(m, n, K, fmt, gated=True, act="SILU", save_z=True)


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("m,n,K", [(1, 32, 64), (5, 96, 160), (33, 64, 1024), (130, 288, 544), (300, 544, 512)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_mx8_out(m, n, K, fmt, gated):
    run_linear(m, n, K, fmt, act="SILU", gated=gated, mx8=True, bias="f32", save_z=gated)


@pytest.mark.parametrize("act", list(A.ACT))
@pytest.mark.parametrize("gated", [False, True])
def test_linear_epilogues(act, gated):
    for m, n, K in ((9, 70, 96), (140, 290, 256)):
        run_linear(m, n, K, "MXFP8", act=act, gated=gated, bias="bf16", residual=True, save_z=True, seed=30)
        run_linear(m, n, K, "MXFP4", act=act, gated=gated, residual=True, seed=40)


@pytest.mark.parametrize("m,n,K", [(1, 33, 96), (20, 63, 544), (150, 261, 1056)])
@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
def test_linear_strides(m, n, K, fmt):
    """Operands inside larger buffers whose other bytes are NaN."""
    run_linear(m, n, K, fmt, residual=True, bias="f32", strides=True)


def test_linear_residual_in_place():
    a, _ = activations(40, 128, 50)
    b, _ = weights(72, 128, "MXFP8", 51)
    r = rand(40, 72, seed=52, dtype=torch.bfloat16).to(DEV)
    want = A.adahop_linear_mx(a, b, residual=r).out
    got = A.adahop_linear_mx(a, b, residual=r, out=r).out
    assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


def test_linear_non_finite():
    """A NaN or an infinity reaches its own row and no other."""
    x = rand(20, 96, seed=53)
    x[3, 5], x[7, 90] = float("nan"), float("inf")
    a = A.adahop_mx8_quant(x.to(DEV))
    b, _ = weights(64, 96, "MXFP4", 54)
    bad = A.adahop_linear_mx(a, b).out.isnan()
    want = torch.zeros(20, dtype=torch.bool)
    want[3] = want[7] = True
    assert torch.equal(bad.all(1).cpu(), want) and torch.equal(bad.any(1).cpu(), want)


def test_linear_no_rows():
    b, _ = weights(64, 96, "MXFP4", 55)
    a = (torch.empty(0, 96, dtype=torch.uint8, device=DEV), torch.empty(0, 3, dtype=torch.uint8, device=DEV))
    assert A.adahop_linear_mx(a, b).out.shape == (0, 64)


def test_linear_deterministic():
    for m, n, K in ((1, 512, 4096), (40, 300, 2048), (300, 600, 4096)):
        a, _ = activations(m, K, 56)
        b, _ = weights(n, K, "MXFP4", 57)
        first = A.adahop_linear_mx(a, b).out
        for _ in range(3):
            assert torch.equal(A.adahop_linear_mx(a, b).out, first)


# ---- gradient of the epilogue -----------------------------------------------
@pytest.mark.parametrize("act", list(A.ACT))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,dt", [(1, 1, "bf16"), (3, 9, "f32"), (70, 256, "bf16"), (65, 263, "f32"),
                                    (600, 40, "bf16")])
def test_act_backward(m, n, dt, act, gated):
    N = 2 * n if gated else n
    z = rand(m, N, seed=60, std=2.0, dtype=torch.bfloat16)
    z[0, 0] = 0.0
    if m > 2:
        z[1, 0], z[2, 0] = 200.0, -200.0
    g = rand(m, n, seed=61).to(DT[dt])
    dz, dbias = A.adahop_act_backward(strided(g, 1, 1), strided(z, 2, 1), act=act, gated=gated, bias_grad=True)
    f, slope = act_ref(z[:, :n].double(), act)
    d = g.double() * slope
    # slopes: 24 roundings of 1 + |z| (below 32; they end there)
    mag = g.double().abs() * (24 * U * (1 + z[:, :n].double().abs().clamp(max=32)))
    if gated:
        up = z[:, n:].double()
        d2, mag2 = g.double() * f, g.double().abs() * 24 * U * z[:, :n].double().abs()
        d, mag = torch.cat((d * up, d2), 1), torch.cat((mag * up.abs(), mag2), 1)
    err = (dz.cpu().double() - d).abs()
    assert bool((err <= mag + BF * (d.abs() + mag)).all()), float((err / (mag + BF * d.abs())).max())
    chain = -(-m // 8) + 8 + 64 + 16
    tol = mag.sum(0) + chain * U * (d.abs() + mag).sum(0)
    assert bool(((dbias.cpu().double() - d.sum(0)).abs() <= tol + 1e-300).all())
    zz = z.to(DEV)
    inplace, none = A.adahop_act_backward(g.to(DEV), zz, act=act, gated=gated, dz=zz)
    assert none is None and torch.equal(inplace, dz) and inplace.data_ptr() == zz.data_ptr()


def test_act_backward_differences():
    for act in A.ACT:
        z = rand(2, 24, seed=62)
        z = torch.where(z.abs() < 0.05, z + 0.1, z).to(torch.bfloat16)     # away from relu's corner
        w = rand(2, 12, seed=63)
        dz, _ = A.adahop_act_backward(w.to(DEV), z.to(DEV), act=act, gated=True)

        def loss(v):
            return float((act_ref(v[:, :12], act)[0] * v[:, 12:] * w.double()).sum())

        for i, j in ((0, 0), (1, 11), (0, 12), (1, 23)):
            d = torch.zeros(2, 24, dtype=torch.float64)
            d[i, j] = 1e-6
            num = (loss(z.double() + d) - loss(z.double() - d)) / 2e-6
            assert abs(num - float(dz[i, j])) <= 2 * BF * abs(num) + 1e-5, (act, i, j)


def test_act_backward_no_rows():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    dz, dbias = A.adahop_act_backward(z[:, :32], z, act="SILU", gated=True, bias_grad=True)
    assert dz.shape == (0, 64) and bool((dbias == 0).all())


# ---- streams and graphs -----------------------------------------------------
def block(x, gain, stream, up, down):
    """Pre-norm gated layer and its output added to the stream."""
    n = A.adahop_rmsnorm(x, gain, stream)
    h = A.adahop_linear_mx((n.codes, n.scales), up, act="SILU", gated=True, out_dtype="MXFP8")
    return A.adahop_linear_mx((h.out, h.scales), down, residual=n.h).out


@pytest.mark.parametrize("m", [1, 40, 300])
def test_block_on_a_stream_and_in_a_graph(m):
    D, F = 256, 512
    x, stream = rand(m, D, seed=70, dtype=torch.bfloat16).to(DEV), rand(m, D, seed=71, dtype=torch.bfloat16).to(DEV)
    gain = torch.ones(D, device=DEV)
    up, _ = weights(2 * F, D, "MXFP4", 72)
    down, _ = weights(D, F, "MXFP8", 73)
    want = block(x, gain, stream, up, down)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(x, gain, stream, up, down)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(x, gain, stream, up, down)
    for k in range(4):
        x.copy_(rand(m, D, seed=74 + k, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, block(x, gain, stream, up, down)), k
        torch.cuda.synchronize()


def test_backward_in_a_graph():
    rows, cols = 300, 512
    dy, h = rand(rows, cols, seed=80).to(DEV), rand(rows, cols, seed=81).to(DEV)
    z = rand(rows, 2 * cols, seed=82, dtype=torch.bfloat16).to(DEV)
    gain, rstd = torch.ones(cols, device=DEV), torch.rand(rows, device=DEV) + 0.5

    def both():
        dx, dgain = A.adahop_rmsnorm_backward(dy, h, gain, rstd)
        dz, dbias = A.adahop_act_backward(dx, z, act="GELU", gated=True, bias_grad=True)
        return dx, dgain, dz, dbias

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(4):
        dy.copy_(rand(rows, cols, seed=83 + k))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, both()):
            assert torch.equal(a, b), k
        torch.cuda.synchronize()


# ---- the binding's refusals ---------------------------------------------------
def test_binding_refusals():
    a, _ = activations(4, 64, 90)
    b, _ = weights(32, 64, "MXFP8", 91)
    x = torch.zeros(4, 64, device=DEV)
    g = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        A.adahop_linear_mx(a, (b[0][:, :48], b[1]))
    with pytest.raises(ValueError):
        A.adahop_linear_mx(a, (b[0], b[1][:, :1]))
    with pytest.raises(ValueError):
        A.adahop_linear_mx(a, b, bias=torch.zeros(31, device=DEV))
    with pytest.raises(ValueError):
        A.adahop_linear_mx(a, b, residual=torch.zeros(4, 31, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        A.adahop_linear_mx(a, b, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        A.adahop_linear_mx((a[0].float(), a[1]), b)
    with pytest.raises(ValueError):
        A.adahop_linear_mx((a[0].cpu(), a[1].cpu()), b)
    with pytest.raises(A.AdahopError):
        A.adahop_linear_mx(a, (b[0][:31], b[1][:31]), gated=True)
    with pytest.raises(KeyError):
        A.adahop_linear_mx(a, b, act="TANH")
    with pytest.raises(ValueError):
        A.adahop_rmsnorm(x.t(), torch.ones(4, device=DEV), mx8=False, bf16=True)
    with pytest.raises(A.AdahopError):
        A.adahop_rmsnorm(x, g, mx8=False)
    with pytest.raises(A.AdahopError):
        A.adahop_rmsnorm(x[:, :40], g[:40])
    with pytest.raises(TypeError):
        A.adahop_rmsnorm(x.half(), g)
    with pytest.raises(ValueError):
        A.adahop_rmsnorm(x, g, h=x)
    with pytest.raises(TypeError):
        A.adahop_rmsnorm_backward(x, x, g, torch.ones(4, device=DEV), dh=x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        A.adahop_rmsnorm_backward(x, x, g, torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        A.adahop_act_backward(x, x.to(torch.bfloat16), gated=True)
    with pytest.raises(A.AdahopError):
        A.adahop_rmsnorm(x[:1].expand(4, 64), g)
