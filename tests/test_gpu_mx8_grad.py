"""Gradients from activations kept in MXFP8 against their definitions in 64 bits
at the kept values. Tolerances as in test_gpu_linear.py: they count roundings (u =
2^-24, bf16's half step 2^-8)."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import BF, DEV, DT, U, act_ref, decode, norm_back_ref, rand, strided

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def kept(rows, cols, seed, std=2.0, outliers=True):
    """MXFP8 codes, scales (CPU) and values (fp64) of a matrix."""
    v = rand(rows, cols, seed=seed, std=std)
    if outliers and cols > 40:
        v[:, 7] *= 100.0
    c, s = (t.cpu() for t in A.adahop_mx8_quant(v.to(DEV)))
    return c, s, decode(c, s)


def spread(c, s, pad, off=0):
    return strided(c, pad, off), strided(s, 1, 1)


# ---- activation ---------------------------------------------------------------
@pytest.mark.parametrize("act", list(A.ACT))
@pytest.mark.parametrize("m,N,gated,dt", [(1, 32, True, "bf16"), (1, 32, False, "f32"), (3, 96, True, "f32"),
                                          (70, 544, True, "bf16"), (65, 288, False, "bf16"),
                                          (300, 64, False, "bf16"), (5000, 96, True, "bf16")])
def test_act_backward(m, N, gated, dt, act):
    say("act", m, N, gated, dt, act)
    n = N // 2 if gated else N
    c, s, z = kept(m, N, seed=1)
    g = rand(m, n, seed=2).to(DT[dt])
    r = A.adahop_act_backward_mx8(strided(g, 1, 1), spread(c, s, 3, 5), act=act, gated=gated, bias_grad=True,
                                  remake_out=True)
    f, slope = act_ref(z[:, :n], act)
    d = g.double() * slope
    # slopes and values: 24 roundings of 1 + |z| (slopes end below 32)
    mag = g.double().abs() * (24 * U * (1 + z[:, :n].abs().clamp(max=32)))
    ef = 24 * U * z[:, :n].abs()
    if gated:
        up = z[:, n:]
        d, mag = (torch.cat((d * up, g.double() * f), 1), torch.cat((mag * up.abs(), g.double().abs() * ef), 1))
        f, ef = f * up, ef * up.abs() + U * (f * up).abs()
    err = (r.dz.cpu().double() - d).abs()
    assert bool((err <= mag + BF * (d.abs() + mag)).all())
    assert bool(((r.out.cpu().double() - f).abs() <= ef + BF * (f.abs() + ef)).all())
    chain = -(-m // 8) + 8 + 64 + 16
    tol = mag.sum(0) + chain * U * (d.abs() + mag).sum(0)
    assert bool(((r.dbias.cpu().double() - d.sum(0)).abs() <= tol + 1e-300).all())
    # the bf16 form at the same values, which bf16 holds
    dz, dbias = A.adahop_act_backward(g.to(DEV), z.to(torch.bfloat16).to(DEV), act=act, gated=gated, bias_grad=True)
    assert torch.equal(r.dz, dz) and torch.equal(r.dbias, dbias)
    alone = A.adahop_act_backward_mx8(strided(g, 1, 1), spread(c, s, 3, 5), act=act, gated=gated)
    assert torch.equal(alone.dz, dz) and alone.out is None and alone.dbias is None


def test_act_backward_differences():
    for act in A.ACT:
        c, s, z = kept(2, 32, seed=3, std=1.0)
        w = rand(2, 16, seed=4)
        dz = A.adahop_act_backward_mx8(w.to(DEV), (c.to(DEV), s.to(DEV)), act=act, gated=True).dz

        def loss(v):
            return float((act_ref(v[:, :16], act)[0] * v[:, 16:] * w.double()).sum())

        for i, j in ((0, 0), (1, 15), (0, 16), (1, 31)):
            if act == "RELU" and abs(float(z[i, j % 16])) < 0.05:
                continue
            d = torch.zeros(2, 32, dtype=torch.float64)
            d[i, j] = 1e-6
            num = (loss(z + d) - loss(z - d)) / 2e-6
            assert abs(num - float(dz[i, j])) <= 2 * BF * abs(num) + 1e-5, (act, i, j)


def test_act_backward_borders_of_rows():
    """dz and out between other rows: nothing beside them changes."""
    m, N = 9, 96
    c, s, _ = kept(m, N, seed=5)
    g = rand(m, N, seed=6)
    buf = torch.full((m, N + 7), -3.0, dtype=torch.bfloat16, device=DEV)
    r = A.adahop_act_backward_mx8(g.to(DEV), (c.to(DEV), s.to(DEV)), act="GELU", dz=buf[:, 5:5 + N])
    want = A.adahop_act_backward_mx8(g.to(DEV), (c.to(DEV), s.to(DEV)), act="GELU").dz
    assert torch.equal(r.dz, want) and bool((buf[:, :5] == -3).all()) and bool((buf[:, 5 + N:] == -3).all())


# ---- norm -----------------------------------------------------------------------
@pytest.mark.parametrize("yt,xt,with_dh", [("bf16", "bf16", True), ("bf16", "f32", False), ("f32", "bf16", False),
                                           ("f32", "f32", True)])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (9, 512), (70, 544), (5, 1024), (6, 2080), (4, 4096),
                                       (3, 8192), (2, 8224), (2, 16416), (1, 32768), (4500, 64), (1300, 2112)])
def test_rmsnorm_backward(rows, cols, yt, xt, with_dh):
    say("norm", rows, cols, yt, xt, with_dh)
    c, s, h = kept(rows, cols, seed=8, std=3.0)
    dy = rand(rows, cols, seed=9).to(DT[yt])
    gain = (1 + rand(cols, seed=10, std=0.2)).to(DT[yt])
    dh = rand(rows, cols, seed=11).to(DT[xt]) if with_dh else None
    rstd = ((h.square().mean(1) + 1e-5) ** -0.5).float()
    kw = dict(dx_dtype=DT[xt])
    dev_dh = None if dh is None else strided(dh, 2, 1)
    dx, dgain = A.adahop_rmsnorm_backward_mx8(strided(dy, 1, 1), spread(c, s, 3), gain.to(DEV), rstd.to(DEV), dev_dh,
                                              **kw)
    want, mag, wgain, mgain = norm_back_ref(dy, h, gain, rstd, dh)
    out = BF if xt == "bf16" else U
    tol = out * want.abs() + (1 + out) * (54 + 10) * U * mag
    assert bool(((dx.cpu().double() - want).abs() <= tol).all())
    chain = -(-rows // 1024) + 4 + 64 + 16 + 3
    assert bool(((dgain.cpu().double() - wgain).abs() <= chain * U * mgain + 1e-300).all())
    # rows at cache lines, and without the gain's gradient
    again, none = A.adahop_rmsnorm_backward_mx8(dy.to(DEV), (c.to(DEV), s.to(DEV)), gain.to(DEV), rstd.to(DEV),
                                                None if dh is None else dh.to(DEV), gain_grad=False, **kw)
    assert none is None and torch.equal(again, dx)
    if with_dh:
        over, g2 = A.adahop_rmsnorm_backward_mx8(strided(dy, 1, 1), spread(c, s, 3), gain.to(DEV), rstd.to(DEV), dev_dh,
                                                 dx=dev_dh)
        assert over.data_ptr() == dev_dh.data_ptr() and torch.equal(over, dx) and torch.equal(g2, dgain)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 96), (70, 544), (6, 2080), (2, 16416), (2, 32768), (4500, 64)])
def test_rmsnorm_backward_over_dy(rows, cols, dt):
    """dx in dy's place: the same bits."""
    c, s, h = kept(rows, cols, seed=12)
    dy = rand(rows, cols, seed=13).to(DT[dt])
    gain = (1 + rand(cols, seed=14, std=0.2)).to(DEV)
    rstd = ((h.square().mean(1) + 1e-5) ** -0.5).float().to(DEV)
    for place in (lambda t: t.to(DEV), lambda t: strided(t, 1, 1)):
        dx, dgain = A.adahop_rmsnorm_backward_mx8(place(dy), spread(c, s, 3), gain, rstd, dx_dtype=DT[dt])
        over = place(dy)
        got, g2 = A.adahop_rmsnorm_backward_mx8(over, spread(c, s, 3), gain, rstd, dx=over)
        assert got.data_ptr() == over.data_ptr() and torch.equal(got, dx) and torch.equal(g2, dgain)


def test_rmsnorm_backward_no_rows():
    z = torch.empty(0, 64, device=DEV)
    h = torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.empty(0, 2, dtype=torch.uint8, device=DEV)
    dx, dgain = A.adahop_rmsnorm_backward_mx8(z, h, torch.ones(64, device=DEV), torch.empty(0, device=DEV))
    assert dx.shape == (0, 64) and bool((dgain == 0).all())


# ---- weight gradient --------------------------------------------------------------
def wgrad_check(gy, x, got, dt, T):
    """Sums of T exact products in any order, the output's rounding."""
    want = gy.double().t() @ x
    mag = gy.double().abs().t() @ x.abs()
    half = BF if dt == torch.bfloat16 else U
    tol = (T + 2) * U * mag * (1 + half) + half * want.abs()
    err = (got.cpu().double() - want).abs()
    say(f"  at most {float((err / tol.clamp(min=1e-300)).amax()):.3f} of the tolerance")
    assert bool((err <= tol).all())


# T, Din, Dout: one of each, T around a stage (64), a pair of stages and where
# codes are loaded three stages ahead, ragged tiles, several tiles a workgroup
# (more than 256) with few and many stages, products split along T
@pytest.mark.parametrize("T,Din,Dout", [(1, 32, 8), (2, 96, 40), (63, 32, 8), (64, 64, 16), (65, 288, 264),
                                        (127, 256, 256), (128, 544, 72), (129, 32, 512), (193, 544, 264),
                                        (300, 96, 1032), (1000, 224, 520), (4100, 288, 264), (70, 8224, 2056),
                                        (130, 5152, 4104), (330, 4128, 4616), (9001, 64, 24)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_wgrad(T, Din, Dout, dt):
    say("wgrad", T, Din, Dout, dt)
    c, s, x = kept(T, Din, seed=12)
    gy = rand(T, Dout, seed=13, dtype=torch.bfloat16)
    got = A.adahop_gemm_wgrad_mx8(gy.to(DEV), (c.to(DEV), s.to(DEV)), out_dtype=dt)
    torch.cuda.synchronize()
    wgrad_check(gy, x, got, dt, T)


@pytest.mark.parametrize("T,Din,Dout", [(5, 32, 8), (200, 288, 264), (1100, 544, 520)])
def test_wgrad_rows_apart(T, Din, Dout):
    """Rows apart, with NaNs between them, whose memory ends with the last row."""
    say("wgrad rows apart", T, Din, Dout)
    c, s, x = kept(T, Din, seed=14)
    gy = rand(T, Dout, seed=15, dtype=torch.bfloat16)

    def ends(t, pad, fill):
        rows, cols = t.shape
        flat = torch.full(((rows - 1) * (cols + pad) + cols,), fill, dtype=t.dtype, device=DEV)
        v = flat.as_strided((rows, cols), (cols + pad, 1))
        v.copy_(t)
        return v

    buf = torch.full((Dout, Din + 9), -7.0, device=DEV)
    out = A.adahop_gemm_wgrad_mx8(ends(gy, 16, float("nan")), (ends(c, 48, 0x7F), ends(s, 5, 255)),
                                  out=buf[:, 3:3 + Din])
    wgrad_check(gy, x, out, torch.float32, T)
    assert bool((buf[:, :3] == -7).all()) and bool((buf[:, 3 + Din:] == -7).all())


def test_wgrad_every_code_and_scale():
    """One row: dW is the values themselves, every code under every scale, as the
    dequantizer gives them in bf16 (below 2^-126 they may be 0)."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).reshape(-1, 32)
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(8)
    c, s = codes.reshape(1, -1).to(DEV), scales.reshape(1, -1).to(DEV)
    want = A.adahop_mx8_dequant(c, s)[0].float()
    gy = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    gy[0, 0] = 1.0
    got = A.adahop_gemm_wgrad_mx8(gy, (c, s), out_dtype=torch.float32)[0]
    tiny = want.abs() < 2.0 ** -126
    bad = ~((got == want) | (got.isnan() & want.isnan()) | (tiny & (got == 0)))
    say("differ:", [(int(i) // 256, int(i) % 256, float(got[i]), float(want[i])) for i in bad.nonzero()[:8, 0]])
    assert not bool(bad.any())


def test_wgrad_no_rows():
    x = torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.empty(0, 2, dtype=torch.uint8, device=DEV)
    gy = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((24, 64), 5.0, dtype=dt, device=DEV)
        assert bool((A.adahop_gemm_wgrad_mx8(gy, x, out=out) == 0).all())


def test_wgrad_non_finite():
    """An infinity of GY and a NaN block of X reach their row and columns alone."""
    T, Din, Dout = 200, 288, 264
    c, s, x = kept(T, Din, seed=16)
    gy = rand(T, Dout, seed=17, dtype=torch.bfloat16)
    plain = A.adahop_gemm_wgrad_mx8(gy.to(DEV), (c.to(DEV), s.to(DEV)))
    s[150, 2] = 255
    c[150, 64:96] = 0x7F
    gy[70, 200] = float("inf")
    got = A.adahop_gemm_wgrad_mx8(gy.to(DEV), (c.to(DEV), s.to(DEV)))
    assert bool(got[:, 64:96].isnan().all())
    assert not bool(got[200].isfinite().any())
    keep = torch.ones(Dout, Din, dtype=torch.bool, device=DEV)
    keep[200], keep[:, 64:96] = False, False
    assert torch.equal(got[keep], plain[keep])


def test_workspaces_of_the_callers():
    T, Din, Dout = 3000, 288, 264
    c, s, _ = kept(T, Din, seed=18)
    x, gy = (c.to(DEV), s.to(DEV)), rand(T, Dout, seed=19, dtype=torch.bfloat16).to(DEV)
    need = A.lib().adahop_gemm_wgrad_mx8_workspace_size(T, Din, Dout)
    assert need > 0
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    got = A.adahop_gemm_wgrad_mx8(gy, x, ws=ws)
    assert torch.equal(got, A.adahop_gemm_wgrad_mx8(gy, x)) and bool((ws[need:] == 0xA5).all())
    with pytest.raises(A.AdahopError):
        A.adahop_gemm_wgrad_mx8(gy, x, ws=ws[:need - 1])


# ---- together ---------------------------------------------------------------------
def test_in_a_graph_and_on_streams():
    """The block's backward pass from its checkpoints, captured, replayed on new
    inputs with eager work between the replays."""
    T, D, F = 300, 256, 512
    gen = [rand(T, D, seed=20), rand(T, 2 * F, seed=21, std=1.5)]
    h, z = (list(A.adahop_mx8_quant(v.to(DEV))) for v in gen)
    dact = rand(T, F, seed=22, dtype=torch.bfloat16).to(DEV)
    dy = rand(T, D, seed=23, dtype=torch.bfloat16).to(DEV)
    gain, rstd = torch.ones(D, device=DEV), torch.rand(T, device=DEV) + 0.5

    def step():
        a = A.adahop_act_backward_mx8(dact, z, act="SILU", gated=True, bias_grad=True, remake_out=True)
        dw = A.adahop_gemm_wgrad_mx8(a.dz, h)
        dx, dgain = A.adahop_rmsnorm_backward_mx8(dy, h, gain, rstd, dy)
        return [*a, dw, dx, dgain]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        for to, v in ((h, rand(T, D, seed=30 + k)), (z, rand(T, 2 * F, seed=40 + k))):
            for t, new in zip(to, A.adahop_mx8_quant(v.to(DEV))):
                t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, step()):
            assert torch.equal(x, y), k
        torch.cuda.synchronize()
