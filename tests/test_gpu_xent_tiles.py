"""The cross entropy, its gradient and the weight gradient from MXFP8 at the sizes
of tile_cases.py, which reach every tile, whole and in parts, and on operands past
4 GB; tolerances as derived in test_gpu_xent.py."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_xent import DEV, U, case, check, expected, gradients, logits, say
from tile_cases import DH, DW, LOGITS, WGRAD, flat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,D", flat(LOGITS))
def test_logits(T, V, D):
    say("logits", T, V, D)
    h, w, y, _, _ = case(T, V, D, seed=T)
    got = A.adahop_xent(h, w, y)
    loss, lse, e_loss, e_lse = expected(h, w, y, 1.0)
    check("lse", got.lse, lse, e_lse)
    check("loss", got.loss, loss, e_loss)
    again = A.adahop_xent(h, w, y)
    assert torch.equal(again.lse, got.lse) and torch.equal(again.loss, got.loss)


@pytest.mark.parametrize("which,c", [("dh", c) for c in flat(DH)] + [("dw", c) for c in flat(DW)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_products(which, c, dt):
    T, V, D = c
    say(which, T, V, D, dt)
    h, w, y, dloss, _ = case(T, V, D, seed=T + 1)
    lse = torch.logsumexp(logits(h, w, 1.0)[0], 1).float()

    def run():
        return A.adahop_xent_backward(h, w, y, lse, dloss, h_grad=which == "dh", w_grad=which == "dw", dh_dtype=dt,
                                      dw_dtype=dt)[0 if which == "dh" else 1]

    got = run()
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, None, 1.0, dt)
    check(which, got, rh if which == "dh" else rw, eh if which == "dh" else ew)
    assert torch.equal(run(), got)


def values(codes, scales):
    """fp64 values of MXFP8 (scale bytes 1 .. 254), on their device."""
    v = codes.view(torch.float8_e4m3fn).double().view(codes.shape[0], -1, 32)
    return (v * torch.exp2(scales.double() - 127)[:, :, None]).view(codes.shape)


@pytest.mark.parametrize("T,Din,Dout", flat(WGRAD))
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_wgrad(T, Din, Dout, dt):
    say("wgrad", T, Din, Dout, dt)
    g = torch.Generator().manual_seed(T + Din)
    x = A.adahop_mx8_quant(torch.randn(T, Din, generator=g).to(DEV))
    gy = torch.randn(T, Dout, generator=g).to(torch.bfloat16).to(DEV)
    got = A.adahop_gemm_wgrad_mx8(gy, x, out_dtype=dt)
    v, gd = values(*x), gy.double()
    half = torch.finfo(dt).eps / 2
    want = gd.t() @ v
    check("dw", got, want, (T + 2) * U * (gd.abs().t() @ v.abs()) * (1 + half) + half * want.abs())
    assert torch.equal(A.adahop_gemm_wgrad_mx8(gy, x, out_dtype=dt), got)


def test_weights_past_4_gb():
    """w and dw of 4.9 GB, in pieces, targets among the last entries."""
    T, V, D = 70, 600011, 4096
    say("past 4 GB", T, V, D)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.empty(V, D, dtype=torch.bfloat16, device=DEV)
    for i in range(0, V, 65536):
        w[i:i + 65536] = torch.randn(min(65536, V - i), D, generator=g, device=DEV) * 0.03
    h = torch.randn(T, D, generator=g, device=DEV).to(torch.bfloat16)
    y = torch.randint(V - 1000, V, (T,), generator=g, device=DEV)
    got = A.adahop_xent(h, w, y)
    hd = h.double()
    z = torch.cat([hd @ w[i:i + 65536].double().t() for i in range(0, V, 65536)], 1)
    lse = torch.logsumexp(z, 1)
    ez = (D + 2) * U * max(float((hd.abs() @ w[i:i + 65536].double().abs().t()).amax()) for i in range(0, V, 65536))
    X = float((z.amax(1) - z.amin(1)).amax())
    tol = ez + ((2 + 3 * X) + V / 1024 + 64) * U + 4 * U * (lse.abs() + float(z.abs().amax()) + 1)
    check("lse", got.lse, lse, tol)
    check("loss", got.loss, lse - z.gather(1, y[:, None])[:, 0], tol + ez + U * 30)
    dloss = torch.rand(T, generator=g, device=DEV) + 0.5
    p = (z - got.lse.double()[:, None]).exp()
    hot = torch.zeros_like(z).scatter_(1, y[:, None], 1.0)
    gz = dloss.double()[:, None] * (p - hot)
    eg = 2.0 ** -8 * gz.abs() + 1.01 * dloss.double()[:, None] * (p * (ez + (4 + 3 * X) * U) + 4 * U * hot)
    del z, p, hot
    dh, dw = A.adahop_xent_backward(h, w, y, got.lse, dloss, piece=70000)
    want, err = torch.zeros(T, D, dtype=torch.float64, device=DEV), torch.zeros(T, D, dtype=torch.float64, device=DEV)
    for i in range(0, V, 65536):
        part, e = w[i:i + 65536].double(), eg[:, i:i + 65536]
        want += gz[:, i:i + 65536] @ part
        err += e @ part.abs() + (V + 2) * U * (gz[:, i:i + 65536].abs() @ part.abs())
    check("dh", dh, want, err * 1.01 + 2.0 ** -8 * want.abs())
    for i in (0, 69999, 300000, V - 1000):
        rows = slice(i, min(i + 1500, V))
        want = gz[:, rows].t() @ hd
        err = eg[:, rows].t() @ hd.abs() + (T + 2) * U * (gz[:, rows].abs().t() @ hd.abs())
        check(f"dw from {i}", dw[rows], want, err * 1.01 + 2.0 ** -8 * want.abs())


def test_long_gradients_past_4_gb():
    """GY of 4.9 GB and X codes of 2.4 GB, contracted over 300007 rows."""
    T, Din, Dout = 300007, 8192, 8192
    say("past 4 GB", T, Din, Dout)
    g = torch.Generator(device=DEV).manual_seed(2)
    gy = torch.empty(T, Dout, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(T, Din, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, Din // 32, dtype=torch.uint8, device=DEV)
    for i in range(0, T, 32768):
        n = min(32768, T - i)
        gy[i:i + n] = torch.randn(n, Dout, generator=g, device=DEV)
        A.adahop_mx8_quant(torch.randn(n, Din, generator=g, device=DEV), codes[i:i + n], scales[i:i + n])
    got = A.adahop_gemm_wgrad_mx8(gy, (codes, scales), out_dtype=torch.float32)
    r, c = torch.tensor([0, 1, 255, 256, 4095, 8190, 8191], device=DEV), slice(7936, 8192)
    a, b = gy[:, r].double(), values(codes[:, c].contiguous(), scales[:, c.start // 32:].contiguous())
    want = a.t() @ b
    check("dw", got[r][:, c], want, (T + 2) * U * (a.abs().t() @ b.abs()) + U * want.abs())


def apart(t, ld):
    """A copy of t in rows ld elements apart; what lies between is NaN."""
    buf = torch.full(((t.shape[0] - 1) * ld + t.shape[1],), float("nan") if t.is_floating_point() else 255,
                     dtype=t.dtype, device=DEV)
    view = buf.as_strided(t.shape, (ld, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("T,Din,Dout", [(70, 288, 264), (300, 96, 1032), (70, 8224, 2056)])
def test_wgrad_rows_nearly_8_mb_apart(T, Din, Dout):
    say("8 MB", T, Din, Dout)
    g = torch.Generator(device=DEV).manual_seed(3)
    gy = torch.randn(T, Dout, generator=g, device=DEV).to(torch.bfloat16)
    x = A.adahop_mx8_quant(torch.randn(T, Din, generator=g, device=DEV))
    far = apart(x[0], (1 << 23) - 16), apart(x[1], (1 << 23) - 1)
    got = A.adahop_gemm_wgrad_mx8(apart(gy, (1 << 22) - 8), far)
    assert torch.equal(got, A.adahop_gemm_wgrad_mx8(gy, x))


@pytest.mark.parametrize("T,V,D", [(37, 300, 520), (300, 200, 520), (520, 777, 264)])
def test_cross_entropy_rows_nearly_8_mb_apart(T, V, D):
    say("8 MB", T, V, D)
    g = torch.Generator(device=DEV).manual_seed(4)
    h = torch.randn(T, D, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g, device=DEV) / D ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    dloss = torch.rand(T, generator=g, device=DEV)
    want = A.adahop_xent(h, w, y)
    far = apart(h, (1 << 22) - 8), apart(w, (1 << 22) - 8)
    got = A.adahop_xent(*far, y)
    assert torch.equal(got.loss, want.loss) and torch.equal(got.lse, want.lse)
    for a, b in zip(A.adahop_xent_backward(*far, y, got.lse, dloss), A.adahop_xent_backward(h, w, y, got.lse, dloss)):
        assert torch.equal(a, b)
