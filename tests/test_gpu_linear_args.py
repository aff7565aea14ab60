"""Arguments of the norm's gradient, the linear layer and the activation's
gradient that the header promises: dx over an input, a caller's workspace."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import DEV, DT, activations, rand, strided, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("over", ["dh", "dy", "h"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (5, 7, 1), (70, 520, 0), (6, 2041, 3), (3, 8200, 0), (2, 16385, 1),
                                           (1, 32768, 0), (4500, 48, 0), (1300, 2104, 8)])
def test_norm_gradient_over_an_input(rows, cols, pad, dt, over):
    """dx written over dh, dy or h is the dx of its own memory."""
    t = {k: strided(rand(rows, cols, seed=s, std=std).to(DT[dt]), pad, pad)
         for k, s, std in (("dy", 1, 1.0), ("h", 2, 3.0), ("dh", 3, 1.0))}
    gain = (1 + rand(cols, seed=4, std=0.2)).to(DEV)
    rstd = ((t["h"].double().square().mean(1) + 1e-5) ** -0.5).float()
    want, wgain = A.adahop_rmsnorm_backward(t["dy"], t["h"], gain, rstd, t["dh"])
    kept = {k: v.clone() for k, v in t.items()}
    dx, dgain = A.adahop_rmsnorm_backward(t["dy"], t["h"], gain, rstd, t["dh"], dx=t[over])
    assert dx.data_ptr() == t[over].data_ptr()
    assert torch.equal(dx, want) and torch.equal(dgain, wgain)
    for k in t:
        assert k == over or torch.equal(t[k], kept[k])


def marked(need):
    """A workspace of `need` bytes and 4096 more, all 0xA5."""
    return torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=DEV)


def untouched(ws, need):
    return bool((ws[need:] == 0xA5).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (70, 520), (4500, 48), (1300, 2104), (3, 16385), (0, 96)])
def test_norm_gradient_workspace(rows, cols):
    dy, h = rand(rows, cols, seed=5).to(DEV), rand(rows, cols, seed=6).to(DEV)
    gain, rstd = torch.ones(cols, device=DEV), torch.ones(rows, device=DEV)
    need = A.lib().adahop_rmsnorm_backward_workspace_size(rows, cols)
    ws = marked(need)
    got = A.adahop_rmsnorm_backward(dy, h, gain, rstd, ws=ws)
    assert untouched(ws, need)
    for a, b in zip(got, A.adahop_rmsnorm_backward(dy, h, gain, rstd)):
        assert torch.equal(a, b)
    with pytest.raises(A.AdahopError):
        A.adahop_rmsnorm_backward(dy, h, gain, rstd, ws=ws[:need - 1])


@pytest.mark.parametrize("m,n,gated", [(1, 1, False), (70, 256, True), (65, 263, False), (5000, 40, True), (0, 64, False)])
def test_act_gradient_workspace(m, n, gated):
    N = 2 * n if gated else n
    z, g = rand(m, N, seed=7, dtype=torch.bfloat16).to(DEV), rand(m, n, seed=8).to(DEV)
    need = A.lib().adahop_act_backward_workspace_size(m, N, int(gated))
    ws = marked(need)
    got = A.adahop_act_backward(g, z, act="SILU", gated=gated, bias_grad=True, ws=ws)
    assert untouched(ws, need)
    for a, b in zip(got, A.adahop_act_backward(g, z, act="SILU", gated=gated, bias_grad=True)):
        assert torch.equal(a, b)
    with pytest.raises(A.AdahopError):
        A.adahop_act_backward(g, z, act="SILU", gated=gated, bias_grad=True, ws=ws[:need - 1])


# Scales in another order (K no multiple of 512; tiles of 256 rows), K parts, both, neither;
# the size asked for is that of the output's type which needs more
@pytest.mark.parametrize("m,n,K,fmt,gated,mx8", [
    (333, 2050, 2080, "MXFP8", False, False), (33, 1024, 4096, "MXFP8", False, True),
    (300, 1000, 4128, "MXFP4", False, False), (2100, 5410, 288, "MXFP8", False, False),
    (333, 8192, 256, "MXFP4", True, True), (200, 4160, 14336, "MXFP4", True, False),
    (100, 4160, 512, "MXFP8", True, True), (3, 64, 96, "MXFP4", False, False)])
def test_linear_workspace(m, n, K, fmt, gated, mx8):
    N = 2 * n if gated else n
    a, _ = activations(m, K, 9)
    b, _ = weights(N, K, fmt, 10)
    need = A.lib().adahop_linear_mx_workspace_size(m, N, K, A.MX_FORMAT[fmt], int(gated))
    ws = marked(need)
    more = dict(gated=gated, out_dtype="MXFP8" if mx8 else torch.bfloat16)
    got = A.adahop_linear_mx(a, b, ws=ws, **more)
    assert untouched(ws, need)
    want = A.adahop_linear_mx(a, b, **more)
    assert torch.equal(got.out, want.out) and (not mx8 or torch.equal(got.scales, want.scales))
    if need:
        with pytest.raises(A.AdahopError):
            A.adahop_linear_mx(a, b, ws=ws[:need - 1], **more)
    # exact products need none
    exact = A.adahop_linear_mx(a, b, ws=ws[:0], products="EXACT", **more)
    again = A.adahop_linear_mx(a, b, products="EXACT", **more)
    assert torch.equal(exact.out, again.out)


def test_one_row_of_strided_operands():
    """Rows 104 bytes apart, of which only the third starts at 16 bytes."""
    a, _ = activations(3, 96, 11)
    b, _ = weights(64, 96, "MXFP4", 12)
    codes, scales = strided(a[0].cpu(), 8), strided(a[1].cpu(), 4)
    assert codes.stride(0) == 104
    got = A.adahop_linear_mx((codes[2:], scales[2:]), b).out
    assert torch.equal(got, A.adahop_linear_mx((a[0][2:], a[1][2:]), b).out)
