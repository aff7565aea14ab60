"""Values of each of the linear layer's kernels at the sizes of linear_cases.py,
on rows and columns at the tiles' borders, against the definition in 64 bits;
tolerances as derived in test_gpu_linear.py."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from linear_cases import all_cases, name
from test_gpu_linear import BF, DEV, check_mx8, linear_ref, rand
from test_gpu_linear_tiles import at_rows, codes, values

pytestmark = pytest.mark.gpu


def borders(n):
    """Ends of tiles of 16 .. 256, those of the last tiles among them."""
    at = {0, 1, n // 2, n - 2, n - 1}
    for step in (16, 32, 64, 128, 256):
        for edge in (step, (n - 1) // step * step):
            at |= {edge - 1, edge}
    return torch.tensor(sorted(i for i in at if 0 <= i < n))


@pytest.mark.parametrize("c", all_cases(), ids=name)
def test_values(c):
    m, n, K, fmt, gated, mx8 = c
    N = 2 * n if gated else n
    a, b = codes(m, K, 300), codes(N, K, 301, fmt)
    bias = rand(N, seed=302, std=4.0)
    residual = None if mx8 else rand(m, n, seed=303, std=40.0, dtype=torch.bfloat16)
    act = "SILU" if gated else "NONE"
    got = A.adahop_linear_mx(a, b, bias=bias.to(DEV), act=act, gated=gated, save_z=True,
                             residual=None if mx8 else residual.to(DEV),
                             out_dtype="MXFP8" if mx8 else torch.bfloat16)
    r, c0 = borders(m), borders(n)
    if mx8:                                    # whole blocks
        blocks = torch.unique(c0 // 32)
        c0 = (32 * blocks[:, None] + torch.arange(32)).flatten()
    cols = torch.cat((c0, n + c0)) if gated else c0
    z, dz, out, dout = linear_ref(values(at_rows(a, r)), values(at_rows(b, cols), fmt), bias[cols], act, gated,
                                  None if mx8 else residual[r][:, c0])
    err = (got.z[r.to(DEV)][:, cols.to(DEV)].cpu().double() - z).abs()
    assert bool((err <= dz + BF * (z.abs() + dz)).all()), float((err / (dz + BF * z.abs())).max())
    if mx8:
        check_mx8(got.out.cpu()[r][:, c0], got.scales.cpu()[r][:, blocks], out, dout)
    else:
        err = (got.out[r.to(DEV)][:, c0.to(DEV)].cpu().double() - out).abs()
        assert bool((err <= dout + BF * (out.abs() + dout)).all()), float((err / (dout + BF * out.abs())).max())


@pytest.mark.parametrize("c", [c for c in all_cases() if c[0] * c[1] < 300000], ids=name)
def test_every_value(c):
    """The whole output against fp32 products of the same values: a tile that is
    left out or stored in another's place."""
    m, n, K, fmt, gated, mx8 = c
    a, b = codes(m, K, 310), codes(2 * n if gated else n, K, 311, fmt)
    got = A.adahop_linear_mx(a, b, gated=gated, out_dtype="MXFP8" if mx8 else torch.bfloat16)
    out = A.adahop_mx8_dequant(got.out, got.scales, torch.float32).cpu().double() if mx8 else got.out.cpu().double()
    z = (values(a).float() @ values(b, fmt).float().t()).double()
    want = z[:, :n] * z[:, n:] if gated else z
    # the output's rounding (MXFP8: of the row's largest magnitude at most) and 1e-3 of
    # the row's root mean square for both products
    scale = want.abs().amax(1, keepdim=True) * 2.0 ** -4 if mx8 else want.abs() * BF
    assert bool(((out - want).abs() <= scale + 1e-3 * want.square().mean(1, keepdim=True).sqrt()
                 + 1e-3 * want.abs()).all())
