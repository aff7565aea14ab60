"""Sizes at which one launch would have 2^32 threads or more: the calls have to
take them in pieces. Rows and columns around the pieces' borders are compared
with calls of their own on them, or with the definition."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_linear import DEV, rand
from test_gpu_linear_tiles import check_at, codes

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free_memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_norm_wide_rows():
    """2^22 rows of which 16 waves share each: 104 GB."""
    rows, cols = (1 << 22) + 40, 8224
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x.copy_(rand(1, cols, seed=1, dtype=torch.bfloat16).to(DEV).expand(rows, cols))
    borders = [slice(0, 40), slice((1 << 21) - 20, (1 << 21) + 20), slice((1 << 22) - 20, (1 << 22) + 40)]
    for k, at in enumerate(borders):
        x[at] = rand(at.stop - at.start, cols, seed=2 + k, dtype=torch.bfloat16).to(DEV)
    gain = (1 + rand(cols, seed=9, std=0.2)).to(DEV)
    got = A.adahop_rmsnorm(x, gain, save_rstd=True)
    for at in borders:
        part = A.adahop_rmsnorm(x[at], gain, save_rstd=True)
        for a, b in zip((got.codes, got.scales, got.rstd), (part.codes, part.scales, part.rstd)):
            assert torch.equal(a[at], b)


@pytest.mark.parametrize("gated", [False, True])
def test_column_sums_of_many_columns(gated):
    """Bias gradients of 2^26 columns and more."""
    m, N = 3, (1 << 26) + 80
    n = N // 2 if gated else N
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn(m, N, device=DEV, generator=g).to(torch.bfloat16)
    dout = torch.randn(m, n, device=DEV, generator=g)
    dz, dbias = A.adahop_act_backward(dout, z, act="RELU", gated=gated, bias_grad=True)
    zf = z.float()
    want = dout * (zf[:, :n] > 0)
    if gated:
        want = torch.cat((want * zf[:, n:], dout * zf[:, :n].clamp(min=0)), 1)
    assert torch.equal(dz, want.to(torch.bfloat16))
    # two additions, each within 2^-24 of sums below sum |dz|
    tol = 2.0 ** -23 * want.abs().sum(0)
    assert bool(((dbias - want.double().sum(0)).abs() <= tol).all())


@pytest.mark.parametrize("gated,N", [(False, (1 << 29) + 96), (True, (1 << 30) - 64)])
def test_linear_of_many_columns(gated, N):
    """Weights of 2^29 rows and more, 9 and 17 GB."""
    check_at(codes(2, 32, 10), codes(N, 32, 11, "MXFP4"), "MXFP4", act="RELU" if gated else "NONE", gated=gated)
