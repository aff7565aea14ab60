"""The cross entropy's gradient at logits of +-1e4, and beside rows whose logits are
infinite or NaN; tolerances as derived in test_gpu_xent.py and test_gpu_xent_g.py."""
import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_gpu_xent import DEV, case, check, say
from test_gpu_xent_g import gradients

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,D", [(65, 515, 64), (300, 257, 136), (9, 4099, 72)])
@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_large_logits(T, V, D, g, dt):
    """No exponential overflows, and what is left of those near the largest is right."""
    say("large logits", T, V, D, g, dt)
    h, w, y, dloss, dlse = case(T, V, D, seed=T, wstd=50.0)
    h = (h.float() * 30).to(torch.bfloat16)
    lse = A.adahop_xent(h, w, y).lse
    assert float(lse.abs().amax()) > 1e4
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, g=g, dh_dtype=dt, dw_dtype=dt)
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, dlse, 1.0, dt, g)
    assert float(rh.abs().amax()) > 10 and bool(torch.isfinite(dh).all()) and bool(torch.isfinite(dw).all())
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)


@pytest.mark.parametrize("shift", [-60.0, 3.0])
def test_lse_of_the_callers(shift):
    """Any lse goes: exponentials far below 1 and above it."""
    T, V, D = 70, 300, 64
    h, w, y, dloss, dlse = case(T, V, D, seed=12)
    lse = A.adahop_xent(h, w, y).lse - shift
    dh, dw = A.adahop_xent_backward(h, w, y, lse, dloss, dlse, dh_dtype=torch.float32, dw_dtype=torch.float32)
    rh, rw, eh, ew = gradients(h, w, y, lse, dloss, dlse, 1.0, torch.float32, "SPLIT")
    check("dh", dh, rh, eh)
    check("dw", dw, rw, ew)


@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
@pytest.mark.parametrize("T,V,D", [(70, 700, 64), (300, 2049, 136)])
def test_infinities_and_nans(T, V, D, g):
    """Row 0 has logits of +inf, row 1 of NaN, row 2 of -inf alone: their dh is NaN
    throughout, as the formula gives, and so is dw, to which every row belongs. The
    other rows' dh is as without them."""
    say("not finite", T, V, D, g)
    h, w, y, dloss, dlse = case(T, V, D, seed=5, ignored=0.0)
    h[:, 0] = 0.0
    w[:, 0] = 0.0
    fine = A.adahop_xent(h, w, y)
    want, _ = A.adahop_xent_backward(h, w, y, fine.lse, dloss, dlse, g=g)
    w[:, 0] = 1.0
    h[0, 0], h[2, 0] = float("inf"), float("-inf")
    h[1, 1] = float("nan")
    got = A.adahop_xent(h, w, y)
    assert torch.equal(got.lse[3:], fine.lse[3:])
    dh, dw = A.adahop_xent_backward(h, w, y, got.lse, dloss, dlse, g=g)
    assert torch.isnan(dh[:3]).all() and torch.isnan(dw).all()
    assert torch.equal(dh[3:, 1:], want[3:, 1:]) and torch.isfinite(dh[3:]).all()


@pytest.mark.parametrize("g", ["SPLIT", "BF16"])
def test_one_infinite_logit(g):
    """A logit of -inf (weight -inf under a hidden state of 1): its probability is 0
    and g of it too, unless it is the target's; g of 0 beside the infinite weight is
    NaN in that column of dh, the rest of dh and dw are finite and right."""
    T, V, D = 70, 300, 64
    say("one infinite logit", g)
    h, w, y, dloss, _ = case(T, V, D, seed=6, ignored=0.0)
    y = torch.where(y == 7, 8, y)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[7, 0] = float("-inf")
    got = A.adahop_xent(h, w, y)
    assert torch.isfinite(got.lse).all() and torch.isfinite(got.loss).all()
    dh, dw = A.adahop_xent_backward(h, w, y, got.lse, dloss, g=g, dh_dtype=torch.float32, dw_dtype=torch.float32)
    # without that entry
    rest = torch.arange(V, device=DEV) != 7
    rh, rw, eh, ew = gradients(h, w[rest], y - (y > 7).long(), got.lse, dloss, None, 1.0, torch.float32, g)
    assert torch.isnan(dh[:, 0]).all() and bool((dw[7] == 0).all())
    check("dh", dh[:, 1:], rh[:, 1:], eh[:, 1:])
    check("dw", dw[rest], rw, ew)
