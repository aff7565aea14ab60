"""How g of the cross entropy's gradient is held, on the host: what is refused, the
workspace that each way asks for, and the binding. No GPU."""
import ctypes

import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_binding_host import OnGpu, standin  # noqa: F401
from test_xent_abi import INVALID, WORKSPACE, bf16, f32, i64, status, u8, xent_back_args


@pytest.mark.parametrize("g,want", [(0, WORKSPACE), (1, WORKSPACE), (2, INVALID), (-1, INVALID)])
def test_refusals(g, want):
    assert status("adahop_xent_backward", xent_back_args(g=g)) == want


def test_reserved():
    for i in range(5):
        a = xent_back_args()
        a.reserved[i] = 1
        assert status("adahop_xent_backward", a) == INVALID


def size(**kw):
    a = xent_back_args(**kw)
    return A.lib().adahop_xent_backward_args_workspace_size(ctypes.byref(a))


@pytest.mark.parametrize("rows", [64, 65, 4096])
def test_workspaces(rows):
    """Two numbers of two bytes an element, or one."""
    padded = -(-rows // 64) * 64
    one = dict(rows=rows, vocab=10000, piece=512, dh=None)
    assert size(g=0, **one) - size(g=1, **one) == 2 * padded * 512
    assert size(g=2, **one) == 0


def test_binding(standin):  # noqa: F811
    kw = dict(h=bf16(4, 64), w=bf16(9, 64), targets=i64(4), lse=f32(4), dloss=f32(4), dh=bf16(4, 64), dw=f32(9, 64),
              ws=u8(64))
    with pytest.raises(KeyError):
        A.adahop_xent_backward(**kw, g="FP8")
    assert standin.launched() == []
    for g in ("SPLIT", "BF16"):
        A.adahop_xent_backward(**kw, g=g)
    assert standin.launched() == ["adahop_xent_backward"] * 2
