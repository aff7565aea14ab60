"""How g of the cross entropy's gradient is held, on the host: what is refused, the
workspace that each way asks for, and the binding. No GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_binding_host import OnGpu, standin  # noqa: F401
from test_xent_abi import INVALID, WORKSPACE, bf16, f32, i64, status, u8, xent_back_args


@pytest.mark.parametrize("g,want", [(0, WORKSPACE), (1, WORKSPACE), (2, INVALID), (-1, INVALID)])
def test_refusals(g, want):
    assert status("adahop_xent_backward", xent_back_args(g=g)) == want


def test_reserved():
    for i in (1, 2, 3):
        a = xent_back_args()
        a.reserved[i] = 1
        assert status("adahop_xent_backward", a) == INVALID


def test_layout(tmp_path):
    """g took a reserved field's place: a program that was compiled when there was
    none passes as many bytes as are read, and asks for SPLIT."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "adahop.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu\\n", sizeof(adahop_xent_backward_args), offsetof(adahop_xent_backward_args, g),'
                   ' offsetof(adahop_xent_backward_args, dw_dtype));\nreturn ADAHOP_XENT_G_SPLIT; }\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-I" + include, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    a = A.XentBackwardArgs
    assert [int(v) for v in got] == [160, 144, 140]
    assert ctypes.sizeof(a) == 160 and a.g.offset == a.reserved.offset == 144 and a.dw_dtype.offset == 140


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
