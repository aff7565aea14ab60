"""The cross entropy's and the MXFP8 gradients' entry points on the host: every
refusal comes back as a status before any launch, workspaces are asked for, and
the listed sizes take the tiles they stand for. No GPU: the pointers are fakes that
no call below dereferences."""
import ctypes
import shutil
import subprocess

import pytest
import torch

import mxfp4_precision_gemms_amd as A
from test_binding_host import OnGpu, standin  # noqa: F401
from test_launch_shapes import CSRC
from tile_cases import DH, DW, LOGITS, WGRAD

P = 4096   # a fake, aligned address
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def status(name, args):
    s = getattr(A.lib(), name)(ctypes.byref(args), None, 0, None)
    assert bool(A.lib().adahop_last_error()) == (s != OK)
    return s


def xent_args(**kw):
    a = dict(rows=4, vocab=100, dim=64, h=P, ld_h=64, w=P, ld_w=64, targets=P, loss=P, lse=P, scale=1.0)
    a.update(kw)
    return A.XentArgs(**a)


def xent_back_args(**kw):
    a = dict(rows=4, vocab=100, dim=64, h=P, ld_h=64, w=P, ld_w=64, targets=P, lse=P, dloss=P, dh=P, ld_dh=64,
             dw=P, ld_dw=64, scale=1.0)
    a.update(kw)
    return A.XentBackwardArgs(**a)


COMMON = [
    (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(dim=0), INVALID), (dict(dim=-8), INVALID),
    (dict(rows=1 << 30), UNSUPPORTED), (dict(vocab=1 << 30), UNSUPPORTED),
    (dict(rows=1 << 21, vocab=1 << 25), UNSUPPORTED),
    (dict(h=None), INVALID), (dict(w=None), INVALID), (dict(targets=None), INVALID), (dict(lse=None), INVALID),
    (dict(ld_h=56), INVALID), (dict(ld_w=63), INVALID), (dict(ld_h=68), UNSUPPORTED), (dict(ld_w=65), UNSUPPORTED),
    (dict(dim=60), UNSUPPORTED), (dict(h=P + 8), UNSUPPORTED), (dict(w=P + 2), UNSUPPORTED),
    (dict(ld_h=1 << 22), UNSUPPORTED), (dict(ld_w=1 << 40), UNSUPPORTED),
    (dict(target_dtype=2), INVALID), (dict(target_dtype=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(), WORKSPACE), (dict(rows=0), OK),
    (dict(ld_h=(1 << 22) - 8), WORKSPACE),
]


@pytest.mark.parametrize("change,want", COMMON + [(dict(loss=None), INVALID)])
def test_xent_refusals(change, want):
    assert status("adahop_xent", xent_args(**change)) == want


@pytest.mark.parametrize("change,want", [c for c in COMMON if c[0] != dict(rows=0)] + [
    (dict(dloss=None), INVALID), (dict(dh=None, dw=None), INVALID), (dict(ld_dh=63), INVALID),
    (dict(ld_dw=63), INVALID), (dict(dh_dtype=2), INVALID), (dict(dw_dtype=-1), INVALID), (dict(piece=-1), INVALID),
    (dict(rows=1 << 22, vocab=64), UNSUPPORTED), (dict(dh=None, ld_dh=0), WORKSPACE), (dict(dw=None, ld_dw=0), WORKSPACE),
    (dict(rows=0, dw=None), OK), (dict(ld_dh=65, ld_dw=77), WORKSPACE),
])
def test_xent_backward_refusals(change, want):
    assert status("adahop_xent_backward", xent_back_args(**change)) == want


def act_args(**kw):
    a = dict(m=4, N=64, dout=P, ld_dout=64, z_codes=P, ld_z_codes=64, z_scales=P, ld_z_scales=2, dz=P, ld_dz=64,
             dbias=P)
    a.update(kw)
    return A.ActBackwardMx8Args(**a)


@pytest.mark.parametrize("change,want", [
    (dict(m=-1), INVALID), (dict(N=0), INVALID), (dict(N=48), INVALID), (dict(m=1 << 30), UNSUPPORTED),
    (dict(N=1 << 30), UNSUPPORTED), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(gated=2), INVALID),
    (dict(dout_dtype=2), INVALID), (dict(ld_dout=63), INVALID), (dict(ld_z_codes=63), INVALID),
    (dict(ld_z_scales=1), INVALID), (dict(ld_dz=63), INVALID), (dict(out=P, ld_out=63), INVALID),
    (dict(gated=1, ld_dout=31), INVALID), (dict(gated=1, ld_dout=32, out=P, ld_out=32), WORKSPACE),
    (dict(dout=None), INVALID), (dict(z_codes=None), INVALID), (dict(z_scales=None), INVALID),
    (dict(dz=None), INVALID), (dict(), WORKSPACE), (dict(m=0, dbias=None, dout=None, dz=None), OK),
])
def test_act_backward_refusals(change, want):
    assert status("adahop_act_backward_mx8", act_args(**change)) == want


def norm_args(**kw):
    a = dict(rows=4, cols=64, dy=P, ld_dy=64, h_codes=P, ld_h_codes=64, h_scales=P, ld_h_scales=2, gain=P, rstd=P,
             dx=P, ld_dx=64, dgain=P)
    a.update(kw)
    return A.RmsnormBackwardMx8Args(**a)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=48), INVALID), (dict(cols=32800), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(dy=None), INVALID), (dict(h_codes=None), INVALID),
    (dict(h_scales=None), INVALID), (dict(gain=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID),
    (dict(ld_dy=63), INVALID), (dict(ld_h_codes=63), INVALID), (dict(ld_h_scales=1), INVALID), (dict(ld_dx=63), INVALID),
    (dict(dh=P, ld_dh=63), INVALID), (dict(dy_dtype=2), INVALID), (dict(dx_dtype=2), INVALID),
    (dict(gain_dtype=-1), INVALID), (dict(), WORKSPACE), (dict(rows=0, dgain=None), OK),
])
def test_rmsnorm_backward_refusals(change, want):
    assert status("adahop_rmsnorm_backward_mx8", norm_args(**change)) == want


def wgrad_args(**kw):
    a = dict(T=3000, Din=96, Dout=64, gy=P, ld_gy=64, x_codes=P, ld_x_codes=96, x_scales=P, ld_x_scales=3, out=P,
             ld_out=96)
    a.update(kw)
    return A.GemmWgradMx8Args(**a)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(Din=0), INVALID), (dict(Dout=0), INVALID), (dict(Din=80), INVALID),
    (dict(T=1 << 30), UNSUPPORTED), (dict(Din=1 << 30), UNSUPPORTED), (dict(Dout=1 << 30), UNSUPPORTED),
    (dict(Din=1 << 24, Dout=1 << 22), UNSUPPORTED), (dict(out_dtype=2), INVALID), (dict(ld_gy=63), INVALID),
    (dict(ld_x_codes=95), INVALID), (dict(ld_x_scales=2), INVALID), (dict(ld_out=95), INVALID),
    (dict(gy=None), INVALID), (dict(x_codes=None), INVALID), (dict(x_scales=None), INVALID), (dict(out=None), INVALID),
    (dict(Dout=60), UNSUPPORTED), (dict(ld_gy=68), UNSUPPORTED), (dict(ld_x_codes=104), UNSUPPORTED),
    (dict(gy=P + 8), UNSUPPORTED), (dict(x_codes=P + 8), UNSUPPORTED), (dict(ld_gy=1 << 22), UNSUPPORTED),
    (dict(ld_x_codes=1 << 23), UNSUPPORTED), (dict(ld_x_scales=1 << 23), UNSUPPORTED), (dict(), WORKSPACE),
    (dict(x_scales=P + 1, ld_x_scales=7, ld_out=97), WORKSPACE),
])
def test_wgrad_refusals(change, want):
    assert status("adahop_gemm_wgrad_mx8", wgrad_args(**change)) == want


@pytest.mark.parametrize("name,make", [
    ("adahop_xent", xent_args), ("adahop_xent_backward", xent_back_args), ("adahop_act_backward_mx8", act_args),
    ("adahop_rmsnorm_backward_mx8", norm_args), ("adahop_gemm_wgrad_mx8", wgrad_args)])
def test_null_reserved_and_workspaces(name, make):
    lib = A.lib()
    call = getattr(lib, name)
    assert call(None, None, 0, None) == INVALID
    a = make()
    a.reserved[3] = 1
    assert call(ctypes.byref(a), None, 0, None) == INVALID
    a = make()
    need = {"adahop_xent": lambda: lib.adahop_xent_workspace_size(4, 100),
            "adahop_xent_backward": lambda: lib.adahop_xent_backward_args_workspace_size(ctypes.byref(a)),
            "adahop_act_backward_mx8": lambda: lib.adahop_act_backward_workspace_size(4, 64, 0),
            "adahop_rmsnorm_backward_mx8": lambda: lib.adahop_rmsnorm_backward_workspace_size(4, 64),
            "adahop_gemm_wgrad_mx8": lambda: lib.adahop_gemm_wgrad_mx8_workspace_size(3000, 96, 64)}[name]()
    assert need > 0
    assert call(ctypes.byref(a), P, need - 1, None) == WORKSPACE
    assert call(ctypes.byref(a), None, need, None) == WORKSPACE
    assert call(ctypes.byref(a), P + 8, need, None) == UNSUPPORTED


def test_workspace_sizes():
    lib = A.lib()
    assert lib.adahop_xent_workspace_size(0, 100) == 0 and lib.adahop_xent_workspace_size(4, 0) == 0
    assert lib.adahop_xent_workspace_size(-1, 5) == 0 and lib.adahop_xent_workspace_size(1 << 30, 5) == 0
    assert lib.adahop_xent_workspace_size(8192, 131072) >= 8192 * (131072 // 64) * 8
    assert lib.adahop_xent_backward_args_workspace_size(None) == 0
    for bad in (dict(rows=0), dict(rows=-4), dict(piece=-1), dict(dim=60), dict(dh=None, dw=None)):
        a = xent_back_args(**bad)
        assert lib.adahop_xent_backward_args_workspace_size(ctypes.byref(a)) == 0, bad

    def size(**kw):
        a = xent_back_args(**kw)
        return lib.adahop_xent_backward_args_workspace_size(ctypes.byref(a))

    big = dict(rows=8192, vocab=131072, dim=4096, ld_h=4096, ld_w=4096, ld_dh=4096, ld_dw=4096)
    # the chosen pieces keep g within 1 GiB; a piece of the caller's is rounded up
    assert 1 << 30 <= size(**big) <= (1 << 30) + 4 * 8192 * 4096 + (256 << 20)
    assert size(piece=1, **big) == size(piece=256, **big) < size(piece=257, **big) == size(piece=512, **big)
    assert size(piece=1 << 40, **big) == size(piece=131072, **big) == size(piece=131071, **big)
    assert lib.adahop_gemm_wgrad_mx8_workspace_size(-1, 96, 64) == 0
    assert lib.adahop_gemm_wgrad_mx8_workspace_size(0, 96, 64) == 0
    assert lib.adahop_gemm_wgrad_mx8_workspace_size(1 << 30, 96, 64) == 0


def plans(tmp_path, cases):
    """(rows, columns, in parts) of the tiles of (m, n, K, a, b, may be split)."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "plans.cpp", tmp_path / "plans"
    src.write_text("\n".join(
        ["#include <cstdio>", '#include "tile_plan.h"', "using namespace adahop::tiles;", "int main() {"] +
        ["{ const ProductPlan p = product_plan(%d, %d, %d, %s, %s, %s, 256);"
         ' printf("%%d %%d %%d %%lld %%lld %%d\\n", tile_rows(p.tile), tile_cols(p.tile), (int)(p.split > 0),'
         " (long long)p.full, (long long)p.split, p.parts); }" % c for c in cases] + ["}", ""]))
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [[int(v) for v in line.split()] for line in out.split("\n")[:-1]]


def test_tiles_of_the_listed_sizes(tmp_path):
    """Each size of tile_cases.py takes the tile that it stands under: a constant
    that is set anew cannot leave a kernel without a test of its values."""
    listed = [(k, (T, V, D, "kAlong", "kAlong", "false")) for k, cs in LOGITS.items() for T, V, D in cs]
    listed += [(k, (T, D, V, "kAlong", "kAcross", "true")) for k, cs in DH.items() for T, V, D in cs]
    listed += [(k, (V, D, T, "kAcross", "kAcross", "true")) for k, cs in DW.items() for T, V, D in cs]
    listed += [(k, (Dout, Din, T, "kAcross", "kCodes", "true")) for k, cs in WGRAD.items() for T, Din, Dout in cs]
    for (k, c), got in zip(listed, plans(tmp_path, [c for _, c in listed])):
        assert (got[0], got[1], bool(got[2])) == k, (c, got)


def test_plans_cover_their_tiles(tmp_path):
    """Whole and split tiles make up all of them, no part is empty, and items stay
    within an int and a launch."""
    sizes = (1, 63, 64, 65, 1000, 4097, (1 << 22) - 1, (1 << 30) - 1)
    cases = [(m, n, K, a, b, s) for m in sizes for n in sizes for K in (1, 128, 1025, (1 << 30) - 1)
             for a, b, s in (("kAlong", "kAlong", "false"), ("kAlong", "kAcross", "true"), ("kAcross", "kCodes", "true"))
             if m * n < 1 << 46]
    for (m, n, K, a, b, s), (rows, cols, split, full, parted, parts) in zip(cases, plans(tmp_path, cases)):
        tiles = -(-m // rows) * -(-n // cols)
        assert full + parted == tiles and full >= 0
        assert parts >= 1 and (parts == 1) == (parted == 0) and (s == "true" or parts == 1)
        units = -(-K // 128)
        assert parts == 1 or 4 * parts <= units
        items = full + parted * parts
        assert items <= 2 ** 31 - 1 and (cols == 256 or items * 512 < 2 ** 32), (m, n, K, items)


# ---- the binding --------------------------------------------------------------
def bf16(*shape):
    return OnGpu(torch.zeros(*shape, dtype=torch.bfloat16))


def f32(*shape):
    return OnGpu(torch.zeros(*shape))


def u8(*shape):
    return OnGpu(torch.zeros(*shape, dtype=torch.uint8))


def i64(*shape):
    return OnGpu(torch.zeros(*shape, dtype=torch.int64))


@pytest.mark.parametrize("change,error", [
    (dict(h=torch.zeros(4, 64, dtype=torch.bfloat16)), ValueError), (dict(h=f32(4, 64)), TypeError),
    (dict(w=bf16(9, 72)), ValueError), (dict(w=torch.zeros(9, 64, dtype=torch.bfloat16)), ValueError),
    (dict(targets=i64(5)), ValueError), (dict(targets=i64(4, 1)), ValueError), (dict(targets=f32(4)), TypeError),
    (dict(targets=torch.zeros(4, dtype=torch.int64)), ValueError), (dict(lse=f32(3)), ValueError),
    (dict(lse=bf16(4)), TypeError), (dict(dloss=torch.zeros(4)), ValueError), (dict(dlse=f32(1)), ValueError),
    (dict(dh=bf16(4, 63)), ValueError), (dict(dw=bf16(8, 64)), ValueError),
    (dict(dh=OnGpu(torch.zeros(4, 64, dtype=torch.float16))), TypeError),
    (dict(ws=torch.zeros(64, dtype=torch.uint8)), ValueError),
])
def test_xent_backward_binding(standin, change, error):  # noqa: F811
    kw = dict(h=bf16(4, 64), w=bf16(9, 64), targets=i64(4), lse=f32(4), dloss=f32(4), dh=bf16(4, 64), dw=f32(9, 64))
    standin.size = 16
    if error is None:
        return
    with pytest.raises(error):
        A.adahop_xent_backward(**{**kw, **change})
    assert standin.launched() == []
    ws = u8(64)
    dh, dw = A.adahop_xent_backward(**kw, ws=ws)
    assert dh is kw["dh"] and dw is kw["dw"] and standin.launched() == ["adahop_xent_backward"]


@pytest.mark.parametrize("change,error", [
    (dict(GY=bf16(5, 8)), ValueError), (dict(GY=f32(4, 8)), TypeError), (dict(x=(u8(4, 64), u8(4, 3))), ValueError),
    (dict(x=(u8(4, 64), torch.zeros(4, 2, dtype=torch.uint8))), ValueError), (dict(x=(f32(4, 64), u8(4, 2))), TypeError),
    (dict(out=f32(8, 63)), ValueError), (dict(out=OnGpu(torch.zeros(8, 64, dtype=torch.float16))), TypeError)])
def test_wgrad_binding(standin, change, error):  # noqa: F811
    kw = dict(GY=bf16(4, 8), x=(u8(4, 64), u8(4, 2)), out=f32(8, 64))
    with pytest.raises(error):
        A.adahop_gemm_wgrad_mx8(**{**kw, **change})
    assert standin.launched() == []
    assert A.adahop_gemm_wgrad_mx8(**kw) is kw["out"]
    assert standin.launched() == ["adahop_gemm_wgrad_mx8"]


@pytest.mark.parametrize("change,error", [
    (dict(dout=bf16(4, 63)), ValueError), (dict(z=(u8(4, 64), u8(4, 1))), ValueError), (dict(act="TANH"), KeyError),
    (dict(gated=True), ValueError), (dict(dz=f32(4, 64)), TypeError)])
def test_act_binding(standin, change, error):  # noqa: F811
    kw = dict(dout=bf16(4, 64), z=(u8(4, 64), u8(4, 2)), act="SILU", dz=bf16(4, 64))
    with pytest.raises(error):
        A.adahop_act_backward_mx8(**{**kw, **change})
    assert standin.launched() == []
    assert A.adahop_act_backward_mx8(**kw).dz is kw["dz"]


@pytest.mark.parametrize("change,error", [
    (dict(dy=bf16(3, 64)), ValueError), (dict(h=(u8(4, 64), u8(5, 2))), ValueError), (dict(gain=f32(63)), ValueError),
    (dict(rstd=f32(3)), ValueError), (dict(rstd=bf16(4)), TypeError), (dict(dh=f32(4, 64)), TypeError),
    (dict(dx=OnGpu(torch.zeros(4, 64, dtype=torch.float16))), TypeError)])
def test_norm_binding(standin, change, error):  # noqa: F811
    kw = dict(dy=bf16(4, 64), h=(u8(4, 64), u8(4, 2)), gain=f32(64), rstd=f32(4), dx=bf16(4, 64), gain_grad=False)
    with pytest.raises(error):
        A.adahop_rmsnorm_backward_mx8(**{**kw, **change})
    assert standin.launched() == []
    assert A.adahop_rmsnorm_backward_mx8(**kw)[0] is kw["dx"]
