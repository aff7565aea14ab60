"""The norm, MXFP8 and linear-layer entry points on the host: every refusal
comes back as a status before any launch. No GPU: the pointers are fakes that
no call below dereferences."""
import ctypes

import pytest

import mxfp4_precision_gemms_amd as A

P = 4096   # a fake, aligned address
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def norm_args(**kw):
    a = dict(rows=4, cols=64, x=P, ld_x=64, gain=P, codes=P, ld_codes=64, scales=P, ld_scales=2,
             eps=1e-5)
    a.update(kw)
    return A.RmsnormArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=32800), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(ld_x=63), INVALID), (dict(x=None), INVALID),
    (dict(gain=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(cols=48), INVALID), (dict(ld_codes=63), INVALID), (dict(ld_scales=1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x_dtype=2), INVALID), (dict(gain_dtype=-1), INVALID),
    (dict(residual=P, ld_residual=64), INVALID),                      # no h
    (dict(residual=P, ld_residual=63, h=P, ld_h=64), INVALID),
    (dict(residual=P, ld_residual=64, h=P, ld_h=63), INVALID),
    (dict(residual=P, ld_residual=64, h=P, ld_h=64, residual_dtype=7), INVALID),
    (dict(y=P, ld_y=63), INVALID),
    (dict(rows=0, x=None), OK),
])
def test_rmsnorm_refusals(change, status):
    assert A.lib().adahop_rmsnorm(ctypes.byref(norm_args(**change)), None) == status
    assert bool(A.lib().adahop_last_error()) == (status != OK)


def test_rmsnorm_null_and_reserved():
    assert A.lib().adahop_rmsnorm(None, None) == INVALID
    a = norm_args()
    a.reserved[2] = 1
    assert A.lib().adahop_rmsnorm(ctypes.byref(a), None) == INVALID


def back_args(**kw):
    a = dict(rows=4, cols=50, dy=P, ld_dy=50, h=P, ld_h=50, gain=P, rstd=P, dx=P, ld_dx=50, dgain=P)
    a.update(kw)
    return A.RmsnormBackwardArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=32769), UNSUPPORTED),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(gain=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(ld_dy=49), INVALID),
    (dict(ld_h=49), INVALID), (dict(ld_dx=49), INVALID), (dict(dh=P, ld_dh=49), INVALID),
    (dict(dy_dtype=2), INVALID), (dict(h_dtype=3), INVALID), (dict(gain_dtype=9), INVALID),
    (dict(), WORKSPACE), (dict(rows=0, dgain=None), OK),
])
def test_rmsnorm_backward_refusals(change, status):
    assert A.lib().adahop_rmsnorm_backward(ctypes.byref(back_args(**change)), None, 0, None) == status


def test_rmsnorm_backward_workspace():
    lib = A.lib()
    need = lib.adahop_rmsnorm_backward_workspace_size(4, 50)
    assert need >= 50 * 4
    args = back_args()
    assert lib.adahop_rmsnorm_backward(ctypes.byref(args), P, need - 1, None) == WORKSPACE
    assert str(need) in lib.adahop_last_error().decode()
    assert lib.adahop_rmsnorm_backward(ctypes.byref(args), P + 4, need, None) == UNSUPPORTED
    assert lib.adahop_rmsnorm_backward(None, P, need, None) == INVALID
    assert lib.adahop_rmsnorm_backward_workspace_size(-1, 50) == 0


def linear_args(**kw):
    a = dict(m=4, N=64, K=96, a_codes=P, ld_a_codes=96, a_scales=P, ld_a_scales=3, b_codes=P,
             ld_b_codes=96, b_scales=P, ld_b_scales=3, out=P, ld_out=64, b_format=1)
    a.update(kw)
    return A.LinearArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=80), INVALID),
    (dict(m=1 << 30), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED), (dict(K=1 << 30), UNSUPPORTED),
    (dict(a_codes=None), INVALID), (dict(a_scales=None), INVALID), (dict(b_codes=None), INVALID),
    (dict(b_scales=None), INVALID), (dict(out=None), INVALID), (dict(b_format=2), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(gated=2), INVALID),
    (dict(gated=1, N=63), INVALID), (dict(ld_a_codes=80), INVALID), (dict(ld_b_codes=95), INVALID),
    (dict(ld_a_scales=2), INVALID), (dict(ld_b_scales=2), INVALID), (dict(ld_out=63), INVALID),
    (dict(bias=P, bias_dtype=2), INVALID), (dict(residual=P, ld_residual=63), INVALID),
    (dict(z=P, ld_z=63), INVALID), (dict(gated=1, z=P, ld_z=32), INVALID),
    (dict(N=48, out_scales=P, ld_out_scales=2), INVALID),
    (dict(out_scales=P, ld_out_scales=1), INVALID),
    (dict(gated=1, out_scales=P, ld_out_scales=0), INVALID),
    (dict(a_codes=P + 8), UNSUPPORTED), (dict(b_codes=P + 4), UNSUPPORTED),
    (dict(ld_a_codes=104), UNSUPPORTED), (dict(b_format=0, ld_b_codes=56), UNSUPPORTED),
    (dict(m=0, a_codes=None, out=None), OK),
])
def test_linear_refusals(change, status):
    assert A.lib().adahop_linear_mx(ctypes.byref(linear_args(**change)), None, 0, None) == status


def test_linear_reserved_and_null():
    a = linear_args()
    a.reserved[0] = 1
    assert A.lib().adahop_linear_mx(ctypes.byref(a), None, 0, None) == INVALID
    assert A.lib().adahop_linear_mx(None, None, 0, None) == INVALID
    assert A.lib().adahop_linear_mx_workspace_size(-1, 64, 96, 1, 0) == 0


def act_call(dout=P, dtype=0, ldd=64, z=P, ldz=64, m=4, N=64, act=2, gated=0, dz=P, lddz=64,
             dbias=None, ws=None, n=0):
    return A.lib().adahop_act_backward(dout, dtype, ldd, z, ldz, m, N, act, gated, dz, lddz, dbias,
                                       ws, n, None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(N=0), INVALID), (dict(m=1 << 30), UNSUPPORTED), (dict(act=5), INVALID),
    (dict(gated=3), INVALID), (dict(gated=1, N=63), INVALID), (dict(dtype=2), INVALID),
    (dict(dout=None), INVALID), (dict(z=None), INVALID), (dict(dz=None), INVALID),
    (dict(ldd=63), INVALID), (dict(ldz=63), INVALID), (dict(lddz=63), INVALID),
    (dict(dbias=P), WORKSPACE), (dict(dbias=P, ws=P, n=8), WORKSPACE),
    (dict(dbias=P, ws=P + 8, n=1 << 20), UNSUPPORTED), (dict(m=0, dout=None, z=None, dz=None), OK),
])
def test_act_backward_refusals(change, status):
    assert act_call(**change) == status


@pytest.mark.parametrize("rows,cols,ld,ldc,lds,dtype,src,status", [
    (-1, 32, 32, 32, 1, 0, P, INVALID), (4, 0, 32, 32, 1, 0, P, INVALID),
    (4, 48, 48, 48, 2, 0, P, INVALID), (4, 64, 63, 64, 2, 0, P, INVALID),
    (4, 64, 64, 63, 2, 0, P, INVALID), (4, 64, 64, 64, 1, 0, P, INVALID),
    (4, 64, 64, 64, 2, 3, P, INVALID), (4, 64, 64, 64, 2, 0, None, INVALID),
    (0, 64, 64, 64, 2, 0, None, OK)])
def test_mx8_refusals(rows, cols, ld, ldc, lds, dtype, src, status):
    lib = A.lib()
    assert lib.adahop_mx8_quant(src, dtype, rows, cols, ld, P, ldc, P, lds, None) == status
    assert lib.adahop_mx8_dequant(P, ldc, P, lds, rows, cols, src, dtype, ld, None) == status


def test_linear_far_rows_of_b():
    for change in (dict(ld_b_codes=1 << 25), dict(ld_b_scales=1 << 25)):
        assert A.lib().adahop_linear_mx(ctypes.byref(linear_args(**change)), None, 0, None) == UNSUPPORTED
