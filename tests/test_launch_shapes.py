"""The launch shapes of the norm and linear layer's kernels, computed on the
host by the headers that the kernels' launches use: no launch may have 2^32
threads or more in a dimension. No GPU."""
import os
import shutil
import subprocess

import pytest

from linear_cases import FEW, TILES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_precision_gemms_amd", "csrc")


def evaluate(tmp_path, lines):
    """Output lines of a program made of statements that print."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "shapes.cpp", tmp_path / "shapes"
    head = [f"#include {h}" for h in ("<cstdio>", "<initializer_list>", '"launch_shapes.h"', '"linear_plan.h"')]
    src.write_text("\n".join([*head, "using namespace adahop;", "int main() {", *lines, "}", ""]))
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]


def numbers(tmp_path, lines):
    return [[int(v) for v in line.split()] for line in evaluate(tmp_path, lines)]


def test_norm_launches(tmp_path):
    """A full launch of every class of columns, and the columns that a row's
    threads hold."""
    cols = sorted({1, 32768} | {c + d for c in (512, 1024, 2048, 4096, 8192, 16384) for d in (0, 1, 32)})
    got = numbers(tmp_path, ['for (long long c : {' + ", ".join(f"{c}ll" for c in cols) + '}) {',
                             'const NormShape s = norm_shape(c);',
                             'printf("%d %d %lld %d\\n", s.waves, s.groups,',
                             '(long long)norm_grid(kNormLaunchRows, s.waves), norm_block(s.waves)); }'])
    assert len(got) == len(cols)
    for c, (waves, groups, grid, block) in zip(cols, got):
        assert block in (256, 64 * waves) and block <= 1024
        assert grid * block < 2 ** 32, c
        assert 64 * waves * groups * 8 >= c and groups <= 4


def test_column_sum_launches(tmp_path):
    (grid, block, cols), = numbers(tmp_path, [
        'printf("%lld %d %lld\\n", (long long)reduce_grid(kReduceLaunchCols), kReduceBlock,',
        '(long long)kReduceLaunchCols);'])
    assert grid * block < 2 ** 32 and grid * 16 >= cols


def test_few_row_launches(tmp_path):
    """A launch of the widest piece, and of the widest gated layer, which goes
    at once."""
    (plain, gated, cols, most), = numbers(tmp_path, [
        'printf("%lld %lld %lld %lld\\n", (long long)few_wide_threads(kFewLaunchCols),',
        '(long long)few_wide_threads(kMaxGatedN / 2), (long long)kFewLaunchCols, (long long)kMaxGatedN);'])
    assert plain < 2 ** 32 and gated < 2 ** 32
    assert cols % 32 == 0 and most < 2 ** 30
    assert plain >= 8 * cols and gated >= 4 * most


@pytest.mark.parametrize("N,gated,status", [((1 << 30) - 1, 0, 1), (1 << 30, 0, 2), ((1 << 30) - 64, 1, 1),
                                            ((1 << 30) - 62, 1, 2), ((1 << 30) - 2, 1, 2)])
def test_widest_layer(N, gated, status):
    """(INVALID for ld_out, which is looked at later, and UNSUPPORTED)"""
    import ctypes

    import mxfp4_precision_gemms_amd as A
    a = A.LinearArgs(m=4, N=N, K=96, a_codes=4096, ld_a_codes=96, a_scales=4096, ld_a_scales=3, b_codes=4096,
                     ld_b_codes=96, b_scales=4096, ld_b_scales=3, out=4096, ld_out=64, b_format=1, gated=gated)
    assert A.lib().adahop_linear_mx(ctypes.byref(a), None, 0, None) == status


def test_exact_products_rule(tmp_path):
    """AUTO is exact for MXFP8 outputs of up to 32768 values, whatever K, the
    weights or the device; SCALED and EXACT are what they say."""
    cases = [(1, 32768), (1, 32800), (32, 1024), (33, 1024), (100, 320), (1024, 32), (1025, 32)]
    got = numbers(tmp_path, [
        f'printf("%d %d %d %d %d %d\\n", (int)exact_products(0, true, {m}, {n}), (int)exact_products(0, false, {m}, {n}),'
        f' (int)exact_products(1, true, {m}, {n}), (int)exact_products(1, false, {m}, {n}),'
        f' (int)exact_products(2, true, {m}, {n}), (int)exact_products(2, false, {m}, {n}));' for m, n in cases])
    for (m, n), g in zip(cases, got):
        assert g == [int(m * n <= 32768), 0, 0, 0, 1, 1], (m, n)


@pytest.mark.parametrize("products,status", [(-1, 1), (3, 1), (1, 3), (0, 3)])
def test_bad_products(products, status):
    """(1: INVALID; 3: WORKSPACE, which is looked at later)"""
    import ctypes

    import mxfp4_precision_gemms_amd as A
    a = A.LinearArgs(m=4096, N=4096, K=96, a_codes=4096, ld_a_codes=96, a_scales=4096, ld_a_scales=3, b_codes=4096,
                     ld_b_codes=96, b_scales=4096, ld_b_scales=3, out=4096, ld_out=4096, b_format=1,
                     products=products)
    assert A.lib().adahop_linear_mx_workspace_size(4096, 4096, 96, 1, 0) > 0
    assert A.lib().adahop_linear_mx(ctypes.byref(a), None, 0, None) == status


def test_kernels_of_the_listed_sizes(tmp_path):
    """Each size of linear_cases.py takes the kernel that it stands under, on a
    device of 256 compute units: a constant that is set anew cannot leave a
    kernel without a test of its values."""
    listed = [(None, c) for c in FEW] + [(kind, c) for kind, cases in TILES for c in cases]
    got = numbers(tmp_path, [
        '{ const TilePlan p = linear_tile_plan(%d, %d, %d, %d, %d, 256);\n'
        '  printf("%%d %%d %%d %%d\\n", (int)exact_products(0, %s, %d, %d),'
        ' (int)take_few(%d, p, %d, %d, %d, %d, %s, 256), 256 >> p.shape, p.parts); }'
        % (m, n, K, fmt == "MXFP4", gated, str(mx8).lower(), m, n, m, n, K, fmt == "MXFP4", gated, str(mx8).lower())
        for _, (m, n, K, fmt, gated, mx8) in listed])
    for (kind, c), (exact, few, rows, parts) in zip(listed, got):
        assert not exact and few == (kind is None), (c, few, rows, parts)
        if kind is not None:
            assert (rows, min(parts, 2)) == kind, (c, rows, parts)


def test_listed_sizes_reach_every_variant():
    """Every kernel with both formats, plain and gated, and, of the smaller tiles,
    with scales as they stand and in another order. (K parts of 128 rows with
    scales in another order come with MXFP8 weights alone.)"""
    for (rows, parts), cases in TILES:
        have = {(c[3], c[4], rows < 256 and c[2] % 512 == 0) for c in cases}
        for fmt in ("MXFP4", "MXFP8"):
            for gated in (False, True):
                for in_place in ((False, True) if rows < 256 else (False,)):
                    if (rows, parts, fmt, in_place) != (128, 2, "MXFP4", False):
                        assert (fmt, gated, in_place) in have, (rows, parts, fmt, gated, in_place)
    wide = {(c[0] <= 16, c[1] <= 8192, c[4], c[5]) for c in FEW}
    assert len(wide) == 16


def test_workspace_of_a_call():
    """The size that is asked for without a call's arguments is that of the type
    of output which needs more; a call's own is 0 where it needs none."""
    import ctypes

    import mxfp4_precision_gemms_amd as A
    lib = A.lib()

    def own(m, N, K, fmt, gated=0, mx8=False, products=0):
        a = A.LinearArgs(m=m, N=N, K=K, b_format=fmt, gated=gated, products=products, out_scales=4096 if mx8 else None)
        return lib.adahop_linear_mx_args_workspace_size(ctypes.byref(a))

    for c in FEW + [c for _, cases in TILES for c in cases]:
        m, n, K, fmt, gated, mx8 = c
        f, N = int(fmt == "MXFP8"), 2 * n if gated else n
        both = [own(m, N, K, f, int(gated), t) for t in (False, True)]
        # (an MXFP8 output of few values is exact, and needs none)
        asked = lib.adahop_linear_mx_workspace_size(m, N, K, f, int(gated))
        assert both[mx8] in (0, asked) and (both[mx8] == 0) == (c in FEW)
        assert max(both) <= asked
        assert own(m, N, K, f, int(gated), mx8, products=2) == 0
    assert own(0, 64, 96, 1) == 0 and own(-1, 64, 96, 1) == 0 and own(4, 64, 80, 1) == 0 and own(4, 63, 96, 1, 1) == 0
    assert lib.adahop_linear_mx_args_workspace_size(None) == 0
    # bf16 from few rows of a layer whose MXFP8 output would take tiles
    assert lib.adahop_linear_mx_workspace_size(31, 3520, 1536, 1, 1) > 0 and own(31, 3520, 1536, 1, 1) == 0
