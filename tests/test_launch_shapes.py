"""The launch shapes of the norm and linear layer's kernels, computed on the
host by the header that the kernels' launches use: no launch may have 2^32
threads or more in a dimension. No GPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_precision_gemms_amd", "csrc")


def evaluate(tmp_path, lines):
    """Output lines of a program made of statements that print."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "shapes.cpp", tmp_path / "shapes"
    src.write_text('#include <cstdio>\n#include <initializer_list>\n#include "launch_shapes.h"\nusing namespace adahop;\nint main() {\n'
                   + "\n".join(lines) + "\n}\n")
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
