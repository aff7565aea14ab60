"""The pieces of the vocabulary that the cross entropy's gradient chooses: g, in
rows rounded up to a multiple of 64, is kept within 1 GiB. No GPU."""
import shutil
import subprocess

import pytest

from test_launch_shapes import CSRC
from test_xent_g_abi import size

GIB = 1 << 30
ROWS = (1, 63, 65, 1025, 4097, 8192, 100000, (1 << 20) - 63, 1 << 20, (1 << 20) + 1, (1 << 21) + 1, (1 << 22) - 1)
VOCABS = (1, 257, 32000, 130816, 131072, 500000, (1 << 23) + 5)


def pieces(tmp_path, cases):
    """(columns, count) of (rows, vocabulary, piece, numbers an element)."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text("\n".join(
        ["#include <cstdio>", '#include "tile_plan.h"', "using namespace adahop::tiles;", "int main() {"] +
        ["{ const XentPieces p = xent_pieces(%d, %d, %d, %d);"
         ' printf("%%lld %%lld\\n", (long long)p.size, (long long)p.count); }' % c for c in cases] + ["}", ""]))
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [[int(v) for v in line.split()] for line in out.split("\n")[:-1]]


def test_g_within_a_gib(tmp_path):
    cases = [(T, V, 0, terms) for T in ROWS for V in VOCABS for terms in (1, 2)]
    for (T, V, _, terms), (columns, count) in zip(cases, pieces(tmp_path, cases)):
        say = T, V, terms, columns, count
        column = 2 * terms * (-(-T // 64) * 64)
        most = max(GIB // column // 256 * 256, 256)
        whole = -(-V // 256) * 256
        assert columns % 256 == 0 and columns * column <= max(GIB, 256 * column), say
        assert (count - 1) * columns < V <= count * columns, say
        # no more pieces than need be, and the first no larger than it has to be
        assert count <= -(-whole // most) and columns - 256 < whole / -(-whole // most), say
        # what the call asks for is the chosen piece's
        if T * V < 1 << 46:
            kw = dict(rows=T, vocab=V, g=0 if terms == 2 else 1)
            assert size(**kw) == size(piece=columns, **kw), say


def test_pieces_that_are_asked_for(tmp_path):
    cases = [(T, V, piece, 2) for T in (1, 4097) for V in (1, 300, 70001) for piece in (1, 256, 257, 4096, 1 << 40)]
    for (T, V, piece, _), (columns, count) in zip(cases, pieces(tmp_path, cases)):
        assert columns == -(-min(piece, V) // 256) * 256 and (count - 1) * columns < V <= count * columns


@pytest.mark.parametrize("rows,vocab,g", [(4097, 130816, 0), (4097, 130816, 1), (1025, 500000, 0), (1025, 500000, 1)])
def test_workspace(rows, vocab, g):
    """g within 1 GiB, and the parts of dw's last round of tiles, at most 256 sums of
    256 x 256 tiles beside it."""
    assert size(rows=rows, vocab=vocab, g=g, dh=None, dim=4096, ld_h=4096, ld_w=4096, ld_dw=4096) <= GIB + 256 * (4 << 16)
