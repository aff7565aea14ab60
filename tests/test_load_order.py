"""The order in which the large tiles' kernel loads a stage of A, on which its waits
count: a slot's first half (loads 0 and 2) lands before the other (1 and 3) is waited
for. Nothing but a scheduling barrier keeps loads into different LDS objects in the
order that the source has them in, so outside the stages, whose own barriers
separate them, one stands between the halves. No GPU: it reads the source."""
import os
import re

from test_launch_shapes import CSRC


def test_halves_are_kept_apart():
    with open(os.path.join(CSRC, "bf16_tiles.h")) as f:
        lines = [re.sub(r"\s*//.*", "", ln).strip() for ln in f]
    lines = [ln for ln in lines if ln]
    second = [i for i, ln in enumerate(lines) if re.match(r"issue\([^;]*, Int<1>\{\}, \w+\);", ln)]
    assert len(second) == 2                          # bf16 operands' first stages, and codes'
    for i in second:
        assert lines[i - 1] == "__builtin_amdgcn_sched_barrier(0);", lines[i - 3:i + 1]
        assert re.match(r"issue\([^;]*, Int<2>\{\}, \w+\);", lines[i - 2])
