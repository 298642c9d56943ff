"""Which gradient kernel a size takes, on the CPU: the sizes that the GPU tests run reach every
tile of the table, in every kind of rows it is compiled for, split and unsplit."""
import ctypes
import os
import re

import pytest

import ternary_weight_linear_token_amd as bw
from ternary_weight_linear_token_amd import build as bw_build
from test_gpu_train_limits import DW_TILES, DX_TILES


def table():
    """(weight, tile rows, tile columns, groups, step) of each line of the table of tiles."""
    with open(os.path.join(bw_build.CSRC, "grad.hip")) as f:
        text = f.read()
    lines = text[text.index("constexpr GradCfg kCfg[] = {"):].split("};")[0]
    rows = re.findall(r"^    \{(\d), (\d+), (\d+), \d+, \d+, (\d), (\d+),", lines, re.M)
    assert len(rows) == lines.count("    {")
    return {(m == "0", int(bm), int(bn), int(g), int(bl)) for m, bm, bn, g, bl in rows}


def taken(M, K, Ns, weight=False):
    """The line of the table, the kind of rows (as launch_cfg picks it) and the slices."""
    bm, bn, g, slices = bw.grad_plan(M, K, Ns, weight)
    if weight:
        N, = Ns
        rows = "whole" if N % 2 == 0 else ("odd end" if N <= bm and M % 2 else "odd")
    else:
        rows = "whole" if K % 16 == 0 and all(n % 8 == 0 for n in Ns) else "odd"
    return (weight, bm, bn, g, bw.grad_plan_step(M, K, Ns, weight)), rows, slices


def test_gpu_sizes_reach_every_kernel():
    seen = set()
    for M, K, Ns in DX_TILES:
        line, rows, slices = taken(M, K, Ns)
        assert slices > 1, (M, K, Ns)
        seen.add((line, rows))
    for M, N, K in DW_TILES:
        line, rows, slices = taken(M, K, [N], weight=True)
        assert slices > 1, (M, N, K)
        seen.add((line, rows))
    want = {(line, rows) for line in table()
            for rows in ("whole", "odd") + (("odd end",) if line[0] else ())}
    assert seen == want
    assert len(table()) == 7


def test_plan_step_validation():
    L = bw.lib()
    n, two, out = (ctypes.c_int64 * 1)(16), (ctypes.c_int64 * 2)(16, 16), ctypes.c_int32(-1)
    f = lambda w, M, K, g, N, o=ctypes.byref(out): L.bitnet_grad_plan_step(w, M, K, g, N, o)
    assert f(0, 4, 256, 1, n) == 0 and out.value in (32, 64)
    assert f(0, 4, 256, 1, n, None) == 1 and f(0, 4, 256, 1, None) == 1
    assert f(0, 0, 256, 1, n) == 1 and f(1, 4, 256, 2, two) == 1 and f(0, 4, 250, 1, n) == 2
    assert f(0, 4, 256, 5, two) == 1 and f(0, (1 << 30) + 1, 256, 1, n) == 1
    with pytest.raises(bw.BitnetError):
        bw.grad_plan_step(4, 256, [16, 16], weight=True)
