"""What a linear layer plans for a shape, on the host: tiles, slices of the summed index, and whether the
backward turns W round."""
import ctypes
import random

import pytest

from layer_wise_top_amd import lags

TILES = ((256, 256), (128, 128), (64, 64), (32, 128))
# (rows, cols, outs) whose product, forward or backward, is made of ragged tiles of each kind, whole and in
# slices; of 16-bit values and of fp32.  Keys: backward, tile, sliced, W turned round.
SHAPES = {
    "f32": {(0, 0, 0, 0): (7187, 340, 1991), (0, 0, 1, 0): (1367, 2886, 1483), (0, 1, 0, 0): (1700, 514, 1862),
            (0, 1, 1, 0): (716, 1564, 1470), (0, 2, 0, 0): (1, 16, 66), (0, 2, 1, 0): (1, 295, 68),
            (0, 3, 0, 0): (67, 17, 8685), (0, 3, 1, 0): (137, 413, 778), (1, 0, 0, 0): (3600, 4032, 359),
            (1, 0, 1, 0): (1228, 2438, 1896), (1, 1, 0, 0): (1968, 1546, 528), (1, 1, 1, 0): (1713, 592, 1561),
            (1, 2, 0, 0): (1, 65, 8), (1, 2, 1, 0): (1, 66, 304), (1, 3, 0, 0): (66, 8393, 11),
            (1, 3, 1, 0): (129, 778, 414)},
    "bf16": {(0, 0, 0, 0): (8196, 16, 963), (0, 0, 1, 0): (2692, 3279, 920), (0, 1, 0, 0): (321, 26, 8299),
             (0, 1, 1, 0): (579, 2889, 797), (0, 2, 0, 0): (1, 70, 65), (0, 2, 1, 0): (1, 700, 65),
             (0, 3, 0, 0): (33, 16, 8), (0, 3, 1, 0): (2, 643, 2744), (1, 0, 0, 0): (1036, 8701, 8),
             (1, 0, 0, 1): (8719, 1607, 1192), (1, 0, 1, 0): (3207, 432, 4151), (1, 0, 1, 1): (7553, 300, 5232),
             (1, 1, 0, 0): (6582, 929, 9), (1, 1, 0, 1): (5680, 519, 1376), (1, 1, 1, 0): (581, 1720, 2233),
             (1, 1, 1, 1): (8351, 277, 5096), (1, 2, 0, 0): (1, 65, 8), (1, 2, 0, 1): (1825, 323, 1288),
             (1, 2, 1, 0): (1, 65, 520), (1, 3, 0, 0): (66, 8393, 11), (1, 3, 1, 0): (792, 202, 919)},
}
SHAPES["f16"] = SHAPES["bf16"]
CASES = [(dtype, key, shape) for dtype, t in SHAPES.items() for key, shape in t.items()]


class LinPlan(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint32) for k in ("tile", "tm", "tn", "split", "k_per")] + [("turn", ctypes.c_bool)]


def linear_plan(dtype, backward, rows, cols, outs):
    """The library's own choice (lags::linear_plan, not part of the C ABI)."""
    f = lags.lib()._ZN4lags11linear_planEiblll
    f.restype, f.argtypes = LinPlan, [ctypes.c_int, ctypes.c_bool, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    code = {"f32": lags.LAGS_F32, "bf16": lags.LAGS_BF16, "f16": lags.LAGS_F16}[dtype]
    return f(code, bool(backward), rows, cols if backward else outs, outs if backward else cols)


@pytest.mark.parametrize("dtype,key,shape", CASES)
def test_shapes_take_every_path(dtype, key, shape):
    backward, tile, sliced, turn = key
    p = linear_plan(dtype, backward, *shape)
    assert (p.tile, p.split > 1, p.turn) == (tile, bool(sliced), bool(turn))


def test_tiles_and_slices_cover_the_product():
    """Any shape: tiles cover the outputs, slices are whole steps of 128 bytes that cover the sum, none
    empty, and the workspace holds what the plans write."""
    rng = random.Random(1)
    for _ in range(3000):
        dtype = rng.choice(["f32", "bf16", "f16"])
        rows, cols, outs = (int(2 ** rng.uniform(0, e)) for e in (15, 13, 13))
        step = 32 if dtype == "f32" else 64
        shape = lags.LinearShape(rows, cols, outs, {"f32": 0, "bf16": 1, "f16": 2}[dtype], 0)
        need = int(lags.lib().lags_linear_workspace_bytes(ctypes.byref(shape)))
        for back in (0, 1):
            p = linear_plan(dtype, back, rows, cols, outs)
            n, k = (cols, outs) if back else (outs, cols)
            bm, bn = TILES[p.tile]
            assert (p.tm - 1) * bm < rows <= p.tm * bm and (p.tn - 1) * bn < n <= p.tn * bn
            assert (p.split - 1) * p.k_per < k <= p.split * p.k_per and (p.split == 1 or p.k_per % step == 0)
            sums = 4 * p.split * rows * n if p.split > 1 else 0
            assert need >= sums + (2 * cols * outs if p.turn else 0)
            assert not p.turn or (back and dtype != "f32" and outs % 8 == 0)


# (rows, cols, outs): a large vocabulary's logits, sums split where an operand has more than 2^32 entries, and
# products whose tiles need more threads than one launch has
LARGE = [(16384, 1500, 262144), (32000, 2048, 151936), (20000, 8192, 262144), (65664, 512, 128256), (5546, 9, 774729),
         (11749, 368010, 1), (1 << 29, 8, 8), ((1 << 30) + 77, 1, 1), ((1 << 31) - 1, 2, 3)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_layers_are_taken(shape, dtype):
    code = {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    for rows in (shape[0], shape[0] - 1, 0):
        of = lags.LinearShape(rows, shape[1], shape[2], code, 0)
        need = int(lags.lib().lags_linear_workspace_bytes(ctypes.byref(of)))
        assert 16 <= need < 1 << 37, (rows, need)
