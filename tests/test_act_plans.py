"""What the activation operators plan for a shape, on the host: workspace sizes, and the weight
gradient's tiles."""
import ctypes
import math
import random

import pytest

from layer_wise_top_amd import lags

DTYPES = {"f32": (lags.LAGS_F32, 4), "bf16": (lags.LAGS_BF16, 2), "f16": (lags.LAGS_F16, 2)}


# Shapes of every tile of the weight gradient, with rows whole and in slices: ragged in the rows, outs
# and cols, and more than one tile.
TILES = ("256x256", "192x256", "128x128", "256x64", "64x256", "64x64")
WGRAD_SHAPES = {
    "f32": {"256x256": ((96, 25001, 401), (2093, 2812, 399)), "192x256": ((94, 21762, 257), (1094, 3659, 257)),
            "128x128": ((76, 25134, 65), (644, 2704, 69)), "64x256": ((78, 67, 16671), (669, 449, 321)),
            "64x64": ((73, 20, 69), (275, 22, 67))},
    "bf16": {"256x256": ((78, 26252, 385), (3117, 3004, 645)), "192x256": ((75, 519, 14482), (2517, 643, 1815)),
             "128x128": ((75, 22025, 131), (16775, 327, 20)), "256x64": ((79, 22341, 266), (14122, 400, 21)),
             "64x256": ((100, 261, 22198), (4681, 643, 711)), "64x64": ((71, 21, 67), (491, 21, 66))},
    "f16": {"256x256": ((75, 27121, 263), (2344, 1163, 1031)), "192x256": ((77, 21761, 259), (2049, 867, 887)),
            "128x128": ((76, 66, 25295), (1070, 1117, 257)), "256x64": ((72, 24821, 259), (1816, 8499, 21)),
            "64x256": ((84, 135, 16471), (1026, 129, 1968)), "64x64": ((73, 20, 67), (357, 65, 24))},
}


class WgradPlan(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_uint32), ("to", ctypes.c_uint32), ("tc", ctypes.c_uint32),
                ("split", ctypes.c_uint32), ("rows_per", ctypes.c_int64)]


def wgrad_plan(rows, outs, cols, dtype):
    """The library's own choice (lags::wgrad_plan, not part of the C ABI)."""
    f = lags.lib()._ZN4lags10wgrad_planEilll
    f.restype, f.argtypes = WgradPlan, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    return f(DTYPES[dtype][0], rows, outs, cols)


class GnPlan(ctypes.Structure):
    _fields_ = [("resident", ctypes.c_bool)] + [(k, ctypes.c_uint32) for k in (
        "threads", "rows", "w", "nslab", "tcl", "nchunk", "chunk", "nper", "nparts")]


def gn_plan(dtype, act, backward, n, s, c, groups):
    """The library's own choice (lags::gn_plan, not part of the C ABI)."""
    f = lags.lib()._ZN4lags7gn_planEiibmmjj
    f.restype = GnPlan
    f.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_bool, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32,
                  ctypes.c_uint32]
    return f(DTYPES[dtype][0], lags.ACTS[act], backward, n, s, c, groups)


# Samples that fill 8 and 13 register rows of a thread in both directions, vectors inside one group and
# cut by groups of three or five channels: (positions of 16-bit values, of fp32), channels, groups.
ROWS = {8: (500, 250), 13: (1500, 750)}
GROUPS = {"inside": (16, 2), "cut": (15, 5)}


def rows_case(dtype, rows, groups):
    c, g = GROUPS[groups]
    return 130, ROWS[rows][dtype == "f32"], c, g


def gn_bytes(n, s, c, g, dtype, act=2):
    shape = lags.GnShape(n, s, c, g, DTYPES[dtype][0], act, 1e-5)
    return int(lags.lib().lags_gn_workspace_bytes(ctypes.byref(shape)))


def log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))


def short_samples(rng):
    """Thousands of samples of one to four positions, groups up to the widest."""
    c = log_int(rng, 32, 4096)
    g = rng.choice([k for k in (1, 2, 3, 4, 8, 32) if c % k == 0])
    return rng.randrange(2000, 100000), rng.randrange(1, 5), c, g


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_group_norm_workspace_of_short_samples(dtype):
    """A workgroup adds up its samples' channel sums, so what is kept for the last sum is a fraction
    of the data: 8 bytes a channel of 1024 workgroups at most while a workgroup has under 32 rows (32
    MiB at the widest slab, 4096 channels), beyond that 8 bytes for every 32 values of a channel."""
    rng = random.Random(4)
    shapes = [(16384, 1, 2048, 1), (16384, 2, 2048, 1), (8192, 4, 1024, 32), (100000, 1, 64, 2)]
    shapes += [(16384, 1, 4096, 1), (16384, 1, 2500, 1), (4000, 4, 4096, 1), (4000, 3, 3001, 1)]
    shapes += [short_samples(rng) for _ in range(500)]
    for n, s, c, g in shapes:
        need, data = gn_bytes(n, s, c, g, dtype), n * s * c * DTYPES[dtype][1]
        assert 16 <= need <= max(8 * 1024 * 4096, data // 8) + 8 * c + 16, (n, s, c, g)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_group_norm_workspace_of_any_shape(dtype):
    """Below the data, or below the 32 MiB (and one slab's edge) that 1024 workgroups' channel sums
    take at the widest slab."""
    rng = random.Random(5)
    seen = 0
    while seen < 3000:
        c = log_int(rng, 1, 1 << 18)
        g = rng.choice([k for k in (1, 2, 3, 5, 8, 32, 64, c // 4, c // 2, c) if k and c % k == 0])
        n, s = log_int(rng, 1, 1 << 20), log_int(rng, 1, 1 << 20)
        need = gn_bytes(n, s, c, g, dtype)
        if not need:                    # groups wider than a slab
            continue
        seen += 1
        assert need <= max(8 * 1024 * 4096 + 8 * c, n * s * c * DTYPES[dtype][1]), (n, s, c, g)


def test_weight_gradient_that_is_not_sliced():
    """Slices of a dW above 2^32 values would take twice its bytes and more threads to add up than a
    launch has; below, a long product has them."""
    f = lags.lib().lags_ckpt_wgrad_workspace_bytes
    for rows, outs, cols, dtype in ((386292, 37480, 233212, 0), (1093745, 73993, 116331, 1), (604912, 65741, 132777, 2)):
        assert f(rows, outs, cols, dtype) == 16
    assert f(200704, 256, 64, 1) > 16


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_weight_gradient_shapes_of_every_tile(dtype):
    """The shapes that the GPU tests compute with take the tiles they are listed for, and no size takes
    a tile that is not listed."""
    for tile, shapes in WGRAD_SHAPES[dtype].items():
        for shape, sliced in zip(shapes, (False, True)):
            p = wgrad_plan(*shape, dtype)
            assert TILES[p.tile] == tile and (p.split > 1) == sliced, (shape, TILES[p.tile], p.split)
    rng = random.Random(6)
    seen = {TILES[wgrad_plan(log_int(rng, 1, 1 << 24), log_int(rng, 1, 1 << 22), log_int(rng, 1, 1 << 22), dtype).tile]
            for _ in range(50000)}
    assert seen == set(WGRAD_SHAPES[dtype])


@pytest.mark.parametrize("act", list(lags.ACTS))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_group_norm_shapes_of_every_row_count(dtype, act):
    """The shapes that the GPU tests compute with run resident, in the kernel of 8 or 13 rows."""
    for rows, least in ((8, 5), (13, 9)):
        for groups in GROUPS:
            for backward in (False, True):
                p = gn_plan(dtype, act, backward, *rows_case(dtype, rows, groups))
                assert p.resident and least <= p.rows <= rows, (dtype, act, rows, groups, backward, p.rows)
