"""What the activation operators plan for a shape, on the host: workspace sizes."""
import ctypes
import math
import random

import pytest

from layer_wise_top_amd import lags

DTYPES = {"f32": (lags.LAGS_F32, 4), "bf16": (lags.LAGS_BF16, 2), "f16": (lags.LAGS_F16, 2)}


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
